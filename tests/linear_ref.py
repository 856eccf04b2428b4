"""The projection and its gradients in 64 bits.

Exactness: with small-integer operands every product and every partial sum is an integer below
2^24, which fp32 holds exactly in whatever order and with whatever truncation it is summed, so
without an activation the stored result is the exact value rounded once.

With an activation, z is exact and act(z) is a few fp32 operations on it: CUDA documents erff
within 2 ulp, expf 2, tanhf 2, division 0 beyond rounding.  Each form is 0.5 z (1 + f) or
z / (1 + e): |error| <= 16 EPS32 (|z| + 1) covers the argument's 4 roundings (amplified by at most
|z| f' <= 1) and the result's; its derivative likewise is within 32 EPS32 (|z| + 1)."""
import math

import torch

EPS32 = 2.0 ** -24


def rows(x):
    return x.transpose(0, 1).reshape(x.shape[1], -1) if x.dim() == 3 else x


def heads(y, n):
    return y.reshape(y.shape[0], n, -1).transpose(0, 1) if n else y


def act(z, a):
    if a == 1:
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if a == 2:
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if a == 3:
        return z * torch.sigmoid(z)
    return z


def act_grad(z, a):
    if a == 0:
        return torch.ones_like(z)
    with torch.enable_grad():
        z = z.clone().requires_grad_()
        g, = torch.autograd.grad(act(z, a).sum(), z)
    return g


def half(t):
    return torch.finfo(t).eps / 2
