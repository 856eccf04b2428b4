"""The projection and its gradients in 64 bits.

Exactness: with small-integer operands every product and every partial sum is an integer below
2^24, which fp32 holds exactly in whatever order and with whatever truncation it is summed, so
without an activation the stored result is the exact value rounded once.

With an activation, z is exact and act(z) is a few fp32 operations on it: CUDA documents
__expf(t) within 2 + 1.173 |t| ulp and __fdividef within 2 ulp.  z Phi(z): the formula is within
0.75e-7 = 1.3 EPS32 of Phi, and its evaluation, q e^(-x^2) / 2 with q <= 1 and x^2 e^(-x^2) <= 0.37, adds
at most (2 (2 + 1.173 0.37) + 4) / 2 EPS32 by the power and 8 by quotient and polynomial: within 16 EPS32 (|z| + 1).
z s with s = 1 / (1 + e^-t): e's relative error 2 EPS32 (2 + 1.173 |t|) and the argument's 4 roundings
(4 |t| EPS32) reach s by the factor s (1 - s), and s (1 - s) |t| < 0.23, s (1 - s) <= 0.25: at most
(1 + 0.6 + 0.9) EPS32, the quotient adds 4 EPS32 s and the product 1: within 16 EPS32 (|z| + 1).
The derivative s + z s (1 - s) t' has |z t'| s (1 - s) < 2 and multiplies one more such s: within
32 EPS32 (|z| + 1).  (Its power is ex2.approx of t log2 e and its quotient rcp.approx, within 2 and
1 ulp: no more than the above.)"""
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
