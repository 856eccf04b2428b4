"""The per-head norm with rotation and its gradients in 64 bits, with the error bounds of a
32-bit evaluation: EPS32 = 2^-24 is half a step of fp32.

Forward, u = x r w with r = rsqrt(mean x^2 + eps): a row's sum of squares takes at most 8 fused
adds in a lane and 4 across lanes, one product and one sum more (14 roundings, halved by the
root), rsqrtf is within 2 ulp (4 half steps), x r w takes 2: u is within 13 half steps; the
rotation adds 2 and the table's rounding 1: y is within 16 EPS32 (|u_a c| + |u_b s|).  Folded as
r (x_a w_a c + x_b w_b s) it is the table's 1, products 2, sum 1, r's 11 and its product 1: the same 16.

Gradients: v = R^T g is within 3 EPS32 (|g_a c| + |g_b s|) =: 3 EPS32 V.  dot = sum w v x over D
channels: 12 sums, 2 products and v's 3: within 17 EPS32 sum w V |x|.  r is within 11, so
k = dot r^2 / D is within 17 + 22 + 3 = 42, k x within 43; dx = r (w v - k x) adds 4 + 1 + 1 and
r's 11 to either part: within 64 EPS32 r (w V + r^2 |x| mean(w V |x|)).
dw: a term is within 3 + 11 + 2 = 16, a lane adds one row per head of its block, a block its
rows (at most 32): (48 + heads) EPS32 sum V |x| r, while no lane walks more than one tile.
"""
import torch

EPS32 = 2.0 ** -24


def pairs(dims, pairing):
    a, b, base = [], [], 0
    for d in dims:
        for p in range(d // 2):
            a.append(base + (2 * p if pairing == 0 else p))
            b.append(base + (2 * p + 1 if pairing == 0 else p + d // 2))
        base += d
    return a, b


def angles(T, H, W, dims, theta, first=0):
    n = torch.arange(T * H * W)
    cols = []
    for pos, d in ((n // (H * W) + first, dims[0]), (n // W % H, dims[1]), (n % W, dims[2])):
        for p in range(d // 2):
            cols.append(pos.double() * theta ** (-2.0 * p / d))
    return torch.stack(cols, 1) if cols else torch.zeros(T * H * W, 0, dtype=torch.float64)


def turn(u, ang, ab, sign=1.0):
    """(R u, |u_a c| + |u_b s|) channel by channel (R^T for sign -1)."""
    a, b = ab
    c, s = ang.cos(), sign * ang.sin()
    y, m = u.clone(), u.abs().clone()
    y[..., a] = u[..., a] * c - u[..., b] * s
    y[..., b] = u[..., a] * s + u[..., b] * c
    m[..., a] = (u[..., a] * c).abs() + (u[..., b] * s).abs()
    m[..., b] = (u[..., a] * s).abs() + (u[..., b] * c).abs()
    return y, m


def forward(x, w, ang, ab, eps):
    x = x.double()
    r = 1 / ((x * x).mean(-1, keepdim=True) + eps).sqrt()
    u = x * r * (1 if w is None else w.double())
    return turn(u, ang, ab)


def backward(g, x, w, ang, ab, eps):
    """dx, its bound in EPS32 units, dw, its magnitude sum."""
    g, x = g.double(), x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    r = 1 / ((x * x).mean(-1, keepdim=True) + eps).sqrt()
    v, V = turn(g, ang, ab, -1.0)
    dw, mag = (v * x * r).sum((0, 1)), (V * x.abs() * r).sum((0, 1))
    dx = r * (w * v - x * r * r * (w * v * x).mean(-1, keepdim=True))
    M = r * (w.abs() * V + r * r * x.abs() * (w.abs() * V * x.abs()).mean(-1, keepdim=True))
    return dx, 64 * M, dw, mag
