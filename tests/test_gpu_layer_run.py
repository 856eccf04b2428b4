"""The layer's operators together, as a program calls them: projection to Q, K, V head-major,
norm and rotation, the sparse attention with every block selected, projection back with the
residual, and the gradients of all of it, against 64-bit autograd of the same layer.

Bounds are first-order sums of the stages' own bars, relative in the 2-norm: the attention's 1e-2
forward and backward (the bars its own tests use), and 2^-8 for every bf16 rounding on the path:
forward 1e-2 + 6 2^-8 (qkv, norm, O, y and the two operand copies), gradients 2 x 1e-2 + 10 2^-8."""
import pytest
import torch

import linear_ref
import norm_rope_ref as nref
from dynamic_block_sparse_indicator_b200 import _lib

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _run(x, Wqkv, b, wq, wk, Wo, dy, grid, H, D, rope):
    """Forward and backward on the GPU; returns y and the gradients."""
    T, Hh, W = grid
    N = T * Hh * W
    qkv, _, st = _lib.linear(x, Wqkv, b, out_heads=3 * H)
    q, k, v = qkv[:H], qkv[H:2 * H], qkv[2 * H:]
    qn, kn = _lib.qk_norm_rope(q, k, wq, wk, rope)
    prm = _lib.make_params(T, Hh, W, H, D, _lib.PRISM_BF16, top_k=1 << 20, top_p=1.0, eps=1e-4, out_dtype=_lib.PRISM_BF16)
    plan = _lib.plan(qn, kn, v, None, prm)
    O, lse = plan.attn_fwd()
    y, _, _ = _lib.linear(O, Wo, residual=x, status=st)
    dO, dWo, _, _ = _lib.linear_bwd(dy, O, Wo, want_db=False, status=st)
    dqkv = torch.empty_like(qkv)
    dqn, dkn, _ = plan.attn_bwd(dO, O, lse, dV=dqkv[2 * H:])
    _, _, dwq, dwk = _lib.qk_norm_rope_bwd(dqn, dkn, q, k, wq, wk, rope, dq=dqkv[:H], dk=dqkv[H:2 * H])
    dx, dWqkv, db, _ = _lib.linear_bwd(dqkv, x, Wqkv, status=st)
    assert plan.status() == _lib.PRISM_OK and _lib.status_read(st)[0] == _lib.PRISM_OK
    return y, dx.float() + dy.float(), dWqkv, db, dwq, dwk, dWo


def _exact(x, Wqkv, b, wq, wk, Wo, dy, grid, H, D, dims, pairing):
    leaves = [t.double().clone().requires_grad_() for t in (x, Wqkv, b, wq, wk, Wo)]
    x, Wqkv, b, wq, wk, Wo = leaves
    ang, ab = nref.angles(*grid, dims, 10000.0).cuda(), nref.pairs(dims, pairing)
    qkv = linear_ref.heads(x @ Wqkv.t() + b, 3 * H)
    q, k, v = qkv[:H], qkv[H:2 * H], qkv[2 * H:]

    def norm(t, w):
        u = t / ((t * t).mean(-1, keepdim=True) + 1e-6).sqrt() * w
        i, j = ab
        return u.index_copy(2, torch.tensor(i, device="cuda"), u[..., i] * ang.cos() - u[..., j] * ang.sin()).index_copy(
            2, torch.tensor(j, device="cuda"), u[..., i] * ang.sin() + u[..., j] * ang.cos())

    p = torch.softmax(norm(q, wq) @ norm(k, wk).transpose(1, 2) / D ** 0.5, -1)
    y = linear_ref.rows(p @ v) @ Wo.t() + x
    y.backward(dy.double())
    return (y.detach(), *(t.grad for t in (x, Wqkv, b, wq, wk, Wo)))


@pytest.mark.parametrize("D,dims,pairing", [(64, (24, 20, 20), 0), (128, (44, 42, 42), 1)])
def test_layer(D, dims, pairing, cuda_device):
    grid, H, F = (8, 8, 16), 2, 192
    N = grid[0] * grid[1] * grid[2]
    g = torch.Generator("cuda").manual_seed(D)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
    x, dy = rnd(N, F).to(BF), rnd(N, F).to(BF)
    Wqkv, Wo = rnd(3 * H * D, F, std=F ** -0.5).to(BF), rnd(F, H * D, std=(H * D) ** -0.5).to(BF)
    b, wq, wk = rnd(3 * H * D, std=0.1), 1 + rnd(D, std=0.2), 1 + rnd(D, std=0.2)
    rope = _lib.make_rope(*grid, dims, 10000.0, pairing)
    got = _run(x, Wqkv, b, wq, wk, Wo, dy, grid, H, D, rope)
    want = _exact(x, Wqkv, b, wq, wk, Wo, dy, grid, H, D, dims, pairing)
    for name, a, e in zip(("y", "dx", "dWqkv", "db", "dwq", "dwk", "dWo"), got, want):
        bar = 1e-2 + 6 / 256 if name == "y" else 2e-2 + 10 / 256
        rel = float((a.double() - e).norm() / e.norm())
        assert rel <= bar, f"{name}: {rel:.3e} > {bar:.3e}"
    again = _run(x, Wqkv, b, wq, wk, Wo, dy, grid, H, D, rope)
    assert torch.equal(got[0], again[0]) and torch.equal(got[6], again[6])
