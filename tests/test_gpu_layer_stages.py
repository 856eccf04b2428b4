"""The layer's operators together, stage by stage: each result against 64 bits of what the stage was given
on the GPU, so that a stage's own error has a bound of half a step instead of the whole layer's bar.
(test_gpu_layer_run compares the layer from end to end.)"""
import pytest
import torch

import linear_ref
import norm_rope_ref as nref
from dynamic_block_sparse_indicator_b200 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
H_ = linear_ref.half(BF)


def _product(got, a, b, bias, res, what):
    """got = a b^T + bias + res of a [M, K], b [N, K] in bf16: the sums lose at most a unit of 2^-23 of the
    terms' size at each step of 16 and chunk, bias and residual and the stored type half a step each."""
    a, b = linear_ref.rows(a).double(), b.double()
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    for t in (bias, res):
        if t is not None:
            want, mag = want + t.double(), mag + t.double().abs()
    err = (a.shape[1] / 16 + a.shape[1] / 768 + 4) * 2 * linear_ref.EPS32 * mag
    h = linear_ref.half(got.dtype)
    bad = ~((linear_ref.rows(got).double() - want).abs() <= h * want.abs() + (1 + h) * err)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} values off"


def _norm(got, x, w, ang, ab, what):
    want, m = nref.forward(x.cpu(), w.cpu(), ang, ab, 1e-6)
    bad = ~((got.cpu().double() - want).abs() <= H_ * want.abs() + (1 + H_) * 16 * nref.EPS32 * m)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} values off"


@pytest.mark.parametrize("grid,H,D,F,dims,pairing", [((8, 8, 16), 3, 64, 200, (24, 20, 20), 0),
                                                     ((8, 16, 16), 5, 128, 640, (44, 42, 42), 1),
                                                     ((8, 8, 16), 2, 128, 330, (32, 48, 48), 1)])
def test_stages(grid, H, D, F, dims, pairing, cuda_device):
    N = grid[0] * grid[1] * grid[2]
    g = torch.Generator("cuda").manual_seed(F)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std
    x, dy = rnd(N, F).to(BF), rnd(N, F).to(BF)
    Wqkv, Wo = rnd(3 * H * D, F, std=F ** -0.5).to(BF), rnd(F, H * D, std=(H * D) ** -0.5).to(BF)
    b, wq, wk = rnd(3 * H * D, std=0.1), 1 + rnd(D, std=0.2), 1 + rnd(D, std=0.2)
    rope = _lib.make_rope(*grid, dims, 10000.0, pairing)
    ang, ab = nref.angles(*grid, dims, 10000.0), nref.pairs(dims, pairing)

    qkv, _, st = _lib.linear(x, Wqkv, b, out_heads=3 * H)
    _product(qkv, x, Wqkv, b, None, "qkv")
    q, k, v = qkv[:H], qkv[H:2 * H], qkv[2 * H:]
    qn, kn = _lib.qk_norm_rope(q, k, wq, wk, rope)
    _norm(qn, q, wq, ang, ab, "q")
    _norm(kn, k, wk, ang, ab, "k")
    prm = _lib.make_params(*grid, H, D, _lib.PRISM_BF16, top_k=1 << 20, top_p=1.0, eps=1e-4, out_dtype=_lib.PRISM_BF16)
    plan = _lib.plan(qn, kn, v, None, prm)
    O, lse = plan.attn_fwd()
    y, _, _ = _lib.linear(O, Wo, residual=x, status=st)
    _product(y, O, Wo, None, x, "y")

    dO, dWo, _, _ = _lib.linear_bwd(dy, O, Wo, want_db=False, status=st)
    _product(dO, dy, Wo.t(), None, None, "dO")
    _product(dWo, dy.t(), linear_ref.rows(O).t(), None, None, "dWo")
    dqkv = torch.empty_like(qkv)
    dqn, dkn, _ = plan.attn_bwd(dO, O, lse, dV=dqkv[2 * H:])
    _, _, dwq, dwk = _lib.qk_norm_rope_bwd(dqn, dkn, q, k, wq, wk, rope, dq=dqkv[:H], dk=dqkv[H:2 * H])
    for got, dw, gy, t, w, n in ((dqkv[:H], dwq, dqn, q, wq, "dq"), (dqkv[H:2 * H], dwk, dkn, k, wk, "dk")):
        want, m, sums, mag = nref.backward(gy.cpu(), t.cpu(), w.cpu(), ang, ab, 1e-6)
        bad = ~((got.cpu().double() - want).abs() <= H_ * want.abs() + (1 + H_) * nref.EPS32 * m)
        assert not bool(bad.any()), f"{n}: {int(bad.sum())} of {bad.numel()} values off"
        assert bool(((dw.cpu().double() - sums).abs() <= (48 + H) * nref.EPS32 * mag).all()), n + " weight"
    dx, dWqkv, db, _ = _lib.linear_bwd(dqkv, x, Wqkv, status=st)
    rows = linear_ref.rows(dqkv)
    _product(dx, dqkv, Wqkv.t(), None, None, "dx")
    _product(dWqkv, rows.t(), x.t(), None, None, "dWqkv")
    sums = rows.double().sum(0)
    assert bool(((db.double() - sums).abs() <= (N / 8 + 16) * linear_ref.EPS32 * rows.double().abs().sum(0)).all())
    assert plan.status() == _lib.PRISM_OK and _lib.status_read(st)[0] == _lib.PRISM_OK
