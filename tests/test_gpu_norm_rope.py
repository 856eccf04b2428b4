"""The per-head norm with rotation and its gradients on the GPU, against 64 bits.

Tolerances are norm_rope_ref's bounds plus half a step of the stored type; none is fitted."""
import pytest
import torch

import norm_rope_ref as ref
from dynamic_block_sparse_indicator_b200 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS, THETA = 1e-6, 10000.0

# name: (T, H, W), heads, D, in dtype, out dtype, weight dtype (None: none), layout, pairing, dims
CASES = {
    "one_token": ((1, 1, 1), 1, 128, BF, BF, F32, "heads", 0, (44, 42, 42)),
    "one_token_40_heads_fused": ((1, 1, 1), 40, 128, BF, BF, F32, "fused", 1, (44, 42, 42)),
    "two_tokens_d64": ((2, 1, 1), 3, 64, BF, BF, BF, "fused", 1, (64, 0, 0)),
    "seventeen_1d": ((17, 1, 1), 2, 128, BF, BF, F32, "padded", 0, (128, 0, 0)),
    "grid_5x7x9": ((5, 7, 9), 5, 128, BF, BF, F32, "fused", 0, (44, 42, 42)),
    "grid_5x7x9_halves": ((5, 7, 9), 5, 128, BF, BF, F32, "fused", 1, (44, 42, 42)),
    "grid_3x11x13_partial": ((3, 11, 13), 7, 64, BF, F32, BF, "heads", 1, (16, 8, 8)),
    "no_time_axis": ((1, 16, 24), 4, 64, F32, F32, F32, "padded", 0, (0, 32, 32)),
    "fp32_to_bf16": ((4, 5, 6), 3, 128, F32, BF, F32, "fused", 0, (32, 48, 48)),
    "fp32_halves": ((4, 5, 6), 3, 128, F32, F32, None, "heads", 1, (32, 48, 48)),
    "lanes_1d": ((37, 1, 1), 5, 128, BF, BF, F32, "fused", 1, (128, 0, 0)),
    "lanes_grid": ((3, 7, 11), 5, 128, BF, BF, BF, "heads", 1, (32, 48, 48)),
    "lanes_d64_fp32": ((5, 3, 7), 3, 64, F32, F32, F32, "padded", 1, (32, 16, 0)),
    "lanes_no_time_axis": ((1, 6, 9), 2, 128, BF, F32, F32, "heads", 1, (0, 64, 48)),
    "two_channels": ((9, 1, 2), 2, 64, F32, F32, BF, "heads", 1, (2, 0, 0)),
    "nothing_rotated": ((6, 5, 4), 2, 64, BF, BF, F32, "heads", 0, (0, 0, 0)),
    "far_positions": ((40000, 1, 1), 1, 64, F32, F32, F32, "heads", 0, (64, 0, 0)),
    "odd_tokens_many_heads": ((33, 1, 31), 23, 64, BF, BF, F32, "fused", 0, (24, 20, 20)),
}


def _make(shape, dtype, layout, gen, scale=1.0):
    """A [heads, N, D] view of the layout."""
    heads, N, D = shape
    if layout == "fused":
        x = torch.randn(N, 3, heads, D, generator=gen).mul(scale).to(dtype).cuda()
        return x[:, 1].transpose(0, 1)
    if layout == "padded":
        x = torch.randn(N, heads, D + 16, generator=gen).mul(scale).to(dtype).cuda()
        return x[:, :, 8:8 + D].transpose(0, 1)
    return torch.randn(heads, N, D, generator=gen).mul(scale).to(dtype).cuda()


def _case(name, seed=0):
    (T, H, W), heads, D, it, ot, wt, layout, pairing, dims = CASES[name]
    g = torch.Generator().manual_seed(seed + 1000)
    N = T * H * W
    q, k = (_make((heads, N, D), it, layout, g, s) for s in (1.0, 3.0))
    ws = [None if wt is None else (1 + 0.3 * torch.randn(D, generator=g)).to(wt).cuda() for _ in range(2)]
    dy = [torch.randn(heads, N, D, generator=g).to(ot).cuda() for _ in range(2)]
    rope = _lib.make_rope(T, H, W, dims, THETA, pairing)
    return q, k, ws, dy, rope, ref.angles(T, H, W, dims, THETA), ref.pairs(dims, pairing), ot


def _half(t):
    return torch.finfo(t).eps / 2


def _within(got, want, tol, what):
    err = (got.detach().double().cpu() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float((err / tol.clamp_min(1e-300)).max()):.2f} of the bound"


@pytest.mark.parametrize("name", list(CASES))
def test_forward(name, cuda_device):
    q, k, ws, _, rope, ang, ab, ot = _case(name)
    qo, ko = _lib.qk_norm_rope(q, k, *ws, rope, eps=EPS, out_dtype=ot)
    for got, x, w, n in ((qo, q, ws[0], "q"), (ko, k, ws[1], "k")):
        assert got.dtype == ot and got.is_contiguous()
        y, m = ref.forward(x.cpu(), None if w is None else w.cpu(), ang, ab, EPS)
        _within(got, y, _half(ot) * y.abs() + (1 + _half(ot)) * 16 * ref.EPS32 * m, n)


@pytest.mark.parametrize("name", list(CASES))
def test_gradients(name, cuda_device):
    q, k, ws, dy, rope, ang, ab, ot = _case(name, 1)
    dq, dk, dwq, dwk = _lib.qk_norm_rope_bwd(*dy, q, k, *ws, rope, eps=EPS)
    for got, gw, x, w, g, n in ((dq, dwq, q, ws[0], dy[0], "dq"), (dk, dwk, k, ws[1], dy[1], "dk")):
        assert got.dtype == x.dtype
        dx, m, dw, mag = ref.backward(g.cpu(), x.cpu(), None if w is None else w.cpu(), ang, ab, EPS)
        h = _half(x.dtype)
        _within(got, dx, h * dx.abs() + (1 + h) * ref.EPS32 * m, n)
        assert (gw is None) == (w is None)
        if gw is not None:
            tiles = -(-x.shape[1] // 16)
            walked = -(-tiles // 592)            # tiles that one block walks at most
            _within(gw, dw, (48 + walked * x.shape[0]) * ref.EPS32 * mag, n + " weight")


@pytest.mark.parametrize("name", ["grid_5x7x9", "fp32_halves", "grid_3x11x13_partial", "lanes_grid"])
def test_gradients_against_differences(name, cuda_device):
    """<dx, d> and <dw, e> against central differences of the 64-bit forward."""
    q, k, ws, dy, rope, ang, ab, ot = _case(name, 2)
    dq, _, dwq, _ = _lib.qk_norm_rope_bwd(*dy, q, k, *ws, rope, eps=EPS)
    x, g = q.cpu().double(), dy[0].cpu().double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if ws[0] is None else ws[0].cpu().double()
    gen = torch.Generator().manual_seed(7)
    d = torch.randn(x.shape, generator=gen, dtype=torch.float64)
    f = lambda xx, ww: float((ref.forward(xx, ww, ang, ab, EPS)[0] * g).sum())
    h = 1e-5
    want = (f(x + h * d, w) - f(x - h * d, w)) / (2 * h)
    _, m, _, mag = ref.backward(dy[0].cpu(), q.cpu(), None if ws[0] is None else ws[0].cpu(), ang, ab, EPS)
    half = _half(q.dtype)
    # the difference's own error: h^2 times a third derivative of order |dx| / r^2-scale, and rounding of f / h
    slack = 1e-6 * float((m / 64).mul(d.abs()).sum())
    tol = float(((half * dq.cpu().double().abs() * 2 + (1 + half) * ref.EPS32 * m) * d.abs()).sum()) + slack
    assert abs(float((dq.cpu().double() * d).sum()) - want) <= tol
    if dwq is not None:
        e = torch.randn(w.shape, generator=gen, dtype=torch.float64)
        want = (f(x, w + h * e) - f(x, w - h * e)) / (2 * h)
        tol = (60 + x.shape[0]) * ref.EPS32 * float((mag * e.abs()).sum()) + 1e-6 * float((mag * e.abs()).sum())
        assert abs(float((dwq.cpu().double() * e).sum()) - want) <= tol


def test_query_alone_no_rotation_no_weight(cuda_device):
    q, *_ = _case("grid_5x7x9")
    qo, ko = _lib.qk_norm_rope(q)
    assert ko is None
    y, m = ref.forward(q.cpu(), None, torch.zeros(q.shape[1], 0, dtype=torch.float64), ([], []), EPS)
    _within(qo, y, _half(BF) * y.abs() + (1 + _half(BF)) * 16 * ref.EPS32 * m, "q")
    dq, dk, dwq, dwk = _lib.qk_norm_rope_bwd(qo, None, q)
    assert dk is None and dwq is None and dwk is None and dq.shape == q.shape


def test_no_tokens(cuda_device):
    q = torch.empty(3, 0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    qo, ko = _lib.qk_norm_rope(q, q, w, w)
    assert qo.shape == (3, 0, 64)
    _, _, dwq, dwk = _lib.qk_norm_rope_bwd(qo, ko, q, q, w, w)
    assert float(dwq.abs().sum()) == 0.0 and float(dwk.abs().sum()) == 0.0


@pytest.mark.parametrize("pairing", [0, 1])
def test_in_place_and_surroundings(pairing, cuda_device):
    """In place through a fused buffer: V's slice and the padding keep their bits, the result's
    equal those of the call into memory of its own; the gradients likewise over dq_out and over q."""
    g = torch.Generator().manual_seed(3)
    heads, T, H, W, D = 3, 3, 5, 7, 128
    buf = torch.randn(T * H * W, 3, heads, D, generator=g).to(BF).cuda()
    w = torch.randn(D, generator=g).cuda()
    rope = _lib.make_rope(T, H, W, (44, 42, 42), THETA, pairing)
    q, k = buf[:, 0].transpose(0, 1), buf[:, 1].transpose(0, 1)
    v0 = buf[:, 2].clone()
    x0, k0 = q.contiguous(), k.contiguous()
    want = _lib.qk_norm_rope(q, k, w, w, rope)
    dy = torch.randn(heads, T * H * W, D, generator=g).to(BF).cuda()
    grads = _lib.qk_norm_rope_bwd(dy, dy, x0, k0, w, w, rope)
    got = _lib.qk_norm_rope(q, k, w, w, rope, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(buf[:, 2], v0)
    d1, d2 = dy.clone(), dy.clone()
    ing = _lib.qk_norm_rope_bwd(d1, d2, x0, k0, w, w, rope, dq=d1, dk=d2)
    over = _lib.qk_norm_rope_bwd(dy, dy, x0, k0, w, w, rope, dq=x0, dk=k0)
    for a, b, c in zip(ing, over, grads):
        assert torch.equal(a, c) and torch.equal(b, c)


def test_bad_values_stay_in_their_row(cuda_device):
    q, _, ws, dy, rope, *_ = _case("grid_5x7x9_halves")
    clean, _ = _lib.qk_norm_rope(q, None, ws[0], None, rope)
    dclean = _lib.qk_norm_rope_bwd(dy[0], None, q, None, ws[0], None, rope)[0]
    bad = q.clone()
    bad[2, 11, 5] = float("nan")
    bad[1, 200, 100] = float("inf")
    bad[0, 3] = 0.0
    got, _ = _lib.qk_norm_rope(bad, None, ws[0], None, rope)
    dgot = _lib.qk_norm_rope_bwd(dy[0], None, bad, None, ws[0], None, rope)[0]
    keep = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    keep[2, 11] = keep[1, 200] = keep[0, 3] = False
    assert torch.equal(got[keep], clean[keep]) and torch.equal(dgot[keep], dclean[keep])
    assert bool((got[0, 3] == 0).all()) and bool(torch.isfinite(dgot[0, 3]).all())
    assert bool(torch.isnan(got[2, 11]).any())


def test_same_bits_twice_and_under_a_graph(cuda_device):
    q, k, ws, dy, rope, *_ = _case("odd_tokens_many_heads")
    qc, kc = q.clone(), k.clone()
    first = (*_lib.qk_norm_rope(qc, kc, *ws, rope), *_lib.qk_norm_rope_bwd(*dy, qc, kc, *ws, rope))
    again = (*_lib.qk_norm_rope(qc, kc, *ws, rope), *_lib.qk_norm_rope_bwd(*dy, qc, kc, *ws, rope))
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = (*_lib.qk_norm_rope(qc, kc, *ws, rope), *_lib.qk_norm_rope_bwd(*dy, qc, kc, *ws, rope))
    qc.mul_(-2)          # other inputs in the captured places
    graph.replay()
    torch.cuda.synchronize()
    want = (*_lib.qk_norm_rope(qc, kc, *ws, rope), *_lib.qk_norm_rope_bwd(*dy, qc, kc, *ws, rope))
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_on_another_stream(cuda_device):
    q, k, ws, _, rope, *_ = _case("grid_5x7x9")
    want = _lib.qk_norm_rope(q, k, *ws, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _lib.qk_norm_rope(q, k, *ws, rope, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_past_32_bits(cuda_device):
    """2.2e9 elements (4.4 GB): the last rows equal those of a small call on them."""
    heads, N, D = 34, 505_001, 128
    x = torch.empty(heads, N, D, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    rope = _lib.make_rope(N, 1, 1, (128, 0, 0))
    y, _ = _lib.qk_norm_rope(x, None, w, None, rope)
    tail = _lib.make_rope(1000, 1, 1, (128, 0, 0), first_frame=N - 1000)
    want, _ = _lib.qk_norm_rope(x[-1:, -1000:], None, w, None, tail)
    assert torch.equal(y[-1:, -1000:], want)
    dx, _, dw, _ = _lib.qk_norm_rope_bwd(y, None, x, None, w, None, rope)
    dwant, *_ = _lib.qk_norm_rope_bwd(y[-1:, -1000:], None, x[-1:, -1000:], None, w, None, tail)
    assert torch.equal(dx[-1:, -1000:], dwant)
    assert bool(torch.isfinite(dw).all())


def test_rotation_table(cuda_device):
    """Each entry within half a step (and the 64-bit functions' own error) of the 64-bit value."""
    T, H, W, dims, first = 500, 9, 31, (44, 42, 42), 123_456
    tab = _lib.make_rope(T, H, W, dims, 10000.0, 0, first_frame=first).table.cpu().double()
    want = []
    for L, d, f in ((T, dims[0], first), (H, dims[1], 0), (W, dims[2], 0)):
        ang = (torch.arange(L).double() + f)[:, None] * 10000.0 ** (-torch.arange(0, d, 2).double() / d)
        want.append(torch.stack([ang.cos(), ang.sin()], -1).reshape(-1))
    want = torch.cat(want)
    # the angle itself (up to 1.2e5) carries a few 2^-53 relative: 1.2e5 * 4 * 2^-53 < 2^-33
    assert bool(((tab - want).abs() <= ref.EPS32 * want.abs() + 2.0 ** -33).all())


def test_refusals_on_the_device(cuda_device):
    x = torch.zeros(2, 40, 64, dtype=BF, device="cuda")
    big = torch.zeros(2, 40, 65, dtype=BF, device="cuda")
    rope = _lib.make_rope(40, 1, 1, (64, 0, 0))
    for call in (lambda: _lib.qk_norm_rope(big[:, :, :64]),                                   # rows off 16 bytes
                 lambda: _lib.qk_norm_rope(torch.zeros(2, 40, 96, dtype=BF, device="cuda")),  # head_dim
                 lambda: _lib.qk_norm_rope(x, eps=0.0),
                 lambda: _lib.qk_norm_rope(x[:, 1:], q_out=x[:, :-1]),                        # overlap
                 lambda: _lib.qk_norm_rope(x, x, q_out=x, k_out=x),                           # one result twice
                 lambda: _lib.qk_norm_rope(x[:1], q_out=x[:1, :1].expand(1, 40, 64)),         # rows onto each other
                 lambda: _lib.qk_norm_rope_bwd(x, None, x, None, torch.ones(64, device="cuda"),
                                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(_lib.PrismError):
            call()
    for call in (lambda: _lib.qk_norm_rope(x, x[:, :39]),
                 lambda: _lib.qk_norm_rope(x[:, :39], None, None, None, rope),
                 lambda: _lib.qk_norm_rope(x.half()),
                 lambda: _lib.qk_norm_rope(x, None, torch.ones(63, device="cuda")),
                 lambda: _lib.qk_norm_rope(x, None, None, torch.ones(64, device="cuda")),
                 lambda: _lib.qk_norm_rope(x.transpose(1, 2)),
                 lambda: _lib.qk_norm_rope(x, x.float()),
                 lambda: _lib.qk_norm_rope_bwd(x, None, x, x),
                 lambda: _lib.qk_norm_rope(x, None, torch.ones(64))):
        with pytest.raises(ValueError):
            call()


def test_table_on_another_stream_takes_no_memory_in_use(cuda_device):
    """A table made on a stream is not laid over a freed tensor that the current stream still writes."""
    T, H, W, dims = 7, 30, 52, (44, 42, 42)
    want = _lib.make_rope(T, H, W, dims).table.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    old = torch.empty_like(want)
    for _ in range(200):                 # (the current stream is behind)
        old.fill_(7.0)
    del old
    rope = _lib.make_rope(T, H, W, dims, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(rope.table, want)
