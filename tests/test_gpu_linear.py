"""The projections on the GPU against 64 bits: exact where small integers make them so (see
linear_ref), within counted roundings otherwise."""
import pytest
import torch

import linear_ref as ref
from dynamic_block_sparse_indicator_b200 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NONE, GELU, TANH, SILU = 0, 1, 2, 3


def _ints(shape, gen, hi=4, dtype=BF):
    return torch.randint(-hi, hi + 1, shape, generator=gen, device="cuda").to(dtype)


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _ok(status):
    st, site = _lib.status_read(status)
    assert st == _lib.PRISM_OK, f"device status {_lib.status_string(st)} at site {site}"


def _x(M, K, in_heads, stride, gen, hi=4):
    if in_heads:
        return _ints((in_heads, M, K // in_heads), gen, hi)
    return _ints((M, K + stride), gen, hi)[:, :K]


# name: M, K, N, in_heads, out_heads, x stride pad, W stride pad, y stride pad
SHAPES = {
    "one_by_one": (1, 1, 1, 0, 0, 0, 0, 0),
    "one_token": (1, 5120, 640, 0, 0, 0, 0, 0),
    "one_token_odd": (1, 203, 77, 0, 0, 0, 0, 0),
    "one_token_heads": (1, 256, 384, 2, 3, 0, 0, 0),
    "tokens_13_split8": (13, 4224, 256, 0, 0, 0, 0, 0),
    "tokens_16_exact_tile": (16, 512, 128, 0, 0, 0, 0, 0),
    "tokens_17": (17, 640, 320, 0, 0, 8, 0, 0),
    "tokens_33_ragged": (33, 1000, 129, 0, 0, 0, 0, 3),
    "tokens_64_heads": (64, 1280, 640, 10, 5, 0, 0, 0),
    "tokens_65": (65, 72, 200, 0, 0, 0, 0, 0),
    "tokens_127_odd_k": (127, 331, 257, 0, 0, 0, 0, 0),
    "tokens_200_padded": (200, 264, 136, 0, 0, 24, 16, 8),
    "odd_strides": (150, 96, 96, 0, 0, 3, 5, 1),
    "mid_many_tiles": (1000, 384, 2304, 0, 0, 0, 0, 0),
    "pairs_exact": (2560, 128, 2048, 0, 0, 0, 0, 0),
    "pairs_ragged": (2571, 200, 2120, 0, 0, 0, 0, 0),
    "pairs_heads": (2571, 640, 1920, 10, 15, 0, 0, 0),
    "pairs_odd": (2571, 203, 2121, 0, 0, 0, 0, 0),
    "pairs_chunks": (2500, 5000, 2000, 0, 0, 0, 0, 0),
    "tiles_192": (520, 640, 4160, 0, 0, 0, 0, 0),
    "tiles_192_ragged_heads": (500, 320, 5120, 5, 40, 0, 0, 0),
    "tiles_128": (300, 256, 6400, 0, 0, 0, 0, 0),
    "single_split8": (300, 8192, 300, 0, 0, 0, 0, 0),
    "single_no_split": (70, 72, 260, 0, 0, 0, 0, 0),
    "pairs_long": (2560, 17000, 2050, 0, 0, 0, 0, 0),
    "pairs_one_column_tile": (20000, 64, 130, 0, 0, 0, 0, 0),
}


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_forward_exact(name, out, cuda_device):
    M, K, N, ih, oh, xs, ws, ys = SHAPES[name]
    g = _gen(1)
    x, W, b = _x(M, K, ih, xs, g), _ints((N, K + ws), g)[:, :K], _ints((N,), g, 9, F32)
    want = ref.rows(x).double() @ W.double().t() + b.double()
    assert float((ref.rows(x).double().abs() @ W.double().abs().t()).max()) < 2 ** 24
    shape = (oh, M, N // oh) if oh else (M, N)
    if oh:
        y = torch.full(shape, 7.0, dtype=out, device="cuda")
        r = _ints(shape, g, 50, out)
    else:
        hold = torch.full((M, N + ys), 7.0, dtype=out, device="cuda")
        y, r = hold[:, :N], _ints((M, N + ys), g, 50, out)[:, :N]
    got, pre, st = _lib.linear(x, W, b, r, y=y, want_pre=True, out_heads=oh)
    _ok(st)
    assert got is y
    assert torch.equal(got, (ref.heads(want, oh) + r.double()).to(out))
    assert torch.equal(pre, ref.heads(want, oh).to(BF))
    if not oh and ys:
        assert bool((hold[:, N:] == 7).all())
    # bias, residual and z are left out where not given
    got, pre, st = _lib.linear(x, W, out_heads=oh, out_dtype=out, status=st)
    _ok(st)
    assert pre is None and torch.equal(got, ref.heads(want - b.double(), oh).to(out))
    got, pre, st = _lib.linear(x, W, b, r, out_heads=oh, status=st)
    _ok(st)
    assert pre is None and torch.equal(got, (ref.heads(want, oh) + r.double()).to(out))


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("dwt", [BF, F32], ids=["bf16", "f32"])
def test_gradients_exact(name, dwt, cuda_device):
    M, K, N, ih, oh, xs, ws, ys = SHAPES[name]
    g = _gen(2)
    x, W = _x(M, K, ih, xs, g), _ints((N, K + ws), g)[:, :K]
    dy = _ints((oh, M, N // oh), g, 4) if oh else _ints((M, N + ys), g, 4)[:, :N]
    dz, xr = ref.rows(dy).double(), ref.rows(x).double()
    if dwt is F32:      # dy of the other type, and through fp32
        dy = dy.float()
    dx, dW, db, st = _lib.linear_bwd(dy, x, W, dw_dtype=dwt)
    _ok(st)
    assert torch.equal(dx, ref.heads(dz @ W.double(), ih).to(BF))
    assert torch.equal(dW, (dz.t() @ xr).to(dwt))
    assert torch.equal(db, dz.sum(0).float())
    for keep in range(3):      # each by itself
        one = _lib.linear_bwd(dy, x, W, want_dx=keep == 0, want_dw=keep == 1, want_db=keep == 2, dw_dtype=dwt, status=st)
        assert [t is not None for t in one[:3]] == [keep == i for i in range(3)]
        assert torch.equal(one[keep], (dx, dW, db)[keep])
    _ok(st)


@pytest.mark.parametrize("a", [GELU, TANH, SILU])
@pytest.mark.parametrize("name", ["one_token_odd", "tokens_33_ragged", "tokens_64_heads", "pairs_ragged", "pairs_odd", "pairs_chunks",
                                  "single_split8"])
def test_activations(name, a, cuda_device):
    M, K, N, ih, oh, *_ = SHAPES[name]
    g = _gen(3)
    x, W = _x(M, K, ih, 0, g, 2), (_ints((N, K), g, 2).float() / 16).to(BF)
    z = ref.rows(x).double() @ W.double().t()
    for out in (BF, F32):
        y, pre, st = _lib.linear(x, W, activation=a, out_dtype=out, out_heads=oh, want_pre=True)
        _ok(st)
        want, h = ref.act(z, a), ref.half(out)
        tol = h * want.abs() + (1 + h) * 16 * ref.EPS32 * (z.abs() + 1)
        assert bool(((ref.rows(y).double() - want).abs() <= tol).all())
        assert torch.equal(pre, ref.heads(z, oh).to(BF))
    # gradients from the kept z: dz is rounded to 16 bits for the products, db sums it unrounded
    dy = _ints((oh, M, N // oh) if oh else (M, N), g, 3)
    zk = ref.rows(pre).double()
    dz = ref.rows(dy).double() * ref.act_grad(zk, a)
    e = ref.rows(dy).double().abs() * 32 * ref.EPS32 * (zk.abs() + 1)       # of dz before it is rounded
    ez = ref.half(BF) * dz.abs() + (1 + ref.half(BF)) * e
    dx, dW, db, st = _lib.linear_bwd(dy, x, W, pre, a, dw_dtype=F32)
    _ok(st)
    steps = lambda k: (k / 16 + 17) * 2 * ref.EPS32                          # summation of the rounded dz
    want = dz @ W.double()
    tol = ez @ W.double().abs() + steps(N) * (dz.abs() @ W.double().abs())
    assert bool(((ref.rows(dx).double() - want).abs() <= ref.half(BF) * want.abs() + 1.01 * tol).all())
    xr = ref.rows(x).double()
    want = dz.t() @ xr
    tol = ez.t() @ xr.abs() + steps(M) * (dz.abs().t() @ xr.abs())
    assert bool(((dW.double() - want).abs() <= tol + ref.EPS32 * want.abs()).all())
    assert bool(((db.double() - dz.sum(0)).abs() <= e.sum(0) + (M / 8 + 16) * ref.EPS32 * dz.abs().sum(0)).all())


@pytest.mark.parametrize("M,K,N", [(7, 8192, 300), (100, 5120, 256), (2600, 8192, 2048)])
def test_long_sums_of_normal_values(M, K, N, cuda_device):
    """The tensor core's sums lose at most one unit of 2^-23 of the running sum at each of a chunk's
    48 steps of 16, the chunks' sums are rounded to nearest: 48 2^-23 + K / 768 2^-24 of the result's
    size, taken over the whole matrix."""
    g = _gen(4)
    x, W = torch.randn(M, K, generator=g, device="cuda").to(BF), torch.randn(N, K, generator=g, device="cuda").to(BF)
    want = x.double() @ W.double().t()
    y, _, st = _lib.linear(x, W, out_dtype=F32)
    _ok(st)
    bound = 96 * ref.EPS32 + max(K, M) / 768 * ref.EPS32
    assert float((y.double() - want).norm() / want.norm()) <= bound
    dy = torch.randn(M, N, generator=g, device="cuda").to(BF)
    _, dW, _, st = _lib.linear_bwd(dy, x, W, want_dx=False)
    _ok(st)
    want = dy.double().t() @ x.double()
    assert float((dW.double() - want).norm() / want.norm()) <= bound


def test_weight_gradient_over_many_rows(cuda_device):
    """A contraction of 100,003 rows: the chunks keep the truncation at that of 768."""
    g = _gen(5)
    M, K, N = 100_003, 256, 128
    x, dy = torch.randn(M, K, generator=g, device="cuda").to(BF), torch.randn(M, N, generator=g, device="cuda").to(BF)
    W = torch.zeros(N, K, dtype=BF, device="cuda")
    _, dW, db, st = _lib.linear_bwd(dy, x, W, want_dx=False)
    _ok(st)
    want = dy.double().t() @ x.double()
    assert float((dW.double() - want).norm() / want.norm()) <= 96 * ref.EPS32 + M / 768 * ref.EPS32
    sums = dy.double().sum(0)
    assert bool(((db.double() - sums).abs() <= (M / 8 / 8 + 16) * ref.EPS32 * dy.double().abs().sum(0)).all())


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_residual_in_place(dt, cuda_device):
    g = _gen(6)
    for M, K, N in ((5, 640, 256), (100, 100, 130), (100, 2000, 136), (2600, 128, 2100), (2600, 2000, 2104), (2600, 900, 2101),
                    (2570, 17000, 2048)):
        x, W, r = _ints((M, K), g), _ints((N, K), g), _ints((M, N), g, 99, dt)
        want = (x.double() @ W.double().t() + r.double()).to(dt)
        y, _, st = _lib.linear(x, W, residual=r, y=r)
        _ok(st)
        assert y is r and torch.equal(r, want)


def test_no_rows(cuda_device):
    W = torch.ones(96, 64, dtype=BF, device="cuda")
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    y, pre, st = _lib.linear(x, W, want_pre=True)
    assert y.shape == (0, 96) and pre.shape == (0, 96)
    dx, dW, db, st = _lib.linear_bwd(y, x, W)
    _ok(st)
    assert dx.shape == (0, 64) and float(dW.abs().sum()) == 0 and float(db.abs().sum()) == 0


def test_bad_values_stay_in_their_rows(cuda_device):
    """An infinity or NaN in a row of x reaches that row of y only, in W that column only."""
    g = _gen(7)
    for M, K, N in ((20, 640, 256), (2600, 192, 2060)):
        x, W = _ints((M, K), g), _ints((N, K), g)
        clean = _lib.linear(x, W)[0]
        x[3, 5], W[17, 100] = float("nan"), float("inf")
        got = _lib.linear(x, W)[0]
        assert bool(torch.isnan(got[3]).all())
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[3], keep[:, 17] = False, False
        assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("act", [GELU, TANH, SILU])
@pytest.mark.parametrize("cols", [256, 251])
def test_derivative_far_out(act, cols, cuda_device):
    """act' from -3e4 to 3e4, 0 and +-tiny included: dy = 1 and W the identity, so dx is act'(z) rounded once."""
    g = _gen(11)
    z = torch.cat([torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e4, -3e4, 1e3, -1e3, 120.0, -120.0], device="cuda"),
                   torch.linspace(-14, 14, 4000, device="cuda"),
                   torch.randn(40 * cols - 4010, generator=g, device="cuda") * 50]).to(BF).reshape(40, cols)
    dy, eye = torch.ones(40, cols, device="cuda", dtype=BF), torch.eye(cols, device="cuda", dtype=BF)
    dx, _, db, st = _lib.linear_bwd(dy, dy, eye, z, act)
    _ok(st)
    want = ref.act_grad(z.double(), act)
    err = 32 * ref.EPS32 * (z.double().abs() + 1)
    # where the derivative is 0 or 1 to 32 bits nothing is lost: s = 0 or 1 exactly
    err = torch.where(z.double().abs() > 20, 1e-7, err)
    assert bool(((dx.double() - want).abs() <= ref.half(BF) * (want.abs() + err) + err).all())
    # the sums: of unrounded values, 39 fp32 additions of values below 1.2
    assert bool(((db.double() - want.sum(0)).abs() <= err.sum(0) + 39 * ref.EPS32 * 1.2 * 40).all())


def test_same_bits_twice_and_under_a_graph(cuda_device):
    g = _gen(8)
    for M, K, N in ((3, 4096, 512), (300, 520, 777), (2600, 520, 2100)):
        x, W, dy = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((M, K), (N, K), (M, N)))
        b, st = torch.randn(N, generator=g, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
        run = lambda: (*_lib.linear(x, W, b, activation=TANH, want_pre=True, status=st)[:2],
                       *_lib.linear_bwd(dy, x, W, status=st)[:3])
        first, again = run(), run()
        assert all(torch.equal(p, q) for p, q in zip(first, again))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = run()
        x.mul_(-2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, run()))
        _ok(st)


def test_two_streams_at_once(cuda_device):
    g = _gen(9)
    x = [_ints((700, 1000), g) for _ in range(2)]
    W = _ints((1500, 1000), g)
    want = [(t.double() @ W.double().t()).to(BF) for t in x]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for i in range(2):
            got[i] = _lib.linear(x[i], W, stream=ss[i])
    torch.cuda.synchronize()
    for i in range(2):
        _ok(got[i][2])
        assert torch.equal(got[i][0], want[i])


def test_offsets_past_32_bits(cuda_device):
    """y of 2.3e9 elements head-major: its last rows are those of a small call."""
    M, K, N = 300_007, 64, 7680
    x = torch.randint(-3, 4, (M, K), generator=_gen(10), device="cuda").to(BF)
    W = _ints((N, K), _gen(11))
    y, _, st = _lib.linear(x, W, out_heads=60)
    _ok(st)
    assert torch.equal(y[:, -300:], _lib.linear(x[-300:], W, out_heads=60)[0])
    dx, dW, db, st = _lib.linear_bwd(y, x, W, want_dw=False)
    _ok(st)
    assert torch.equal(dx[-300:], _lib.linear_bwd(y[:, -300:].contiguous(), x[-300:], W, want_dw=False)[0])


def test_refusals(cuda_device):
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")
    x, W = z(10, 64), z(96, 64)
    for call in (lambda: _lib.linear(z(100, 65).reshape(-1)[1:641].view(10, 64), W),      # address off 16 bytes
                 lambda: _lib.linear(x, W, activation=9),
                 lambda: _lib.linear(x, z(64, 64), y=x),                                  # the result over the input
                 lambda: _lib.linear_bwd(z(10, 96), x, W, dx=x),
                 lambda: _lib.linear_bwd(z(10, 96), x, W, workspace=z(1, dtype=torch.uint8))):
        with pytest.raises(_lib.PrismError):
            call()
    buf = z(10, 200)
    with pytest.raises(_lib.PrismError):                                                  # overlapping, not the same
        _lib.linear(x, W, residual=buf[:, 8:104], y=buf[:, :96])
    _lib.linear(x, W, residual=buf[:, 96:192], y=buf[:, :96])                             # columns side by side
    for call in (lambda: _lib.linear(x.float(), W), lambda: _lib.linear(x, W.float()), lambda: _lib.linear(x, z(96, 63)),
                 lambda: _lib.linear(x, W, z(95, dtype=F32)), lambda: _lib.linear(x, W, residual=z(10, 95)),
                 lambda: _lib.linear(x, W, out_heads=2), lambda: _lib.linear(x.t(), z(96, 10)),
                 lambda: _lib.linear(z(2, 10, 32), W), lambda: _lib.linear(x, W.cpu()),
                 lambda: _lib.linear(x, W, out_dtype=torch.float16), lambda: _lib.linear(x[:, ::2], z(96, 32)),
                 lambda: _lib.linear_bwd(z(10, 96), x, W, None, TANH), lambda: _lib.linear_bwd(z(9, 96), x, W),
                 lambda: _lib.linear_bwd(z(10, 96), x, W, dx=z(10, 64, dtype=F32))):
        with pytest.raises(ValueError):
            call()
