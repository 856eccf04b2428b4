"""What an fp32 result of the projections holds, on the GPU against 64 bits."""
import pytest
import torch

import linear_ref as ref
from dynamic_block_sparse_indicator_b200 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# M, K, N of weights' gradients: k_few (N <= 64), single CTAs whole and split, pairs; rows of any alignment
DW_SHAPES = [(1, 72, 40), (100, 640, 48), (13, 331, 257), (127, 203, 77), (300, 300, 130), (2000, 256, 128), (90, 2050, 2560), (1500, 2120, 2048)]


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _ints(gen, hi, *shape, dtype=F32):
    return torch.randint(-hi, hi + 1, shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("M,K,N", DW_SHAPES)
def test_weight_gradient_keeps_fp32_dy(M, K, N, cuda_device):
    """dy of integers that bf16 does not hold (12 bits, 16 for few rows), x of small ones: every partial
    sum is an integer below 2^24, so an fp32 dW is exact.  dx and a bf16 dW have 16 bits themselves and
    take dy rounded to them."""
    g = _gen(M)
    dy, x, W = _ints(g, 1 << (15 if M <= 128 else 11), M, N), _ints(g, 3, M, K, dtype=BF), _ints(g, 1, N, K, dtype=BF)
    assert float((dy.double().abs().t() @ x.double().abs()).max()) < 2 ** 24
    dx, dW, db, st = _lib.linear_bwd(dy, x, W)
    assert torch.equal(dW, (dy.double().t() @ x.double()).float())
    assert bool(((db.double() - dy.double().sum(0)).abs() <= (M / 8 + 16) * ref.EPS32 * dy.double().abs().sum(0)).all())
    dz = dy.to(BF).double()
    if float((dz.abs() @ W.double().abs()).max()) < 2 ** 24:
        assert torch.equal(dx, (dz @ W.double()).to(BF))
    one = _lib.linear_bwd(dy, x, W, want_dx=False, want_db=False, status=st)[1]
    assert torch.equal(one, dW)
    if float((dz.abs().t() @ x.double().abs()).max()) < 2 ** 24:
        low = _lib.linear_bwd(dy, x, W, want_dx=False, dw_dtype=BF, status=st)[1]
        assert torch.equal(low, (dz.t() @ x.double()).to(BF))
    assert _lib.status_read(st)[0] == _lib.PRISM_OK


@pytest.mark.parametrize("M,heads,D,N", [(1, 2, 64, 192), (50, 3, 128, 257), (700, 5, 64, 320), (1500, 10, 128, 2048)])
@pytest.mark.parametrize("slices", [False, True], ids=["own", "slices"])
def test_weight_gradient_keeps_fp32_dy_of_heads_and_slices(M, heads, D, N, slices, cuda_device):
    """The same with x and dy head-major, and with both as columns of wider buffers of odd strides."""
    g = _gen(M)
    K, oh = heads * D, N // 64 if N % 64 == 0 else 0
    dy, x = _ints(g, 1 << (15 if M <= 128 else 11), M, N), _ints(g, 3, M, K, dtype=BF)
    want, W = (dy.double().t() @ x.double()).float(), _ints(g, 1, N, K, dtype=BF)
    if slices:
        hold = [torch.full((M, t.shape[1] + 5), 7.0, dtype=t.dtype, device="cuda") for t in (dy, x)]
        for h, t in zip(hold, (dy, x)):
            h[:, :t.shape[1]] = t
        dy, x = hold[0][:, :N], hold[1][:, :K]
    else:
        dy, x = (ref.heads(t, n).contiguous() for t, n in ((dy, oh), (x, heads)))
    dW, st = _lib.linear_bwd(dy, x, W, want_dx=False, want_db=False)[1::2]
    assert torch.equal(dW, want)
    assert _lib.status_read(st)[0] == _lib.PRISM_OK


@pytest.mark.parametrize("act", [1, 2, 3])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", DW_SHAPES)
def test_weight_gradient_keeps_fp32_dz(M, K, N, dt, act, cuda_device):
    """Through an activation: dz's own error is linear_ref's 32 EPS32 (|z| + 1) of dy, two bf16 parts
    leave half a bf16 step of half a step, and the sums of both parts at most a unit of 2^-23 of the
    terms' size at each of their M / 16 steps and the chunks' and the parts' additions."""
    g = _gen(M + act)
    dy, x, pre = (torch.randn(M, n, generator=g, device="cuda").to(t) for n, t in ((N, dt), (K, BF), (N, BF)))
    W = torch.zeros(N, K, dtype=BF, device="cuda")
    dW = _lib.linear_bwd(dy, x, W, pre, act, want_dx=False)[1]
    z, xd = pre.double(), x.double()
    dz = dy.double() * ref.act_grad(z, act)
    want = dz.t() @ xd
    h = ref.half(BF)
    each = (1 + h) * 32 * ref.EPS32 * (z.abs() + 1) * dy.double().abs() + h * h * dz.abs()
    tol = each.t() @ xd.abs() + (2 * (M / 16 + 2) + M / 768 + 4) * ref.EPS32 * (dz.abs().t() @ xd.abs())
    assert bool(((dW.double() - want).abs() <= tol).all())
    # over the matrix: the parts' 2^-18 and the sums' 48 2^-23 a chunk, where one bf16 part leaves 1e-3
    assert float((dW.double() - want).norm() / want.norm()) <= 2.0 ** -18 + 96 * ref.EPS32 + (M / 768 + 4) * ref.EPS32 + 32 * 2 * ref.EPS32


def test_weight_gradient_of_values_that_are_not_finite(cuda_device):
    """An infinity or NaN of dy reaches its feature's row of dW and no other value; the largest finite bf16 is kept."""
    g = _gen(5)
    dy, x = torch.randn(40, 96, generator=g, device="cuda"), torch.randn(40, 64, generator=g, device="cuda").to(BF)
    x[x == 0] = 1
    W = torch.zeros(96, 64, dtype=BF, device="cuda")
    clean = _lib.linear_bwd(dy, x, W, want_dx=False)[1]
    dy[3, 5], dy[4, 7] = float("inf"), float("nan")
    dW = _lib.linear_bwd(dy, x, W, want_dx=False)[1]
    assert bool(torch.isnan(dW[7]).all())
    assert torch.equal(dW[5], float("inf") * x[3].float().sign())
    keep = torch.ones(96, dtype=torch.bool, device="cuda")
    keep[5] = keep[7] = False
    assert torch.equal(dW[keep], clean[keep])


# M, K, N: k_few whole and split; single CTAs whole, split and of any alignment; pairs of one chunk, of several (768 and
# 16,384 elements), ragged, with a column tile that is partly outside, and of any alignment
RES_SHAPES = [(5, 640, 256), (13, 4224, 256), (60, 1280, 129), (100, 640, 136), (100, 5000, 136), (100, 900, 131),
              (2571, 640, 2120), (2500, 5000, 2000), (2571, 1700, 2120), (600, 5000, 4160), (2560, 17000, 2056), (2571, 5000, 2121)]


@pytest.mark.parametrize("M,K,N", RES_SHAPES)
@pytest.mark.parametrize("heads", [False, True], ids=["rows", "heads"])
@pytest.mark.parametrize("bias", [False, True], ids=["no_bias", "bias"])
def test_a_large_residual_is_added_once(M, K, N, heads, bias, cuda_device):
    """x W^T + b of integers below 2^24 is exact, so y is the residual plus it with one rounding, however
    large the residual: 30,000 times a normal value, with all its fraction bits.  In place too."""
    if heads:
        N = -(-N // 64) * 64
    g = _gen(K)
    x, W = _ints(g, 3, M, K, dtype=BF), _ints(g, 3, N, K, dtype=BF)
    b = _ints(g, 9, N) if bias else None
    shape = (N // 64, M, 64) if heads else (M, N)
    z = x.double() @ W.double().t() + (b.double() if bias else 0)
    z = ref.heads(z, N // 64) if heads else z
    r = torch.randn(shape, generator=g, device="cuda") * 3e4
    want = (z + r.double()).float()
    y, _, st = _lib.linear(x, W, b, r, out_heads=N // 64 if heads else 0)
    assert torch.equal(y, want)
    y, _, st = _lib.linear(x, W, b, r, y=r, status=st)
    assert y is r and torch.equal(r, want)
    assert _lib.status_read(st)[0] == _lib.PRISM_OK
