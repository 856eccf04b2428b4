"""fp32 results keep the truncation of chunks of 768 elements however long the contraction is.

The tensor core drops what its fp32 sum cannot hold at each step of 16: at most a unit in the last place
of the running sum S_j, half a unit on average, always towards zero.  A unit is between 2^-24 and 2^-23 of
S_j, on average over the mantissas (1 / ln 2)(1 - 1/2) 2^-23 = 0.72 2^-23.  Projected on the chunk's sum, S_j
of 48 steps counts j / 48, so a chunk of independent values is low by at most
    0.5 0.72 2^-23 sum_{j <= 48} j / 48 = 24.5 0.72 2^-24 = 1.05e-6
of itself, and so is the sum of any number of chunks, each by the same share.  A chunk of 1,536 elements
loses twice that, an uncut contraction in proportion to its length.  What is measured is the signed loss,
the mean of (y - exact) sign(exact) over the mean of |exact|: what rounds to nearest cancels in it."""
import pytest
import torch

import linear_ref as ref
from dynamic_block_sparse_indicator_b200 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
LOSS = 24.5 * 0.72 * 2.0 ** -24


def _signed_loss(got, want):
    d = (got.double() - want) * want.sign()
    return float(-d.mean() / want.abs().mean())


# contractions that no cluster splits: more tiles than CTAs
@pytest.mark.parametrize("M,K,N", [(2600, 16_000, 2048), (2600, 8192, 2120)])
def test_forward(M, K, N, cuda_device):
    g = torch.Generator("cuda").manual_seed(K)
    x, W = (torch.randn(n, K, generator=g, device="cuda").to(BF) for n in (M, N))
    want = x.double() @ W.double().t()
    y = _lib.linear(x, W, out_dtype=F32)[0]
    assert abs(_signed_loss(y, want)) <= LOSS
    r = torch.zeros(M, N, device="cuda")
    assert torch.equal(_lib.linear(x, W, residual=r)[0], y)


@pytest.mark.parametrize("M,K,N", [(50_000, 2048, 2048), (30_011, 2500, 1900)])
def test_weight_gradient(M, K, N, cuda_device):
    g = torch.Generator("cuda").manual_seed(M)
    x, dy = (torch.randn(M, n, generator=g, device="cuda").to(BF) for n in (K, N))
    dW = _lib.linear_bwd(dy, x, torch.zeros(N, K, dtype=BF, device="cuda"), want_dx=False, want_db=False)[1]
    want = dy.double().t() @ x.double()
    assert abs(_signed_loss(dW, want)) <= LOSS
    # and all of it: the loss's spread and M / 768 additions rounded to nearest, no longer than the sum
    assert float((dW.double() - want).norm() / want.norm()) <= 48 * 2.0 ** -23 + (M / 768) ** 0.5 * ref.EPS32
