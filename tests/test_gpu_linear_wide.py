"""prism_linear and its gradients with very many features, exact on integers (see linear_ref)."""
import pytest
import torch

from dynamic_block_sparse_indicator_b200 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _ints(gen, *shape, hi=3, dtype=BF):
    return torch.randint(-hi, hi + 1, shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("M,K,N", [(1, 64, 600_000), (70, 72, 600_001), (2, 600_008, 64)])
def test_wide(M, K, N, cuda_device):
    g = torch.Generator("cuda").manual_seed(M)
    x, W, b, dy = _ints(g, M, K), _ints(g, N, K), _ints(g, N, dtype=F32), _ints(g, M, N)
    y, _, st = _lib.linear(x, W, b, out_dtype=F32)
    assert torch.equal(y, (x.double() @ W.double().t() + b.double()).float())
    dx, dW, db, _ = _lib.linear_bwd(dy, x, W, status=st)
    assert torch.equal(dx, (dy.double() @ W.double()).to(BF))
    assert torch.equal(dW, (dy.double().t() @ x.double()).float())
    assert torch.equal(db, dy.double().sum(0).float())
    assert _lib.status_read(st)[0] == _lib.PRISM_OK
