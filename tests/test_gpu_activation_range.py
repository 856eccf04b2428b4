"""Activations and their derivatives over all of bf16's range: where 64 bits give 0, 1 or z, so do the kernels."""
import pytest
import torch

import linear_ref as ref
from dynamic_block_sparse_indicator_b200 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
MAGNITUDES = [0.0, 1e-38, 1e-20, 25.0, 88.0, 104.0, 1e4, 1e9, 1e13, 1e15, 1.8e19, 1.9e19, 3e19, 1e25, 1e38, 3.3e38]


def _values(cols):
    v = torch.tensor(MAGNITUDES, device="cuda")
    return torch.cat([v, -v])[:, None].expand(-1, cols).to(BF).contiguous()


@pytest.mark.parametrize("act", [1, 2, 3])
@pytest.mark.parametrize("cols", [64, 61])
def test_forward(act, cols, cuda_device):
    """W is the identity, so z is the value itself; act(z) within linear_ref's bound."""
    z = _values(cols)
    eye = torch.eye(cols, device="cuda", dtype=BF)
    want = ref.act(z.double(), act)
    err = torch.where(z.double().abs() > 20, 1e-7, 16 * ref.EPS32 * (z.double().abs() + 1))
    for dt in (BF, F32):
        y = _lib.linear(z, eye, activation=act, out_dtype=dt)[0].double()
        assert bool(((y - want).abs() <= ref.half(dt) * want.abs() + 1.01 * err).all())


@pytest.mark.parametrize("act", [1, 2, 3])
@pytest.mark.parametrize("cols", [64, 61])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_derivative(act, cols, dt, cuda_device):
    """dy is 1 and W the identity, so dx is act'(z) rounded."""
    z = _values(cols)
    dy, eye = torch.ones(z.shape, device="cuda", dtype=dt), torch.eye(cols, device="cuda", dtype=BF)
    dx, _, db, _ = _lib.linear_bwd(dy, z, eye, z, act, want_dw=False)
    want = ref.act_grad(z.double(), act)
    err = torch.where(z.double().abs() > 20, 1e-7, 32 * ref.EPS32 * (z.double().abs() + 1))
    assert bool(((dx.double() - want).abs() <= ref.half(BF) * (want.abs() + err) + err).all())
    assert bool(((db.double() - want.sum(0)).abs() <= err.sum(0) + 31 * ref.EPS32 * 32).all())
