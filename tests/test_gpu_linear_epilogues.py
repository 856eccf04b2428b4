"""Bias, kept z, activation and residual together, in their order, through every epilogue of the projections."""
import pytest
import torch

import linear_ref as ref
from dynamic_block_sparse_indicator_b200 import _lib

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# M, K, N, out_heads
SHAPES = {
    "few_whole": (17, 448, 320, 0),
    "few_split": (13, 4224, 250, 0),
    "few_heads": (64, 1280, 640, 5),
    "single_aligned": (100, 72, 264, 0),
    "single_any": (100, 72, 261, 0),
    "single_split": (300, 8192, 304, 0),
    "single_split_any": (300, 8192, 301, 0),
    "pairs_one_chunk": (2571, 200, 2120, 0),
    "pairs_one_chunk_heads": (2571, 640, 1920, 15),
    "pairs_chunks_f32": (2500, 1700, 2008, 0),
    "pairs_chunks_f32_192": (600, 1000, 4160, 0),
    "pairs_chunks_bf16": (2560, 17000, 2056, 0),
    "pairs_any": (2571, 203, 2121, 0),
    "pairs_any_chunks": (2571, 1700, 2121, 0),
}


@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(SHAPES))
def test_composition(name, out, act, cuda_device):
    """z = x W^T + b in sixteenths, exact in fp32; y = act(z) + r with linear_ref's error of act, one
    rounding of the sum in 32 bits and one to the result's type (none of them without an activation)."""
    M, K, N, oh = SHAPES[name]
    g = torch.Generator("cuda").manual_seed(act)
    ints = lambda hi, *s: torch.randint(-hi, hi + 1, s, generator=g, device="cuda").float()
    x, W = ints(2, M, K).to(BF), (ints(2, N, K) / 16).to(BF)
    b = ints(9, N) / 16
    shape = (oh, M, N // oh) if oh else (M, N)
    z0 = x.double() @ W.double().t()
    r0 = (ints(50, *shape) / 16).to(out)                         # (exact in both types)
    h = ref.half(out)
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bias in (None, b, b.to(BF)):
        z = ref.heads(z0 if bias is None else z0 + bias.double(), oh)
        a = ref.act(z, act)
        for residual, keep, inplace in ((False, False, False), (False, True, False), (True, False, False), (True, True, False),
                                        (True, False, True), (True, True, True)):
            r = r0.clone() if residual else None
            y, pre, _ = _lib.linear(x, W, bias, r, act, y=r if inplace else None, out_dtype=out, out_heads=oh, want_pre=keep, status=st)
            what = f"bias {None if bias is None else bias.dtype}, residual {residual}, z kept {keep}, in place {inplace}"
            want = a + r0.double() if residual else a
            if act == 0:
                assert torch.equal(y, want.to(out)), what
            else:
                e = 16 * ref.EPS32 * (z.abs() + 1)
                e = e + ref.EPS32 * (want.abs() + e)
                assert bool(((y.double() - want).abs() <= h * want.abs() + (1 + h) * e).all()), what
            assert (pre is not None) == keep and (not keep or torch.equal(pre, z.to(BF))), what
            assert not inplace or y is r
            assert not residual or inplace or torch.equal(r, r0), what
    assert _lib.status_read(st)[0] == _lib.PRISM_OK
