"""The whole documented range of prism_linear's sizes and strides is taken (no GPU)."""
import ctypes as C

import pytest

from dynamic_block_sparse_indicator_b200 import _lib

TOP = 1 << 24


@pytest.fixture(scope="module")
def lib():
    from dynamic_block_sparse_indicator_b200 import build
    build.build_library()
    return _lib.load()


def _bytes(lib, M, K, N, xs=None, ws=None, ys=None, rs=None, out=1):
    p = _lib.PrismLinearParams(M, K, N, 0, 0, 0, out, 1, 1, xs or K, ws or K, ys or N, rs or N)
    return lib.prism_linear_workspace_bytes(C.byref(p)), lib.prism_linear_bwd_workspace_bytes(C.byref(p))


@pytest.mark.parametrize("M,K,N", [(1, 64, 600_000), (1, 64, TOP), (1, TOP, 64), (16_000, 8, TOP), (16_000, TOP, 8), (100, 16_000, TOP),
                                   ((1 << 31) - 256, 128, 128), (0, TOP, 1), (1, 1, 1)])
def test_sizes(lib, M, K, N):
    f, b = _bytes(lib, M, K, N)
    assert f > 0 and b > 0


def test_a_stride_counts_its_own_rows(lib):
    """Columns of a wide buffer: the rows of x, y and residual are M, W's are N."""
    assert all(_bytes(lib, 10_000_000, 64, 64, ws=TOP))
    assert all(_bytes(lib, 10, 64, 1 << 20, xs=1 << 30, ys=1 << 30, rs=1 << 30))


@pytest.mark.parametrize("M,K,N,kw", [(1 << 20, 64, 1 << 20, {}), (1 << 20, 1 << 20, 64, {}), (1, 1 << 20, 1 << 20, {}),
                                      (1 << 20, 64, 64, dict(xs=1 << 18)), (1 << 20, 64, 64, dict(ys=1 << 18)),
                                      (1 << 20, 64, 64, dict(rs=1 << 18)), (1, 64, 1 << 20, dict(ws=1 << 18))])
def test_a_tensor_of_2_38_elements_is_refused(lib, M, K, N, kw):
    assert _bytes(lib, M, K, N, **kw) == (0, 0)
