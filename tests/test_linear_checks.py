"""prism_linear and its gradients refuse bad arguments before touching a device (no GPU)."""
import ctypes as C

import pytest
import torch

from dynamic_block_sparse_indicator_b200 import _lib


@pytest.fixture(scope="module")
def lib():
    from dynamic_block_sparse_indicator_b200 import build
    build.build_library()
    return _lib.load()


def _params(**kw):
    base = dict(M=10, K=128, N=256, in_heads=0, out_heads=0, activation=0, out_dtype=0, bias_dtype=1, dw_dtype=1,
                x_stride=128, w_stride=128, y_stride=256, r_stride=256)
    base.update(kw)
    return _lib.PrismLinearParams(*[base[f] for f, _ in _lib.PrismLinearParams._fields_])


BAD = (dict(M=-1), dict(M=1 << 31), dict(K=0), dict(N=0), dict(K=1 << 25, x_stride=1 << 25, w_stride=1 << 25),
       dict(in_heads=-1), dict(in_heads=3), dict(in_heads=4), dict(out_heads=8), dict(out_heads=5), dict(activation=4),
       dict(activation=-1), dict(out_dtype=2), dict(bias_dtype=-1), dict(dw_dtype=7), dict(x_stride=127),
       dict(w_stride=100), dict(y_stride=255), dict(r_stride=0), dict(x_stride=1 << 40), dict(in_heads=2, x_stride=136),
       dict(out_heads=2, y_stride=264), dict(out_heads=4, r_stride=260))
INV, WS = _lib.PRISM_ERR_INVALID_ARG, _lib.PRISM_ERR_WORKSPACE
X, W, B, R, Y, P, S, T = ((i + 1) << 24 for i in range(8))


def test_forward_refusals(lib):
    def call(x=X, w=W, b=B, r=R, y=Y, pre=P, ws=S, nb=1 << 20, st=T, **kw):
        return lib.prism_linear(C.byref(_params(**kw)), x, w, b, r, y, pre, ws, nb, st, None)

    for bad in BAD:
        assert call(**bad) == INV, bad
    for name in ("x", "w", "y", "st"):
        assert call(**{name: None}) == INV, name
    for name in ("x", "w", "b", "r", "y", "pre", "ws", "st"):
        assert call(**{name: (9 << 24) + 8}) == INV, name
    assert call(y=X) == INV and call(y=W + 1024) == INV and call(y=B) == INV and call(pre=X) == INV
    assert call(pre=Y) == INV and call(pre=R) == INV
    assert call(r=Y + 512) == INV                                  # over the residual, shifted
    assert call(r=Y, r_stride=264) == INV                          # over the residual with other rows
    assert call(x_stride=131, ws=None) == INV and call(x_stride=131, nb=16) == WS
    assert call(w_stride=129, nb=16) == WS
    assert call(M=0) == _lib.PRISM_OK                              # nothing to do, no device needed


def test_backward_refusals(lib):
    def call(dy=Y, x=X, w=W, pre=P, dx=B, dw=R, db=9 << 24, ws=S, nb=1 << 20, st=T, **kw):
        return lib.prism_linear_bwd(C.byref(_params(**kw)), dy, x, w, pre, dx, dw, db, ws, nb, st, None)

    for bad in BAD:
        assert call(**bad) == INV, bad
    assert call(dy=None) == INV and call(st=None) == INV and call(w=None) == INV and call(x=None) == INV
    assert call(activation=2, pre=None) == INV
    for name in ("dy", "x", "w", "pre", "dx", "dw", "db", "ws", "st"):
        assert call(**{name: (10 << 24) + 8}) == INV, name
    assert call(dx=X) == INV and call(dw=W) == INV and call(dx=R + 256) == INV and call(db=Y) == INV
    assert call(ws=None) == INV and call(nb=16) == WS
    assert call(dx=None, dw=None, db=None) == _lib.PRISM_OK
    assert call(M=0, dw=None, db=None) == _lib.PRISM_OK


def test_workspace_bytes(lib):
    f, b = lib.prism_linear_workspace_bytes, lib.prism_linear_bwd_workspace_bytes
    for bad in BAD:
        assert f(C.byref(_params(**bad))) == 0 and b(C.byref(_params(**bad))) == 0, bad
    n = f(C.byref(_params()))
    assert 0 < n <= 256                                            # operands are read where they lie
    assert f(C.byref(_params(x_stride=131))) >= n + 10 * 128 * 2
    assert f(C.byref(_params(w_stride=131))) >= n + 256 * 128 * 2
    m = b(C.byref(_params()))
    assert b(C.byref(_params(activation=1))) >= m + 10 * 256 * 2   # dz
    assert b(C.byref(_params(out_dtype=1))) >= m + 10 * 256 * 2


def test_binding_refuses_host_tensors_and_bad_shapes():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    x, w = z(10, 64), z(96, 64)
    for call in (lambda: _lib.linear(x, w), lambda: _lib.linear(x, z(96, 32)), lambda: _lib.linear(x.float(), w),
                 lambda: _lib.linear(x, w, out_heads=2), lambda: _lib.linear(z(2, 10, 32), w),
                 lambda: _lib.linear(x.t(), z(96, 10)), lambda: _lib.linear_bwd(z(10, 96), x, w),
                 lambda: _lib.linear_bwd(z(10, 95), x, w), lambda: _lib.linear_bwd(z(10, 96), x, w, None, 1)):
        with pytest.raises(ValueError):
            call()
