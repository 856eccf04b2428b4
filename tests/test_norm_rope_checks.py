"""prism_qk_norm_rope, its gradients and the rotation table refuse bad arguments before touching a
device, and the gradients' formulas agree with differences (64 bits, no GPU)."""
import ctypes as C

import pytest
import torch

import norm_rope_ref as ref
from dynamic_block_sparse_indicator_b200 import _lib


@pytest.fixture(scope="module")
def lib():
    from dynamic_block_sparse_indicator_b200 import build
    build.build_library()
    return _lib.load()


def _params(**kw):
    base = dict(N=24, T=2, H=3, W=4, heads=2, head_dim=64, dtype=0, out_dtype=0, w_dtype=1, dim_t=16, dim_h=8, dim_w=8,
                pairing=0, eps=1e-6)
    base.update(kw)
    return _lib.PrismNormRopeParams(*[base[f] for f, _ in _lib.PrismNormRopeParams._fields_])


def _rows(at, hs=24 * 64, ts=64):
    return _lib.PrismRows(at, hs, ts)


A, B, Cc, Dd = (1 << 20, 1 << 21, 1 << 22, 1 << 23)
BAD_PARAMS = (dict(N=-1), dict(heads=0), dict(heads=1 << 16), dict(head_dim=96), dict(dtype=2), dict(out_dtype=-1),
              dict(w_dtype=5), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")))
BAD_ROPE = (dict(T=3), dict(H=0), dict(W=-4), dict(dim_t=15), dict(dim_h=-2), dict(dim_t=60), dict(pairing=2),
            dict(T=1 << 30, H=1 << 30, W=1 << 30))


def test_forward_refusals(lib):
    def call(p=None, q=None, k=None, wq=None, wk=None, rope=1 << 24, qo=None, ko=None, **kw):
        r = lambda x: None if x is None else C.byref(x)
        return lib.prism_qk_norm_rope(C.byref(p or _params(**kw)), r(q or _rows(A)), r(k), wq, wk, rope,
                                      r(qo or _rows(B)), r(ko), None)

    for bad in BAD_PARAMS + BAD_ROPE:
        assert call(**bad) == _lib.PRISM_ERR_INVALID_ARG, bad
    bad = _lib.PRISM_ERR_INVALID_ARG
    assert call(q=_rows(0)) == bad and call(qo=_rows(None)) == bad
    assert call(q=_rows(A + 8)) == bad and call(q=_rows(A, ts=68)) == bad and call(q=_rows(A, hs=-64)) == bad
    assert call(k=_rows(Cc)) == bad                          # k without its result
    assert call(ko=_rows(Cc)) == bad
    assert call(wk=1 << 25) == bad and call(wq=(1 << 25) + 4) == bad and call(rope=(1 << 24) + 8) == bad
    assert call(qo=_rows(B, ts=32)) == bad                   # rows written onto each other
    assert call(qo=_rows(A + 128)) == bad                    # partly over the input
    assert call(k=_rows(Cc), ko=_rows(B)) == bad             # both results in one place
    assert call(qo=_rows(A), out_dtype=1) == bad             # in place with another type
    # no tokens: nothing to do, no device needed
    assert call(N=0) == _lib.PRISM_OK


def test_interleaved_slices_are_not_an_overlap(lib):
    """Slices of one fused [N][3][heads][D] buffer pass the checks (and end at the missing device here)."""
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a device")
    s = lambda i: _rows(A + i * 2 * 64 * 2, hs=64, ts=3 * 2 * 64)
    st = lib.prism_qk_norm_rope(C.byref(_params()), C.byref(s(0)), C.byref(s(1)), None, None, None, C.byref(s(0)),
                                C.byref(s(1)), None)
    assert st == _lib.PRISM_ERR_UNSUPPORTED
    half = _rows(A + 64, hs=64, ts=3 * 2 * 64)               # half a row off
    st = lib.prism_qk_norm_rope(C.byref(_params()), C.byref(s(0)), None, None, None, None, C.byref(half), None, None)
    assert st == _lib.PRISM_ERR_INVALID_ARG


def test_backward_refusals(lib):
    def call(dqo=None, dko=None, q=None, k=None, wq=None, wk=None, rope=1 << 24, dq=None, dk=None, dwq=None, dwk=None,
             ws=1 << 26, nb=1 << 20, **kw):
        r = lambda x: None if x is None else C.byref(x)
        return lib.prism_qk_norm_rope_bwd(C.byref(_params(**kw)), r(dqo or _rows(A)), r(dko), r(q or _rows(B)), r(k), wq,
                                          wk, rope, r(dq or _rows(Cc)), r(dk), dwq, dwk, ws, nb, None)

    bad = _lib.PRISM_ERR_INVALID_ARG
    for b in BAD_PARAMS + BAD_ROPE:
        assert call(**b) == bad, b
    assert call(k=_rows(Dd)) == bad and call(dk=_rows(Dd)) == bad and call(dwk=1 << 25) == bad
    assert call(dwq=1 << 25, ws=None) == bad and call(dwq=1 << 25, ws=(1 << 26) + 4) == bad
    assert call(dwq=1 << 25, nb=16) == _lib.PRISM_ERR_WORKSPACE
    assert call(dq=_rows(B + 64)) == bad and call(dq=_rows(A + 64)) == bad
    assert call(dq=_rows(B), dqo=_rows(B + 16)) == bad


def test_table_refusals(lib):
    call = lambda theta=1e4, first=0, tab=1 << 20, **kw: lib.prism_rope_table(C.byref(_params(**kw)), theta, first, tab, None)
    for b in BAD_PARAMS + BAD_ROPE + (dict(N=0), dict(theta=0.0), dict(theta=float("nan")), dict(first=-1), dict(tab=None),
                                      dict(tab=(1 << 20) + 4)):
        assert call(**b) == _lib.PRISM_ERR_INVALID_ARG, b


def test_workspace_bytes(lib):
    n = lib.prism_qk_norm_rope_bwd_workspace_bytes(C.byref(_params()))
    assert n > 0
    # never more than 16 blocks' rows per SM, however many tokens
    assert lib.prism_qk_norm_rope_bwd_workspace_bytes(C.byref(_params(N=1 << 30))) <= 16 * 148 * 64 * 4
    for b in BAD_PARAMS:
        assert lib.prism_qk_norm_rope_bwd_workspace_bytes(C.byref(_params(**b))) == 0, b


def test_binding_refuses_host_tensors_and_bad_shapes():
    x = torch.zeros(2, 24, 64, dtype=torch.bfloat16)
    for call in (lambda: _lib.qk_norm_rope(x), lambda: _lib.qk_norm_rope(x, x[:1]), lambda: _lib.qk_norm_rope(x[0]),
                 lambda: _lib.qk_norm_rope(x.double()), lambda: _lib.qk_norm_rope(x, None, torch.ones(3)),
                 lambda: _lib.qk_norm_rope_bwd(x, x, x), lambda: _lib.qk_norm_rope_bwd(x, None, x),
                 lambda: _lib.make_rope(2, 3, 4, (15, 8, 8), device="cpu"),
                 lambda: _lib.make_rope(2, 0, 4, (16, 8, 8), device="cpu")):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("pairing", [0, 1])
def test_formulas_against_autograd_and_differences(pairing):
    g = torch.Generator().manual_seed(0)
    T, H, W, dims = 2, 3, 4, (16, 8, 8)
    ang, ab = ref.angles(T, H, W, dims, 100.0), ref.pairs(dims, pairing)
    x = torch.randn(2, 24, 64, generator=g, dtype=torch.float64)
    w = torch.randn(64, generator=g, dtype=torch.float64)
    gy = torch.randn(2, 24, 64, generator=g, dtype=torch.float64)
    dx, _, dw, _ = ref.backward(gy, x, w, ang, ab, 1e-3)
    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    (ref.forward(xr, wr, ang, ab, 1e-3)[0] * gy).sum().backward()
    assert torch.allclose(dx, xr.grad, rtol=1e-12, atol=1e-12) and torch.allclose(dw, wr.grad, rtol=1e-12, atol=1e-12)
    f = lambda xx: float((ref.forward(xx, w, ang, ab, 1e-3)[0] * gy).sum())
    d = torch.randn(x.shape, generator=g, dtype=torch.float64)
    assert abs((f(x + 1e-5 * d) - f(x - 1e-5 * d)) / 2e-5 - float((dx * d).sum())) < 1e-6
