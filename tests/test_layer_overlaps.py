"""What the layer's operators write may share no byte with what else a call reads or writes: weights,
rotation table, weights' gradients, workspace and status block included.  Addresses only; a call that
passes the checks ends at the missing device (no GPU)."""
import ctypes as C

import pytest
import torch

from dynamic_block_sparse_indicator_b200 import _lib

INV = _lib.PRISM_ERR_INVALID_ARG
N, HEADS, D = 24, 2, 64
ROWS = HEADS * N * D * 2                                            # bytes of a bf16 tensor of rows
Q, K, QO, KO, WQ, WK, TAB, DWQ, DWK, WS = ((i + 1) << 24 for i in range(10))
TABLE = (2 * 16 + 3 * 8 + 4 * 8) * 4


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("addresses that no device may see")
    from dynamic_block_sparse_indicator_b200 import build
    build.build_library()
    return _lib.load()


def _norm_params(w_dtype=1):
    return _lib.PrismNormRopeParams(N, 2, 3, 4, HEADS, D, 0, 0, w_dtype, 16, 8, 8, 0, 1e-6)


def _rows(at):
    return C.byref(_lib.PrismRows(at, N * D, D))


def _norm(lib, q=Q, k=K, wq=WQ, wk=WK, tab=TAB, qo=QO, ko=KO):
    return lib.prism_qk_norm_rope(C.byref(_norm_params()), _rows(q), _rows(k), wq, wk, tab, _rows(qo), _rows(ko), None)


def _norm_bwd(lib, dqo=Q, dko=K, q=11 << 24, k=12 << 24, wq=WQ, wk=WK, tab=TAB, dq=QO, dk=KO, dwq=DWQ, dwk=DWK, ws=WS):
    p = _norm_params()
    n = lib.prism_qk_norm_rope_bwd_workspace_bytes(C.byref(p))
    return lib.prism_qk_norm_rope_bwd(C.byref(p), _rows(dqo), _rows(dko), _rows(q), _rows(k), wq, wk, tab, _rows(dq),
                                      _rows(dk), dwq, dwk, ws, n, None)


def _ends(at, size, other):
    """Addresses at which `other` bytes touch the first and the last 16 bytes of [at, at + size)."""
    return at + 16 - other, at + size - 16


def test_norm(lib):
    assert _norm(lib) == _lib.PRISM_ERR_UNSUPPORTED
    for out in (QO, KO):
        for a in _ends(out, ROWS, D * 4):
            assert _norm(lib, wq=a) == INV and _norm(lib, wk=a) == INV
        for a in _ends(out, ROWS, TABLE):
            assert _norm(lib, tab=a) == INV
    # beside it, and shared between what is only read
    assert _norm(lib, wq=QO + ROWS, wk=QO + ROWS, tab=QO - TABLE) == _lib.PRISM_ERR_UNSUPPORTED
    assert _norm(lib, wq=Q, wk=TAB, tab=TAB) == _lib.PRISM_ERR_UNSUPPORTED


def test_norm_gradients(lib):
    ok = _lib.PRISM_ERR_UNSUPPORTED
    n = lib.prism_qk_norm_rope_bwd_workspace_bytes(C.byref(_norm_params()))
    assert _norm_bwd(lib) == ok
    for name, size in (("wq", D * 4), ("wk", D * 4), ("tab", TABLE), ("dwq", D * 4), ("dwk", D * 4), ("ws", n)):
        for at, rows in ((QO, ROWS), (KO, ROWS), (DWQ, D * 4), (DWK, D * 4), (WS, n)):
            if at != dict(dwq=DWQ, dwk=DWK, ws=WS).get(name):
                for a in _ends(at, rows, size):
                    assert _norm_bwd(lib, **{name: a}) == INV, (name, at)
    for name in ("dqo", "dko", "q", "k"):
        for at, size in ((DWQ, D * 4), (DWK, D * 4), (WS, n)):
            for a in _ends(at, size, ROWS):
                assert _norm_bwd(lib, **{name: a}) == INV, (name, at)
    assert _norm_bwd(lib, dwq=QO + ROWS, dwk=QO + ROWS + D * 4, ws=KO + ROWS) == ok
    assert _norm_bwd(lib, dwq=None, dwk=None, ws=QO) == ok          # an unused workspace is not looked at


# ---- projections: [10][136] by [256][136], the operands packed in the workspace
M_, K_, N_ = 10, 136, 256
X, W, B, R, Y, PRE, S, ST, DX, DW, DB = ((i + 1) << 24 for i in range(11))


def _linear_params(**kw):
    base = dict(M=M_, K=K_, N=N_, in_heads=0, out_heads=0, activation=2, out_dtype=0, bias_dtype=1, dw_dtype=1, x_stride=137,
                w_stride=137, y_stride=N_, r_stride=N_)
    base.update(kw)
    return _lib.PrismLinearParams(*[base[f] for f, _ in _lib.PrismLinearParams._fields_])


def test_linear(lib):
    ok, p = _lib.PRISM_ERR_UNSUPPORTED, _linear_params()
    need = lib.prism_linear_workspace_bytes(C.byref(p)) - 256

    def call(x=X, w=W, b=B, r=R, y=Y, pre=PRE, ws=S, st=ST):
        return lib.prism_linear(C.byref(p), x, w, b, r, y, pre, ws, need, st, None)

    assert call() == ok
    sizes = dict(x=(X, ((M_ - 1) * 137 + K_) * 2), w=(W, ((N_ - 1) * 137 + K_) * 2), b=(B, N_ * 4), r=(R, M_ * N_ * 2),
                 y=(Y, M_ * N_ * 2), pre=(PRE, M_ * N_ * 2))
    for at, size in sizes.values():
        for a in (at + 16 - need, at + (size - 1) // 16 * 16):
            assert call(ws=a) == INV
    for at, size in (sizes["y"], sizes["pre"], (S, need)):
        for a in _ends(at, size, 16):
            assert call(st=a) == INV
    assert call(ws=Y + M_ * N_ * 2, st=Y - 16) == ok


def test_linear_gradients(lib):
    ok, p = _lib.PRISM_ERR_UNSUPPORTED, _linear_params()
    need = lib.prism_linear_bwd_workspace_bytes(C.byref(p)) - 256

    def call(dy=Y, x=X, w=W, pre=PRE, dx=DX, dw=DW, db=DB, ws=12 << 24, st=ST):
        return lib.prism_linear_bwd(C.byref(p), dy, x, w, pre, dx, dw, db, ws, need, st, None)

    assert call() == ok
    outs = ((DX, M_ * K_ * 2), (DW, N_ * K_ * 4), (DB, N_ * 4))
    for at, size in ((X, ((M_ - 1) * 137 + K_) * 2), (W, ((N_ - 1) * 137 + K_) * 2), (Y, M_ * N_ * 2), (PRE, M_ * N_ * 2), *outs):
        for a in (at + 16 - need // 16 * 16, at + (size - 1) // 16 * 16):
            assert call(ws=a) == INV
    for at, size in (*outs, (12 << 24, need)):
        for a in _ends(at, size // 16 * 16, 16):
            assert call(st=a) == INV
    assert call(ws=DX + M_ * K_ * 2, st=DW - 16) == ok


def test_binding_refuses_a_workspace_that_is_not_its_bytes():
    """A strided or expanded workspace has fewer bytes in one piece than its elements say."""
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    x, w, q = z(10, 64), z(96, 64), z(2, 24, 64)
    for ws in (z(1, dtype=torch.uint8).expand(1 << 20), z(1 << 20, dtype=torch.uint8)[::2], z(64, 64).t()[:32]):
        for call in (lambda: _lib.linear(x, w, workspace=ws), lambda: _lib.linear_bwd(z(10, 96), x, w, workspace=ws),
                     lambda: _lib.qk_norm_rope_bwd(q, None, q, workspace=ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()


def test_rope_refuses_a_table_that_is_not_its_grids():
    """The kernels read T dim_t + H dim_h + W dim_w consecutive fp32 of it."""
    good = torch.zeros(2 * 16 + 3 * 8 + 4 * 8)
    _lib.Rope(good, 2, 3, 4, (16, 8, 8), 0)
    for table in (good[:-1], good.double(), torch.zeros(1).expand(good.numel()), torch.zeros(2 * good.numel())[::2]):
        with pytest.raises(ValueError, match="table"):
            _lib.Rope(table, 2, 3, 4, (16, 8, 8), 0)
