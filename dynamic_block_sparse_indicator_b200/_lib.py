"""ctypes binding of libprism (include/prism.h): argument marshalling only.

Every step of the plan and of the attention runs in the library's CUDA
kernels; this module passes device pointers, sizes and the current CUDA stream
through, allocates outputs with torch, and raises on a non-zero status.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libprism.so")

PRISM_OK = 0
PRISM_ERR_INVALID_ARG = 1
PRISM_ERR_WORKSPACE = 2
PRISM_ERR_CUDA = 3
PRISM_ERR_TIMEOUT = 4
PRISM_ERR_DEVICE_CHECK = 5
PRISM_ERR_UNSUPPORTED = 6
PRISM_ERR_SCRATCH_LIMIT = 7

PRISM_BF16 = 0
PRISM_F32 = 1

ITEMS = {
    "shape_id": (0, np.uint8), "nblocks": (1, np.int32), "blk_start": (2, np.int32),
    "sel_bits": (3, np.uint32), "row_ptr": (4, np.int32), "col_idx": (5, np.int32),
    "col_ptr": (6, np.int32), "row_idx": (7, np.int32), "qbar": (8, np.float32),
    "kbar": (9, np.float32), "src": (10, np.int32), "zone_stats": (11, np.float32),
    "zone_cut": (12, np.uint8), "shape_id2": (13, np.uint8), "zone_energy": (14, np.float32),
    "region_stats": (15, np.float32), "list_offsets": (16, np.int64), "qkv_max": (17, np.uint32),
}


PRISM_SHAPE_DYNAMIC = 0
PRISM_SHAPE_ISOTROPIC = 1
PRISM_SHAPE_FIXED = 2


class PrismParams(C.Structure):
    _fields_ = [("T", C.c_int32), ("H", C.c_int32), ("W", C.c_int32), ("heads", C.c_int32),
                ("head_dim", C.c_int32), ("dtype", C.c_int32), ("out_dtype", C.c_int32),
                ("top_k", C.c_int32),
                ("top_p", C.c_float), ("eps", C.c_float), ("tau128", C.c_float),
                ("tau256", C.c_float), ("alpha", C.c_float), ("shape_mode", C.c_int32),
                ("fixed_shape", C.c_int32), ("top_k_frac", C.c_float), ("cut_ratio", C.c_float)]


PRISM_PAIR_ADJACENT = 0
PRISM_PAIR_HALVES = 1


class PrismNormRopeParams(C.Structure):
    _fields_ = [("N", C.c_int64), ("T", C.c_int32), ("H", C.c_int32), ("W", C.c_int32), ("heads", C.c_int32),
                ("head_dim", C.c_int32), ("dtype", C.c_int32), ("out_dtype", C.c_int32), ("w_dtype", C.c_int32),
                ("dim_t", C.c_int32), ("dim_h", C.c_int32), ("dim_w", C.c_int32), ("pairing", C.c_int32),
                ("eps", C.c_float)]


class PrismRows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("head_stride", C.c_int64), ("token_stride", C.c_int64)]


PRISM_ACT_NONE = 0
PRISM_ACT_GELU = 1
PRISM_ACT_GELU_TANH = 2
PRISM_ACT_SILU = 3


class PrismLinearParams(C.Structure):
    _fields_ = [("M", C.c_int64), ("K", C.c_int32), ("N", C.c_int32), ("in_heads", C.c_int32), ("out_heads", C.c_int32),
                ("activation", C.c_int32), ("out_dtype", C.c_int32), ("bias_dtype", C.c_int32), ("dw_dtype", C.c_int32),
                ("x_stride", C.c_int64), ("w_stride", C.c_int64), ("y_stride", C.c_int64), ("r_stride", C.c_int64)]


class PrismError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


_lib = None


def load(path: str | None = None) -> C.CDLL:
    """Load libprism.so; raises if it is missing (there is no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or os.environ.get("PRISM_LIB") or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"libprism.so not built at {p}: run "
                          "`python -m dynamic_block_sparse_indicator_b200.build`")
    lib = C.CDLL(p)
    vp, i32, sz = C.c_void_p, C.c_int, C.c_size_t
    pp = C.POINTER(PrismParams)
    sig = {
        "prism_plan_workspace_bytes": (sz, [pp]),
        "prism_plan_core_bytes": (sz, [pp]),
        "prism_plan_list_bytes": (i32, [vp, C.POINTER(sz), vp]),
        "prism_plan_attach_lists": (i32, [vp, vp, sz, vp]),
        "prism_plan": (i32, [pp, vp, vp, vp, vp, vp, sz, vp, C.POINTER(vp)]),
        "prism_plan_sharded": (i32, [pp, C.POINTER(vp), C.POINTER(vp), C.POINTER(vp), i32, i32, i32, vp,
                                     vp, sz, vp, C.POINTER(vp)]),
        "prism_plan_import_sharded": (i32, [pp, C.POINTER(vp), C.POINTER(vp), C.POINTER(vp), i32, i32, i32, vp,
                                            vp, vp, vp, vp, sz, vp, C.POINTER(vp)]),
        "prism_plan_import": (i32, [pp, vp, vp, vp, vp, vp, vp, sz, vp, C.POINTER(vp)]),
        "prism_plan_import_cuts": (i32, [pp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, C.POINTER(vp)]),
        "prism_attn_fwd": (i32, [vp, vp, vp, vp]),
        "prism_attn_fwd_sharded": (i32, [vp, C.POINTER(vp), i32, i32, i32, vp, vp]),
        "prism_attn_bwd_sharded": (i32, [vp, C.POINTER(vp), C.POINTER(vp), vp, C.POINTER(vp), C.POINTER(vp),
                                         C.POINTER(vp), i32, i32, i32, vp]),
        "prism_attn_bwd": (i32, [vp, vp, vp, vp, vp, vp, vp, vp]),
        "prism_plan_item_bytes": (sz, [vp, i32]),
        "prism_plan_export": (i32, [vp, i32, vp, sz, vp]),
        "prism_get_status": (i32, [vp, vp]),
        "prism_get_status_ex": (i32, [vp, C.POINTER(C.c_int32), vp]),
        "prism_selftest_timeout": (i32, [vp, vp]),
        "prism_plan_destroy": (None, [vp]),
        "prism_status_string": (C.c_char_p, [i32]),
        "prism_version": (C.c_char_p, []),
        "prism_profile_enable": (i32, [vp, i32]),
        "prism_profile_plans": (i32, [i32]),
        "prism_profile_read": (i32, [vp, C.POINTER(C.c_float), C.POINTER(C.c_int), vp]),
        "prism_launch_count": (C.c_int64, [vp]),
        "prism_zone_shapes_noalloc": (i32, [pp, vp, vp, vp, vp, vp]),
        "prism_av_norm": (i32, [C.c_int64, C.c_int32, C.c_int32, C.c_int32, vp, vp, vp, vp, vp,
                                C.c_int32, vp, vp]),
        "prism_linear_workspace_bytes": (sz, [C.POINTER(PrismLinearParams)]),
        "prism_linear": (i32, [C.POINTER(PrismLinearParams), vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]),
        "prism_linear_bwd_workspace_bytes": (sz, [C.POINTER(PrismLinearParams)]),
        "prism_linear_bwd": (i32, [C.POINTER(PrismLinearParams), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]),
        "prism_rope_table": (i32, [C.POINTER(PrismNormRopeParams), C.c_float, C.c_int64, vp, vp]),
        "prism_qk_norm_rope": (i32, [C.POINTER(PrismNormRopeParams), C.POINTER(PrismRows), C.POINTER(PrismRows), vp, vp,
                                     vp, C.POINTER(PrismRows), C.POINTER(PrismRows), vp]),
        "prism_qk_norm_rope_bwd_workspace_bytes": (sz, [C.POINTER(PrismNormRopeParams)]),
        "prism_qk_norm_rope_bwd": (i32, [C.POINTER(PrismNormRopeParams), C.POINTER(PrismRows), C.POINTER(PrismRows),
                                         C.POINTER(PrismRows), C.POINTER(PrismRows), vp, vp, vp, C.POINTER(PrismRows),
                                         C.POINTER(PrismRows), vp, vp, vp, sz, vp]),
        "prism_status_read": (i32, [vp, C.POINTER(C.c_int32), vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def profile_plans(on: bool = True) -> bool:
    """Plans created afterwards time their own plan kernels (process-wide); returns the old setting."""
    return bool(load().prism_profile_plans(1 if on else 0))


def status_string(st: int) -> str:
    return load().prism_status_string(st).decode()


def make_params(T, H, W, heads, head_dim, dtype, top_k, top_p, eps, tau128=0.5, tau256=0.25,
                out_dtype=PRISM_F32, alpha=0.5, shape_mode=PRISM_SHAPE_DYNAMIC, fixed_shape=0,
                top_k_frac=0.0, cut_ratio=0.0):
    return PrismParams(T, H, W, heads, head_dim, dtype, out_dtype, top_k, float(top_p),
                       float(eps), float(tau128), float(tau256), float(alpha), int(shape_mode),
                       int(fixed_shape), float(top_k_frac), float(cut_ratio))


def workspace_bytes(params: PrismParams) -> int:
    """Workspace of a plan ready in one call (index lists at their dense bound)."""
    return int(load().prism_plan_workspace_bytes(C.byref(params)))


def core_bytes(params: PrismParams) -> int:
    """Workspace without the index lists (they go to a second buffer sized after planning)."""
    return int(load().prism_plan_core_bytes(C.byref(params)))


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _addresses(xs):
    """A ctypes array of device addresses from tensors or ints."""
    return (C.c_void_p * len(xs))(*[x if isinstance(x, int) else x.data_ptr() for x in xs])


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


class Plan:
    """A plan handle plus the device buffers it points into (kept alive here)."""

    def __init__(self, params, handle, workspace, inputs, lists=None):
        self.params = params
        self._h = handle
        self._ws = workspace
        self._lists = lists            # the index lists' buffer of a two-call plan
        self._inputs = inputs          # Q, K, V must outlive the plan

    @property
    def handle(self):
        return self._h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            _lib.prism_plan_destroy(h)
            self._h = None

    @property
    def N(self):
        p = self.params
        return p.T * p.H * p.W

    def _out_dtype(self):
        import torch
        return torch.float32 if self.params.out_dtype == PRISM_F32 else torch.bfloat16

    def attn_fwd(self, O=None, lse=None, stream=None):
        import torch
        p = self.params
        dev = self._ws.device
        if O is None:
            O = torch.empty(p.heads, self.N, p.head_dim, dtype=self._out_dtype(), device=dev)
        if lse is None:
            lse = torch.empty(p.heads, self.N, dtype=torch.float32, device=dev)
        st = load().prism_attn_fwd(self._h, _ptr(O), _ptr(lse), _stream(stream))
        if st:
            raise PrismError(st, "prism_attn_fwd")
        return O, lse

    def attn_bwd(self, dO, O, lse, dQ=None, dK=None, dV=None, stream=None):
        import torch
        p = self.params
        dev = self._ws.device
        mk = lambda: torch.empty(p.heads, self.N, p.head_dim, dtype=self._out_dtype(), device=dev)
        dQ = mk() if dQ is None else dQ
        dK = mk() if dK is None else dK
        dV = mk() if dV is None else dV
        st = load().prism_attn_bwd(self._h, _ptr(dO), _ptr(O), _ptr(lse), _ptr(dQ), _ptr(dK),
                                   _ptr(dV), _stream(stream))
        if st:
            raise PrismError(st, "prism_attn_bwd")
        return dQ, dK, dV

    def attn_fwd_sharded(self, O_shards, head0, heads_total, lse=None, stream=None):
        """The forward writing O into token shards (lists of [heads_total, N/n, D] tensors or
        device addresses, shard s = frames [s T/n, (s + 1) T/n)): rows of this plan's heads
        head0 .. head0 + heads - 1.  The LSE stays [heads, N] on this device."""
        import torch
        p = self.params
        if lse is None:
            lse = torch.empty(p.heads, self.N, dtype=torch.float32, device=self._ws.device)
        arr = _addresses(O_shards)
        st = load().prism_attn_fwd_sharded(self._h, arr, len(O_shards), int(heads_total), int(head0), _ptr(lse),
                                           _stream(stream))
        if st:
            raise PrismError(st, "prism_attn_fwd_sharded")
        return lse

    def attn_bwd_sharded(self, dO_shards, O_shards, lse, dQ_shards, dK_shards, dV_shards, head0, heads_total,
                         stream=None):
        """The backward reading dO and O from token shards and writing dQ, dK, dV into token
        shards (the layout of attn_fwd_sharded)."""
        n = len(dO_shards)
        if not all(len(x) == n for x in (O_shards, dQ_shards, dK_shards, dV_shards)):
            raise ValueError("every shard list must have the same length")
        st = load().prism_attn_bwd_sharded(self._h, _addresses(dO_shards), _addresses(O_shards), _ptr(lse),
                                           _addresses(dQ_shards), _addresses(dK_shards), _addresses(dV_shards),
                                           n, int(heads_total), int(head0), _stream(stream))
        if st:
            raise PrismError(st, "prism_attn_bwd_sharded")

    def export(self, item: str, stream=None) -> np.ndarray:
        code, dt = ITEMS[item]
        lib = load()
        nbytes = int(lib.prism_plan_item_bytes(self._h, code))
        out = np.empty(nbytes // np.dtype(dt).itemsize, dtype=dt)
        st = lib.prism_plan_export(self._h, code, out.ctypes.data_as(C.c_void_p), nbytes,
                                   _stream(stream))
        if st:
            raise PrismError(st, f"prism_plan_export({item})")
        return out

    STAGES = ("fwd", "bwd_pre", "bwd_dkdv", "bwd_dq", "plan_stats", "plan_shapes", "plan_gather",
              "plan_select", "plan_lists")

    def profile(self, on: bool = True):
        load().prism_profile_enable(self._h, 1 if on else 0)

    def profile_read(self, stream=None):
        """{stage: (ms, launches)} accumulated since the last read (synchronises)."""
        ms = (C.c_float * len(self.STAGES))()
        n = (C.c_int * len(self.STAGES))()
        st = load().prism_profile_read(self._h, ms, n, _stream(stream))
        if st:
            raise PrismError(st, "prism_profile_read")
        return {k: (float(ms[i]), int(n[i])) for i, k in enumerate(self.STAGES)}

    def launches(self) -> int:
        return int(load().prism_launch_count(self._h))

    def status(self, stream=None) -> int:
        return int(load().prism_get_status(self._h, _stream(stream)))

    def status_ex(self, stream=None):
        """(status, site of a timed-out wait) -- synchronises and clears."""
        site = C.c_int32(0)
        st = load().prism_get_status_ex(self._h, C.byref(site), _stream(stream))
        return int(st), int(site.value)

    def selftest_timeout(self, stream=None):
        st = load().prism_selftest_timeout(self._h, _stream(stream))
        if st:
            raise PrismError(st, "prism_selftest_timeout")


def _check_inputs(Q, K, V, params):
    import torch
    want = torch.float32 if params.dtype == PRISM_F32 else torch.bfloat16
    N = params.T * params.H * params.W
    for t in (Q, K, V):
        if t.dtype != want or not t.is_cuda or not t.is_contiguous():
            raise ValueError("Q, K, V must be contiguous CUDA tensors of the plan's dtype")
        if tuple(t.shape) != (params.heads, N, params.head_dim):
            raise ValueError(f"expected [heads, N, D] = {(params.heads, N, params.head_dim)}, "
                             f"got {tuple(t.shape)}")


def _attach_lists(lib, h, device, stream):
    """Size and build a two-call plan's index lists in a buffer of their own."""
    import torch
    nbytes = C.c_size_t(0)
    st = lib.prism_plan_list_bytes(h, C.byref(nbytes), _stream(stream))
    if st:
        raise PrismError(st, "prism_plan_list_bytes")
    lists = torch.empty(max(int(nbytes.value), 16), dtype=torch.uint8, device=device)
    st = lib.prism_plan_attach_lists(h, _ptr(lists), lists.numel(), _stream(stream))
    if st:
        raise PrismError(st, "prism_plan_attach_lists")
    return lists


def plan(Q, K, V, a_map, params: PrismParams, workspace=None, stream=None, compact=False) -> Plan:
    """Stages 1-3 on the GPU.  Q, K, V: [heads, N, D] CUDA tensors (raster order).
    compact=True plans with the core workspace and sizes the index lists from
    their counts (one stream synchronisation) instead of their dense bound."""
    import torch
    lib = load()
    _check_inputs(Q, K, V, params)
    need = core_bytes(params) if compact else workspace_bytes(params)
    if need == 0:
        raise PrismError(PRISM_ERR_INVALID_ARG, "prism_plan_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    h = C.c_void_p()
    st = lib.prism_plan(C.byref(params), _ptr(Q), _ptr(K), _ptr(V), _ptr(a_map), _ptr(workspace),
                        workspace.numel(), _stream(stream), C.byref(h))
    if st:
        raise PrismError(st, "prism_plan")
    lists = None
    if workspace.numel() < workspace_bytes(params):
        try:
            lists = _attach_lists(lib, h, Q.device, stream)
        except PrismError:
            lib.prism_plan_destroy(h)
            raise
    return Plan(params, h, workspace, (Q, K, V, a_map), lists)


def _shard_args(Qs, Ks, Vs, params, heads_total):
    """Checks a shard layout; returns (address arrays, heads_total, device, tensors)."""
    import torch
    n = len(Qs)
    if n == 0 or len(Ks) != n or len(Vs) != n:
        raise ValueError("Qs, Ks, Vs must be non-empty lists of the same length")
    N = params.T * params.H * params.W
    if params.T % n:
        raise ValueError(f"{n} shards do not divide T = {params.T}")
    want = torch.float32 if params.dtype == PRISM_F32 else torch.bfloat16
    device, tensors = None, []
    for t in (*Qs, *Ks, *Vs):
        if isinstance(t, int):
            continue
        if t.dtype != want or not t.is_cuda or not t.is_contiguous():
            raise ValueError("shards must be contiguous CUDA tensors of the plan's dtype (or device addresses)")
        if heads_total is None:
            heads_total = t.shape[0]
        if tuple(t.shape) != (heads_total, N // n, params.head_dim):
            raise ValueError(f"expected shards of [heads_total, N/shards, D] = "
                             f"{(heads_total, N // n, params.head_dim)}, got {tuple(t.shape)}")
        device = device or t.device
        tensors.append(t)
    if heads_total is None:
        raise ValueError("heads_total is needed when every shard is given as an address")
    device = device or torch.device("cuda", torch.cuda.current_device())
    return [_addresses(xs) for xs in (Qs, Ks, Vs)], int(heads_total), device, tuple(tensors)


def plan_import_sharded(Qs, Ks, Vs, shape_id, sel_bits, params: PrismParams, head0=0, heads_total=None,
                        zone_cut=None, shape_id2=None, workspace=None, stream=None, compact=False) -> Plan:
    """plan_import for inputs held as token shards (the layout of plan_sharded)."""
    import torch
    lib = load()
    arrs, heads_total, device, tensors = _shard_args(Qs, Ks, Vs, params, heads_total)
    need = core_bytes(params) if compact else workspace_bytes(params)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    h = C.c_void_p()
    st = lib.prism_plan_import_sharded(C.byref(params), arrs[0], arrs[1], arrs[2], len(Qs), heads_total,
                                       int(head0), _ptr(shape_id), _ptr(zone_cut), _ptr(shape_id2),
                                       _ptr(sel_bits), _ptr(workspace), workspace.numel(), _stream(stream),
                                       C.byref(h))
    if st:
        raise PrismError(st, "prism_plan_import_sharded")
    lists = None
    if workspace.numel() < workspace_bytes(params):
        try:
            lists = _attach_lists(lib, h, device, stream)
        except PrismError:
            lib.prism_plan_destroy(h)
            raise
    return Plan(params, h, workspace, (tensors, shape_id, sel_bits, zone_cut, shape_id2), lists)


def plan_sharded(Qs, Ks, Vs, a_map, params: PrismParams, head0=0, heads_total=None, workspace=None,
                 stream=None, compact=False) -> Plan:
    """Stages 1-3 for heads head0 .. head0 + params.heads - 1 of inputs held as
    token shards: Qs, Ks, Vs are equal-length lists (one entry per shard, shard s
    holding frames [s T/n, (s + 1) T/n) of every head as [heads_total, N/n, D]),
    each a contiguous CUDA tensor or a raw device address (an int: another GPU's
    shard mapped for peer access).  The plan then runs like `plan` on those heads."""
    import torch
    lib = load()
    arrs, heads_total, device, tensors = _shard_args(Qs, Ks, Vs, params, heads_total)
    n = len(Qs)
    need = core_bytes(params) if compact else workspace_bytes(params)
    if need == 0:
        raise PrismError(PRISM_ERR_INVALID_ARG, "prism_plan_workspace_bytes")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    h = C.c_void_p()
    st = lib.prism_plan_sharded(C.byref(params), arrs[0], arrs[1], arrs[2], n, int(heads_total), int(head0),
                                _ptr(a_map), _ptr(workspace), workspace.numel(), _stream(stream), C.byref(h))
    if st:
        raise PrismError(st, "prism_plan_sharded")
    lists = None
    if workspace.numel() < workspace_bytes(params):
        try:
            lists = _attach_lists(lib, h, device, stream)
        except PrismError:
            lib.prism_plan_destroy(h)
            raise
    return Plan(params, h, workspace, (tensors, a_map), lists)


def plan_import(Q, K, V, shape_id, sel_bits, params: PrismParams, workspace=None, stream=None,
                zone_cut=None, shape_id2=None, compact=False) -> Plan:
    """A plan from given shape ids [heads, Nz] (uint8) and selection bitmap (int32/uint32 words);
    with adaptive temporal boundaries also the split frames zone_cut and the second parts'
    shapes shape_id2 ([heads, Nz] uint8 each)."""
    import torch
    lib = load()
    _check_inputs(Q, K, V, params)
    need = core_bytes(params) if compact else workspace_bytes(params)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    h = C.c_void_p()
    if zone_cut is None:
        st = lib.prism_plan_import(C.byref(params), _ptr(Q), _ptr(K), _ptr(V), _ptr(shape_id),
                                   _ptr(sel_bits), _ptr(workspace), workspace.numel(), _stream(stream),
                                   C.byref(h))
    else:
        st = lib.prism_plan_import_cuts(C.byref(params), _ptr(Q), _ptr(K), _ptr(V), _ptr(shape_id),
                                        _ptr(zone_cut), _ptr(shape_id2), _ptr(sel_bits), _ptr(workspace),
                                        workspace.numel(), _stream(stream), C.byref(h))
    if st:
        raise PrismError(st, "prism_plan_import")
    lists = None
    if workspace.numel() < workspace_bytes(params):
        try:
            lists = _attach_lists(lib, h, Q.device, stream)
        except PrismError:
            lib.prism_plan_destroy(h)
            raise
    return Plan(params, h, workspace, (Q, K, V, shape_id, sel_bits, zone_cut, shape_id2), lists)


def av_norm(Qv, Ka, Va, a_map=None, h_hat=None, hhat_dtype=None, want_hhat=False, status=None,
            stream=None):
    """The guidance map a [N] (fp32) = || CrossAttn(Qv, Ka, Va) ||_2 over the heads, and
    optionally h_hat [heads, N, D].  Qv [heads, N, D], Ka, Va [heads, M, D]: contiguous
    bf16 CUDA tensors.  `status` is a device int32[4] block (zeroed here when created);
    read it with status_read()."""
    import torch
    for t in (Qv, Ka, Va):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 3:
            raise ValueError("Qv, Ka, Va must be contiguous 3-D bf16 CUDA tensors")
    heads, N, D = Qv.shape
    M = Ka.shape[1]
    if tuple(Ka.shape) != (heads, M, D) or tuple(Va.shape) != (heads, M, D):
        raise ValueError(f"Ka, Va must be [heads, M, D] = [{heads}, M, {D}]")
    dev = Qv.device
    if a_map is None:
        a_map = torch.empty(N, dtype=torch.float32, device=dev)
    if hhat_dtype is None:
        hhat_dtype = PRISM_BF16 if h_hat is None or h_hat.dtype == torch.bfloat16 else PRISM_F32
    if h_hat is None and want_hhat:
        dt = torch.float32 if hhat_dtype == PRISM_F32 else torch.bfloat16
        h_hat = torch.empty(heads, N, D, dtype=dt, device=dev)
    if status is None:
        status = torch.zeros(4, dtype=torch.int32, device=dev)
    st = load().prism_av_norm(int(N), int(M), int(heads), int(D), _ptr(Qv), _ptr(Ka), _ptr(Va),
                              _ptr(a_map), _ptr(h_hat), int(hhat_dtype), _ptr(status),
                              _stream(stream))
    if st:
        raise PrismError(st, "prism_av_norm")
    return a_map, h_hat, status


def status_read(status, stream=None):
    """(status, site) of a device status block; synchronises and clears it."""
    site = C.c_int32(0)
    st = load().prism_status_read(_ptr(status), C.byref(site), _stream(stream))
    return int(st), int(site.value)


# ---- the layer's operators around the attention -----------------------------------------

_codes: dict = {}


def _code(dtype, what):
    """PRISM_BF16 / PRISM_F32 of a torch dtype."""
    if not _codes:
        import torch
        _codes.update({torch.bfloat16: PRISM_BF16, torch.float32: PRISM_F32})
    code = _codes.get(dtype)
    if code is None:
        raise ValueError(f"{what} must be bfloat16 or float32, got {dtype}")
    return code


class _Launch:
    """The device and stream of a call.  The library is called with the tensors' device current.
    Where the call runs on another stream than torch's current one, what it allocates comes from
    that stream (memory that the current stream may still be using is not written) and counts as
    used by both, and the tensors given count as used there: none is handed out again before that
    work is done.  Ordering the two streams is the caller's, as everywhere."""
    __slots__ = ("first", "tensors", "device", "s", "cur", "other", "stream", "guard")

    def __init__(self, tensors, stream):
        import torch
        first = self.first = tensors[0]
        d = first.get_device()
        for t in tensors:
            if t is not None and (t.get_device() != d or d < 0):
                raise ValueError("the tensors must be on one CUDA device")
        self.tensors = tensors
        self.guard = None
        if torch.cuda.current_device() != d:
            self.guard = torch.cuda.device(d)
        self.other = False
        if stream is None:
            self.s = self.cur = None
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            self.stream = raw(d) if raw is not None else torch.cuda.current_stream(d).cuda_stream
        else:
            if stream.device.index != d:
                raise ValueError(f"the stream is on {stream.device}, the tensors are on {first.device}")
            self.s, self.cur = stream, torch.cuda.current_stream(d)
            self.stream = stream.cuda_stream
            self.other = self.stream != self.cur.cuda_stream

    def empty(self, shape, dtype):
        """Memory for the call."""
        if not self.other:
            return self.first.new_empty(shape, dtype=dtype)
        import torch
        with torch.cuda.stream(self.s):
            t = self.first.new_empty(shape, dtype=dtype)
        t.record_stream(self.cur)
        return t

    def zero_status(self):
        """A device status block for the call, cleared on its stream."""
        import torch
        if not self.other:
            return self.first.new_zeros(4, dtype=torch.int32)
        with torch.cuda.stream(self.s):
            t = self.first.new_zeros(4, dtype=torch.int32)
        t.record_stream(self.cur)
        return t

    def call(self, what, fn, *args):
        """fn(*args, stream) with the device current; raises on a status."""
        if self.guard is None:
            status = fn(*args, self.stream)
        else:
            with self.guard:
                status = fn(*args, self.stream)
        if status:
            raise PrismError(status, what)
        if self.other:
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.s)


def _at(t):
    """A tensor's address, or None."""
    return None if t is None else t.data_ptr()


class Rope:
    """A rotation table on the device with the grid and channels it belongs to (make_rope)."""

    def __init__(self, table, T, H, W, dims, pairing):
        import torch
        n = T * dims[0] + H * dims[1] + W * dims[2]
        if table.dtype != torch.float32 or not table.is_contiguous() or table.numel() < n:
            raise ValueError(f"the table must be {n} consecutive fp32")
        self.table, self.T, self.H, self.W, self.dims, self.pairing = table, T, H, W, tuple(dims), pairing

    def __repr__(self):
        return f"Rope({self.T} x {self.H} x {self.W}, channels {self.dims}, pairing {self.pairing})"


def _norm_rope_params(N, heads, D, dtype, out_dtype, w_dtype, rope, eps):
    r = (rope.T, rope.H, rope.W, *rope.dims, rope.pairing) if rope is not None else (0, 0, 0, 0, 0, 0, 0)
    return PrismNormRopeParams(N, r[0], r[1], r[2], heads, D, dtype, out_dtype, w_dtype, r[3], r[4], r[5], r[6],
                               float(eps))


def make_rope(T, H, W, dims, theta=10000.0, pairing=PRISM_PAIR_ADJACENT, first_frame=0, device=None, stream=None) -> Rope:
    """The rotation of a T x H x W grid whose axes turn dims = (dim_t, dim_h, dim_w) channels
    of each head (made once per grid; a 1-D sequence is (N, 1, 1) with dims (d, 0, 0))."""
    import torch
    dims = tuple(int(d) for d in dims)
    if len(dims) != 3 or any(d < 0 or d % 2 for d in dims) or min(T, H, W) < 1:
        raise ValueError(f"dims must be three even counts of channels and T, H, W positive, got {dims} and {(T, H, W)}")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.stream(stream):          # (None: the current one)
        table = torch.empty(max(T * dims[0] + H * dims[1] + W * dims[2], 4), dtype=torch.float32, device=dev)
    if stream is not None:                   # (its memory is that stream's, its readers the current one)
        table.record_stream(torch.cuda.current_stream(dev))
    rope = Rope(table, int(T), int(H), int(W), dims, int(pairing))
    D = 64 if sum(dims) <= 64 else 128
    p = _norm_rope_params(T * H * W, 1, D, PRISM_BF16, PRISM_BF16, PRISM_F32, rope, 1.0)
    _Launch([table], stream).call("prism_rope_table", load().prism_rope_table, C.byref(p), float(theta), int(first_frame),
                                  table.data_ptr())
    return rope


def _rows(t, what):
    """A pointer to the rows of [heads, N, D], or None."""
    if t is None:
        return None
    hs, ts, cs = t.stride()
    if cs != 1 and t.shape[2] > 1:
        raise ValueError(f"{what} must be [heads, N, D] with consecutive channels (any head and token strides)")
    return C.byref(PrismRows(t.data_ptr(), hs, ts))


def _weights(ws, D, what):
    ws = [w for w in ws if w is not None]
    for w in ws:
        if w.shape != (D,) or not w.is_contiguous() or w.dtype != ws[0].dtype:
            raise ValueError(f"{what} must be contiguous vectors of the {D} channels, of one type")
    return _code(ws[0].dtype, what) if ws else PRISM_F32


def _qk_pair(named, rope):
    """Checks a list of (name, query side, key side); returns heads, N, D."""
    shape = named[0][1].shape
    if len(shape) != 3:
        raise ValueError("q must be [heads, N, D]")
    alone = named[0][2] is None
    for name, a, b in named:
        if a.shape != shape or (b is not None and b.shape != shape):
            raise ValueError(f"{name}: expected [heads, N, D] = {tuple(shape)}")
        if (b is None) != alone:
            raise ValueError("the key's tensors must all be given or none")
        if b is not None and b.dtype != a.dtype:
            raise ValueError(f"{name}: query and key must be of one type")
    heads, N, D = shape
    if rope is not None and rope.T * rope.H * rope.W != N:
        raise ValueError(f"the rotation is for {rope.T} x {rope.H} x {rope.W} tokens, q has {N}")
    return heads, N, D


def qk_norm_rope(q, k=None, wq=None, wk=None, rope=None, eps=1e-6, q_out=None, k_out=None, out_dtype=None, stream=None):
    """(q_out, k_out): every head's rows of q and k [heads, N, D] scaled to unit root mean square,
    multiplied by the weights [D] and rotated by `rope` (make_rope), each where given.  q and k are
    bf16 or fp32 CUDA tensors of any head and token strides (slices of a fused projection); the
    results are contiguous [heads, N, D] of out_dtype (q's type if not given), as `plan` takes them,
    or the q_out, k_out given (of any strides; a result may be its own input)."""
    import torch
    out_dtype = out_dtype or (q_out.dtype if q_out is not None else q.dtype)
    named = [("q, k", q, k)]
    if q_out is None:
        if k_out is not None:
            raise ValueError("k_out without q_out")
    else:
        named.append(("q_out, k_out", q_out, k_out))
        if q_out.dtype != out_dtype:
            raise ValueError(f"q_out is {q_out.dtype}, out_dtype is {out_dtype}")
    heads, N, D = _qk_pair(named, rope)
    if wk is not None and k is None:
        raise ValueError("wk without k")
    dt, odt, wdt = _code(q.dtype, "q"), _code(out_dtype, "the result"), _weights((wq, wk), D, "wq and wk")
    table = None if rope is None else rope.table
    go = _Launch((q, k, wq, wk, q_out, k_out, table), stream)
    if q_out is None:
        q_out = go.empty(q.shape, out_dtype)
        k_out = go.empty(k.shape, out_dtype) if k is not None else None
    p = _norm_rope_params(N, heads, D, dt, odt, wdt, rope, eps)
    go.call("prism_qk_norm_rope", load().prism_qk_norm_rope, C.byref(p), _rows(q, "q"), _rows(k, "k"), _at(wq), _at(wk),
            _at(table), _rows(q_out, "q_out"), _rows(k_out, "k_out"))
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k=None, wq=None, wk=None, rope=None, eps=1e-6, dq=None, dk=None,
                     want_dw=True, workspace=None, stream=None):
    """(dq, dk, dwq, dwk): the gradients of qk_norm_rope by q, k (of their types, token-major as q is if q
    is, or the dq, dk given) and by the weights (fp32 [D] for each weight given), from the gradients
    dq_out, dk_out by its results and its own inputs."""
    import torch
    named = [("q, k", q, k), ("dq_out, dk_out", dq_out, dk_out)]
    if dq is None:
        if dk is not None:
            raise ValueError("dk without dq")
    else:
        named.append(("dq, dk", dq, dk))
        if dq.dtype != q.dtype:
            raise ValueError(f"dq is {dq.dtype}, q is {q.dtype}")
    heads, N, D = _qk_pair(named, rope)
    if wk is not None and k is None:
        raise ValueError("wk without k")
    dt, gdt, wdt = _code(q.dtype, "q"), _code(dq_out.dtype, "dq_out"), _weights((wq, wk), D, "wq and wk")
    table = None if rope is None else rope.table
    ws_bytes = _size(workspace)
    go = _Launch((q, k, dq_out, dk_out, wq, wk, dq, dk, workspace, table), stream)

    def like(x):
        """Dense, in the order of x's strides: token-major rows stay token-major."""
        if x.stride(1) > x.stride(0):
            return go.empty((N, heads, D), x.dtype).transpose(0, 1)
        return go.empty((heads, N, D), x.dtype)

    if dq is None:
        dq = like(q)
        dk = like(k) if k is not None else None
    dwq = go.empty((D,), torch.float32) if want_dw and wq is not None else None
    dwk = go.empty((D,), torch.float32) if want_dw and wk is not None else None
    p = _norm_rope_params(N, heads, D, dt, gdt, wdt, rope, eps)
    lib = load()
    if workspace is None and (dwq is not None or dwk is not None):
        ws_bytes = max(int(lib.prism_qk_norm_rope_bwd_workspace_bytes(C.byref(p))), 16)
        workspace = go.empty((ws_bytes,), torch.uint8)
    go.call("prism_qk_norm_rope_bwd", lib.prism_qk_norm_rope_bwd, C.byref(p), _rows(dq_out, "dq_out"),
            _rows(dk_out, "dk_out"), _rows(q, "q"), _rows(k, "k"), _at(wq), _at(wk), _at(table), _rows(dq, "dq"),
            _rows(dk, "dk"), _at(dwq), _at(dwk), _at(workspace), ws_bytes)
    return dq, dk, dwq, dwk


def _features(t, what, dtype=None):
    """(rows M, features, heads, row stride) of rows [M, F] or a contiguous [heads, M, D]."""
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if t.dim() == 2:
        M, F = t.shape
        if F > 1 and t.stride(1) != 1:
            raise ValueError(f"{what}: the features of a row must be consecutive")
        stride = t.stride(0) if M > 1 else F
        if stride < F:
            raise ValueError(f"{what}: rows must not overlap")
        return M, F, 0, stride
    if t.dim() == 3:
        if not t.is_contiguous() or t.shape[2] not in (64, 128) or t.shape[0] < 1:
            raise ValueError(f"{what}: head-major tensors are contiguous [heads, M, 64 or 128]")
        return t.shape[1], t.shape[0] * t.shape[2], t.shape[0], t.shape[0] * t.shape[2]
    raise ValueError(f"{what} must be [M, features] or [heads, M, D]")


def _shape_like(M, F, heads):
    return (heads, M, F // heads) if heads else (M, F)


def _in_layout(t, what, shape, dtype):
    """The row stride of a tensor that must have this shape and type."""
    if t.shape != shape:
        raise ValueError(f"{what}: expected {shape}, got {tuple(t.shape)}")
    return _features(t, what, dtype)[3]


def _size(workspace):
    """Bytes of a workspace."""
    if workspace is None:
        return 0
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.numel() * workspace.element_size()


def _check_status(t):
    import torch
    if t is not None and (t.dtype != torch.int32 or t.numel() < 4 or not t.is_contiguous()):
        raise ValueError("status must be four contiguous int32")


def linear(x, W, bias=None, residual=None, activation=PRISM_ACT_NONE, y=None, out_dtype=None, out_heads=0, pre=None,
           want_pre=False, workspace=None, status=None, stream=None):
    """(y, pre, status): y = act(x W^T + bias) + residual.  x is bf16 rows [M, K] (any row stride) or
    head-major [heads, M, D]; W bf16 [N, K]; bias [N]; y and residual are rows [M, N], or head-major
    [out_heads, M, N / out_heads] where out_heads is given (a given y or residual says it too), of
    out_dtype (bf16 if nothing says otherwise).  A given y may be the residual.  pre is the bf16
    x W^T + bias for linear_bwd, if wanted.  `status` as in av_norm."""
    import torch
    M, K, in_heads, xs = _features(x, "x", torch.bfloat16)
    N, WK, wh, ws_ = _features(W, "W", torch.bfloat16)
    if wh or WK != K:
        raise ValueError(f"W must be [N, {K}], got {tuple(W.shape)}")
    like = y if y is not None else residual
    if like is not None:
        out_dtype = out_dtype or like.dtype
        if like.dim() == 3:
            out_heads = out_heads or like.shape[0]
    out_dtype = out_dtype or torch.bfloat16
    if out_heads and (out_heads < 0 or N % out_heads or N // out_heads not in (64, 128)):
        raise ValueError(f"{N} features are not {out_heads} heads of 64 or 128 channels")
    want = _shape_like(M, N, out_heads)
    y_stride = N if y is None else _in_layout(y, "y", want, out_dtype)
    r_stride = N if residual is None else _in_layout(residual, "residual", want, out_dtype)
    if pre is not None and (pre.shape != want or pre.dtype != torch.bfloat16 or not pre.is_contiguous()):
        raise ValueError(f"pre must be a contiguous bf16 {want}")
    if bias is not None and (bias.shape != (N,) or not bias.is_contiguous()):
        raise ValueError(f"bias must be [{N}]")
    p = PrismLinearParams(M, K, N, in_heads, out_heads, int(activation), _code(out_dtype, "y"),
                          PRISM_F32 if bias is None else _code(bias.dtype, "bias"), PRISM_F32, xs, ws_, y_stride, r_stride)
    _check_status(status)
    ws_bytes = _size(workspace)
    lib = load()
    go = _Launch((x, W, bias, residual, y, pre, workspace, status), stream)
    if y is None:
        y = go.empty(want, out_dtype)
    if want_pre and pre is None:
        pre = go.empty(want, torch.bfloat16)
    if workspace is None and (xs % 8 or ws_ % 8):
        ws_bytes = max(int(lib.prism_linear_workspace_bytes(C.byref(p))), 16)
        workspace = go.empty((ws_bytes,), torch.uint8)
    if status is None:
        status = go.zero_status()
    go.call("prism_linear", lib.prism_linear, C.byref(p), x.data_ptr(), W.data_ptr(), _at(bias), _at(residual),
            y.data_ptr(), _at(pre), _at(workspace), ws_bytes, status.data_ptr())
    return y, pre, status


def linear_bwd(dy, x, W, pre=None, activation=PRISM_ACT_NONE, dx=None, dW=None, db=None, want_dx=True, want_dw=True,
               want_db=True, dw_dtype=None, workspace=None, status=None, stream=None):
    """(dx, dW, db, status): the gradients of linear by x (bf16, in x's layout), W ([N, K] of dw_dtype,
    fp32 if not given) and bias (fp32 [N]), each where wanted, from dy (in y's layout), the forward's x
    and W, and with an activation its `pre`.  The residual's gradient is dy.  An fp32 dW through an
    activation or from an fp32 dy takes two products; a bf16 one holds dz rounded to bf16 and takes one."""
    import torch
    M, K, in_heads, xs = _features(x, "x", torch.bfloat16)
    N, WK, wh, ws_ = _features(W, "W", torch.bfloat16)
    Mo, No, out_heads, ys = _features(dy, "dy")
    if wh or WK != K:
        raise ValueError(f"W must be [N, {K}], got {tuple(W.shape)}")
    if (Mo, No) != (M, N):
        raise ValueError(f"dy has {Mo} rows of {No} features, expected {M} of {N}")
    want = _shape_like(M, N, out_heads)
    if activation != PRISM_ACT_NONE:
        if pre is None or pre.shape != want or pre.dtype != torch.bfloat16 or not pre.is_contiguous():
            raise ValueError(f"the activation's gradient needs pre, a contiguous bf16 {want}")
    else:
        pre = None
    dw_dtype = dw_dtype or (dW.dtype if dW is not None else torch.float32)
    for t, shape, dtype, what in ((dx, tuple(x.shape), torch.bfloat16, "dx"), (dW, (N, K), dw_dtype, "dW"),
                                  (db, (N,), torch.float32, "db")):
        if t is not None and (tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous()):
            raise ValueError(f"{what} must be a contiguous {dtype} {shape}")
    # (an fp32 dW may take a second part of dz in the workspace: not where none is wanted)
    dw_code = _code(dw_dtype, "dW") if want_dw or dW is not None else PRISM_BF16
    p = PrismLinearParams(M, K, N, in_heads, out_heads, int(activation), _code(dy.dtype, "dy"), PRISM_F32, dw_code, xs, ws_,
                          ys, N)
    _check_status(status)
    ws_bytes = _size(workspace)
    lib = load()
    go = _Launch((dy, x, W, pre, dx, dW, db, workspace, status), stream)
    if dx is None and want_dx:
        dx = go.empty(x.shape, torch.bfloat16)
    if dW is None and want_dw:
        dW = go.empty((N, K), dw_dtype)
    if db is None and want_db:
        db = go.empty((N,), torch.float32)
    if workspace is None:
        ws_bytes = max(int(lib.prism_linear_bwd_workspace_bytes(C.byref(p))), 16)
        workspace = go.empty((ws_bytes,), torch.uint8)
    if status is None:
        status = go.zero_status()
    go.call("prism_linear_bwd", lib.prism_linear_bwd, C.byref(p), dy.data_ptr(), x.data_ptr(), W.data_ptr(), _at(pre),
            _at(dx), _at(dW), _at(db), _at(workspace), ws_bytes, status.data_ptr())
    return dx, dW, db, status
