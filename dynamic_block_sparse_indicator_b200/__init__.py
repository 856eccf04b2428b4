"""Prism dynamic block-sparse video self-attention for NVIDIA B200 (sm_100a).

The compute lives in libprism.so (CUDA kernels behind the C ABI declared in
include/prism.h); this package is the thin Python binding over it.  There is
no CPU fallback: calls fail loudly when the library is missing or no sm_100
device is present.
"""
from ._lib import (PRISM_ACT_GELU, PRISM_ACT_GELU_TANH, PRISM_ACT_NONE, PRISM_ACT_SILU, PRISM_BF16, PRISM_F32,
                   PRISM_PAIR_ADJACENT, PRISM_PAIR_HALVES, Plan, PrismError, PrismParams, Rope, linear, linear_bwd, load,
                   make_params, make_rope, plan, plan_import, qk_norm_rope, qk_norm_rope_bwd, status_string,
                   workspace_bytes)

__all__ = ["PRISM_ACT_GELU", "PRISM_ACT_GELU_TANH", "PRISM_ACT_NONE", "PRISM_ACT_SILU", "PRISM_BF16", "PRISM_F32",
           "PRISM_PAIR_ADJACENT", "PRISM_PAIR_HALVES", "Plan", "PrismError", "PrismParams", "Rope", "linear",
           "linear_bwd", "load", "make_params", "make_rope", "plan", "plan_import", "qk_norm_rope", "qk_norm_rope_bwd",
           "status_string", "workspace_bytes"]
