"""MI355X-native 3D GroupNorm (NCDHW or channels-last; fp32, bf16 or fp16 in; fp32
statistics) behind a C ABI.

Beside it the root-mean-square norm over rows with the residual's addition (also with an
8-bit output), and the norm of many gradients with clipping.

The kernels live in libgn.so (csrc/); this package is its torch binding.
"""
from .gn import (  # noqa: F401
    GnError,
    GroupNormFn,
    as_layout,
    gn_backward,
    gn_backward_apply,
    gn_backward_finish,
    gn_backward_partials,
    gn_backward_reduce,
    gn_backward_shard_merge,
    gn_backward_shard_sums,
    gn_forward,
    gn_forward_apply,
    gn_forward_finish,
    gn_forward_noalloc,
    gn_forward_partials,
    gn_forward_shard_merge,
    gn_forward_shard_stats,
    gn_forward_stats,
    gn_plan_query,
    gn_plan_query_cl,
    gn_workspace_bytes,
    group_norm,
    layout_of,
    workspace_for,
)
from .ops import (  # noqa: F401
    RmsNormFn,
    clip_gradients,
    gn_grad_clip,
    gn_grad_norm,
    gn_grad_workspace_bytes,
    gn_q8_dequantize,
    gn_rms_backward,
    gn_rms_forward,
    gn_rms_forward_q8,
    gn_rms_workspace_bytes,
    rms_norm,
)
