"""Local MoE expert forward on the non-expand routed layout, for NVIDIA B200 (sm_100a).

The computation lives in ``libmoe_nonexpand.so`` (C ABI: include/moe_nonexpand.h);
``binding`` passes torch tensors' device pointers and the current stream to it.
"""
from .binding import (  # noqa: F401
    ACT_SWIGLU, LAYOUT_CONCATENATED, LAYOUT_INTERLEAVED, MoeError, add_rmsnorm,
    add_rmsnorm_backward, alloc_meta, alloc_workspace, combine, forward, forward_fp8,
    grouped_linear_fp8, intermediates_from_workspace, linear_fp8, meta_from_workspace,
    metadata, quantize_rows_fp8, quantize_weight_fp8, read_error, workspace_bytes,
    workspace_layout,
)
