"""GB300-native MoE expert-parallel route / layout / dispatch / combine.

The compute path is libep_gb300.so (hand-written CUDA for sm_103a, C ABI in
include/ep.h); ``ep`` is its thin Python binding and ``workloads`` the seeded
synthetic inputs.
"""
from .ep import (EP_ACT_NONE, EP_ACT_SWIGLU, EP_DTYPE_BF16, EP_DTYPE_F32, EP_DTYPE_FP8_E4M3_B128,
                 EP_LAYOUT_CONTIG, EP_LAYOUT_MASKED, EP_SCORE_SIGMOID, EP_SCORE_SOFTMAX,
                 EPError, Layout, Norm, alloc_layout, alloc_norm, ep_combine,
                 ep_dequantize_blocks, ep_dispatch, ep_dispatch_layout,
                 ep_dispatch_layout_workspace_size, ep_expert_balance_map, ep_expert_matmul,
                 ep_expert_matmul_fp8, ep_gate_topk, ep_gate_topk_backward,
                 ep_kernel_launch_count, ep_quantize_blocks, ep_quantize_rows, ep_rms_norm,
                 ep_rms_norm_backward, ep_rms_norm_backward_workspace_size,
                 ep_route_dispatch, ep_route_dispatch_workspace_size,
                 ep_route_layout, ep_route_layout_workspace_size, ep_route_topk,
                 ep_selftest_wait_timeout, ep_swiglu_backward, scale_blocks)

__all__ = [
    "EP_ACT_NONE", "EP_ACT_SWIGLU", "EP_DTYPE_BF16", "EP_DTYPE_F32", "EP_DTYPE_FP8_E4M3_B128",
    "EP_LAYOUT_CONTIG", "EP_LAYOUT_MASKED", "EP_SCORE_SIGMOID", "EP_SCORE_SOFTMAX", "EPError",
    "Layout", "Norm", "alloc_layout", "alloc_norm", "ep_combine", "ep_dequantize_blocks",
    "ep_dispatch", "ep_dispatch_layout", "ep_dispatch_layout_workspace_size",
    "ep_expert_balance_map", "ep_expert_matmul", "ep_expert_matmul_fp8", "ep_gate_topk",
    "ep_gate_topk_backward", "ep_kernel_launch_count", "ep_quantize_blocks", "ep_quantize_rows",
    "ep_rms_norm", "ep_rms_norm_backward", "ep_rms_norm_backward_workspace_size",
    "ep_route_dispatch", "ep_route_dispatch_workspace_size", "ep_route_layout",
    "ep_route_layout_workspace_size", "ep_route_topk", "ep_selftest_wait_timeout",
    "ep_swiglu_backward", "scale_blocks",
]
