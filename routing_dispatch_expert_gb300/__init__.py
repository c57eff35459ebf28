"""GB300-native hot path of an expert-parallel MoE layer: route -> dispatch -> SwiGLU grouped GEMM
-> combine, as hand-written sm_103a CUDA kernels behind a C ABI (include/moe.h)."""
from .moe import (Fp4Activations, Graph, GraphedMoeLayer, MoeConfig, MoeError, MoeLayer, Placement, Weights,
                  alloc_workspace, balance, balance_loss, balance_loss_backward, balance_loss_workspace, combine,
                  dequantize_fp4, device_status, dispatch, dispatch_fp4, dispatch_noalloc, eplb_plan, expert_ffn,
                  expert_ffn_fp4, forward, forward_fp4, launch_count, load, make_config, matmul_fp4, matmul_fp4_status,
                  quantize_fp4, quantize_weights_fp8, quantize_weights_nvfp4, route, selftest_wait_timeout,
                  workspace_layout, workspace_size, ws_view)

__all__ = ["Fp4Activations", "Graph", "GraphedMoeLayer", "MoeConfig", "MoeError", "MoeLayer", "Placement", "Weights",
           "alloc_workspace", "balance", "balance_loss", "balance_loss_backward", "balance_loss_workspace", "combine",
           "dequantize_fp4", "device_status", "dispatch", "dispatch_fp4", "dispatch_noalloc", "eplb_plan", "expert_ffn",
           "expert_ffn_fp4", "forward", "forward_fp4", "launch_count", "load", "make_config", "matmul_fp4",
           "matmul_fp4_status", "quantize_fp4", "quantize_weights_fp8", "quantize_weights_nvfp4", "route",
           "selftest_wait_timeout", "workspace_layout", "workspace_size", "ws_view"]
