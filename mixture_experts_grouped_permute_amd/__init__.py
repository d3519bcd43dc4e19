"""MI355X-native grouped expert MLP (permute -> grouped GEMM -> ScaledSwiGLU*prob
-> grouped GEMM -> combine) in BF16 and MXFP8 (forward and backward) and in
per-tensor-scaled FP8 (forward), behind the C ABI of libmoe.so.

The functions below are thin ctypes wrappers; all computation happens in the
library's HIP kernels for gfx950.
"""
from ._lib import (MOE_BF16, MOE_F32, MOE_FP8_BLOCK, MOE_FP8_E4M3, MOE_MXFP8_E4M3, EXPORTS, MoeError, load, fp8_tensor_quantize,
                   moe_grouped_mlp_bwd, moe_grouped_mlp_fwd, moe_grouped_mlp_fwd_loop, moe_permute,
                   moe_permute_noalloc, moe_read_device_error, moe_route_permute, moe_route_topk, mxfp8_quantize,
                   mxfp8_quantize_weights, quantize_weights, set_tile_stats, tile_stats_new, tile_stats_summary, mfma_probe,
                   load_probe, moe_route_balance, moe_route_balance_bwd, fp8_block_quantize,
                   fp8_block_quantize_weights, fp8_block_grouped_gemm, fp8_block_grouped_wgrad,
                   moe_route_grouped, moe_route_grouped_bwd, moe_add_rmsnorm, moe_add_rmsnorm_bwd, GradTable,
                   moe_grad_sumsq, moe_grad_clip, LIB_PATH)

__all__ = [
    "MOE_BF16", "MOE_F32", "MOE_FP8_BLOCK", "MOE_FP8_E4M3", "MOE_MXFP8_E4M3", "EXPORTS", "MoeError", "load",
    "fp8_tensor_quantize", "moe_grouped_mlp_bwd", "moe_grouped_mlp_fwd", "moe_grouped_mlp_fwd_loop", "moe_permute",
    "moe_permute_noalloc", "moe_read_device_error", "moe_route_permute", "moe_route_topk", "mxfp8_quantize",
    "mxfp8_quantize_weights", "quantize_weights", "set_tile_stats", "tile_stats_new", "tile_stats_summary", "mfma_probe", "load_probe",
    "moe_route_balance", "moe_route_balance_bwd", "fp8_block_quantize", "fp8_block_quantize_weights",
    "fp8_block_grouped_gemm", "fp8_block_grouped_wgrad", "moe_route_grouped", "moe_route_grouped_bwd",
    "moe_add_rmsnorm", "moe_add_rmsnorm_bwd", "GradTable", "moe_grad_sumsq", "moe_grad_clip",
    "LIB_PATH",
]
