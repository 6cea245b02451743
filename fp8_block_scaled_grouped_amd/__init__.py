"""libmoe355: FP8 block-scale Mixture-of-Experts layer for MI355X (gfx950).

The compute lives in libmoe355.so (HIP kernels behind the C ABI declared in
include/moe355.h); `moe355` is its ctypes binding and `inputs` the seeded
synthetic workload generator.
"""
from . import inputs  # noqa: F401
from .moe355 import (  # noqa: F401
    MoELayer,
    Moe355Error,
    fp4_dequant_groups,
    fp4_quant_groups,
    fp8_quant_128x128,
    fp8_quant_1x128,
    fp8_quant_ragged,
    fp8_ragged_blocks,
    gemm_fp4_groupscale,
    gemm_fp4_groupscale_workspace,
    gemm_fp8_blockscale,
    gemm_fp8_blockscale_plan,
    gemm_fp8_blockscale_tiled,
    gemm_fp8_blockscale_tiled_workspace,
    gemm_fp8_blockscale_workspace,
    grouped_gemm,
    grouped_gemm_dgrad,
    grouped_gemm_fp4,
    grouped_gemm_fp8,
    grouped_gemm_fp8_wgrad,
    grouped_gemm_wgrad,
    grouped_linear,
    grouped_linear_fp8,
    grouped_topk,
    lib,
    moe_block_m,
    moe_combine,
    moe_combine_grad,
    moe_dispatch,
    moe_down_combine,
    moe_down_combine_workspace,
    moe_fp8_blockscale_fused,
    moe_fp8_blockscale_fused_workspace,
    moe_fp8_blockscale_g1u1,
    moe_group,
    moe_group_workspace,
    moe_sort,
    moe_sort_sizes,
    shuffle_weight_128x128,
)
