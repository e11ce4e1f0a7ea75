"""GB300-native (sm_103a) MXFP8 block-scaled quantize engine.

BF16 [M, N] -> FP8 (E4M3 / E5M2) with one E8M0 scale per 32-element block,
rowwise (1x32) and columnwise (32x1) in one pass, with optional fused dbias
and a device noop flag, plus a grouped (MoE, ragged row offsets) variant; the MXFP4 (4-bit)
cast with its products (``mxfp4``), and expert routing, planning and combination (``moe``).
The compute runs in the CUDA library built from ``csrc/``; this package is its
ctypes binding.
"""
from .binding import (  # noqa: F401
    BLOCK, E4M3, E5M2, MAX_GROUPS, MXFP8Error, MXFP8Tensor, STATUS_NAMES,
    lib, mxfp8_device_fault_word, mxfp8_kernel_launch_count, mxfp8_quantize,
    mxfp8_quantize_grouped, mxfp8_quantize_grouped_workspace_bytes, mxfp8_quantize_host,
    mxfp8_quantize_host_staging_bytes, mxfp8_quantize_dbias_noalloc, quantize_host,
    mxfp8_quantize_workspace_bytes, mxfp8_status_string, quantize, quantize_grouped, grouped_scale_col_rows,
    mxfp8_quantize_grouped_dbias, mxfp8_quantize_grouped_dbias_workspace_bytes,
    mxfp8_quantize_dact, quantize_dact, mxfp8_quantize_gated, quantize_gated, mxfp8_quantize_dgated,
    quantize_dgated, mxfp8_quantize_gated_grouped, quantize_gated_grouped, mxfp8_quantize_grouped_activated,
    mxfp8_quantize_grouped_swizzled, mxfp8_grouped_swizzled_scale_bytes, mxfp8_selftest_bounded_wait, mxfp8_activation_values,
    mxfp8_quantize_grouped_host, mxfp8_quantize_grouped_host_staging_bytes, mxfp8_grouped_host_chunks,
    quantize_grouped_host, mxfp8_quantize_ex_host, mxfp8_quantize_ex_host_staging_bytes,
    mxfp8_quantize_dact_host, mxfp8_quantize_dact_host_staging_bytes, quantize_dact_host,
    mxfp8_quantize_gated_host, mxfp8_quantize_gated_host_staging_bytes, quantize_gated_host,
    mxfp8_quantize_dgated_host, mxfp8_quantize_dgated_host_staging_bytes, quantize_dgated_host,
    QuantizeConfig, SCALES_PLAIN, SCALES_SWIZZLED, make_config, mxfp8_quantize_ex, mxfp8_scale_bytes,
)
from .mxfp4 import (  # noqa: F401
    MXFP4Matrix, MXFP4Tensor, dequantize_mxfp4, matmul_mxfp4, matmul_mxfp4_grouped, mxfp4_dequantize,
    mxfp4_grouped_scale_bytes, mxfp4_matmul, mxfp4_matmul_grouped, mxfp4_quantize, mxfp4_quantize_grouped,
    mxfp4_quantize_grouped_workspace_bytes,    mxfp4_row_bytes, mxfp4_scale_bytes, quantize_mxfp4, quantize_mxfp4_grouped,
    linear_mxfp4, linear_mxfp4_grouped, mxfp4_linear, mxfp4_linear_grouped, mxfp4_linear_grouped_workspace_bytes,
    mxfp4_linear_workspace_bytes,
)
from .moe import (  # noqa: F401
    MoEPlan, MoERoute, RouteConfig, make_route_config, moe_combine, moe_combine_backward, moe_combine_backward_c,
    moe_combine_c, moe_plan, moe_plan_c, moe_plan_workspace_bytes, moe_route, moe_route_backward,
    moe_route_backward_c, moe_route_c,
)
from .mxfp8_matmul import (  # noqa: F401
    matmul_mxfp8_grouped, matmul_mxfp8_grouped_dgrad, matmul_mxfp8_grouped_wgrad, mxfp8_matmul_grouped,
)
from .norm import (  # noqa: F401
    BlockNorm, BlockNormConfig, BlockNormGrads, block_norm, block_norm_backward, block_norm_backward_c,
    block_norm_backward_workspace_bytes, block_norm_c,
)
