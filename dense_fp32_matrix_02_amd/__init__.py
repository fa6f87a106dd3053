"""MI355X-native FP32 GEMM: C = A.B on row-major matrices (alpha = 1, beta = 0).

The computation lives in libsgemm_mi355.so (hand-written HIP for gfx950,
C ABI in include/sgemm_mi355.h); this package only loads it and marshals
arguments. Beside it: FP8 products with a scale for each block of 128 and their
quantisers (include/sgemm_mi355_fp8.h), routing to experts
(include/sgemm_mi355_route.h), norms, activations and epilogues around the
products (include/sgemm_mi355_layer.h), and experts' products of 16-bit operands
(include/sgemm_mi355_experts.h). Build it with ``python -m dense_fp32_matrix_02_amd.build``.
"""
from ._binding import (  # noqa: F401
    ERR_ALIAS, ERR_ALIGN, ERR_CONFIG, ERR_DIM, ERR_EXTENT, ERR_LAUNCH, ERR_LD, ERR_NULL, ERR_OP,
    ERR_SCRATCH, ERR_STRIDE, ERR_WORKSPACE, LIB_PATH, SCRATCH_BYTES, OK, OP_N, OP_T, SgemmError, config_id, config_names, gemm,
    gemm_splitk, gemm_streamk, gemm_strided_batched, load, matmul, sgemm_mi355, sgemm_mi355_config_info,
    sgemm_mi355_config_name, sgemm_mi355_config_occupancy, sgemm_mi355_config_ops, sgemm_mi355_ex,
    sgemm_mi355_num_configs,
    sgemm_mi355_select_config, sgemm_mi355_select_config_ex, sgemm_mi355_select_config_valu,
    sgemm_mi355_selected_config, sgemm_mi355_config_staging,
    sgemm_mi355_select_splitk, sgemm_mi355_select_streamk, sgemm_mi355_config_streamk,
    sgemm_mi355_streamk, sgemm_mi355_streamk_with_config, sgemm_mi355_streamk_workspace_size,
    sgemm_mi355_splitk, sgemm_mi355_splitk_noalloc, sgemm_mi355_splitk_with_config, sgemm_mi355_splitk_workspace_size, sgemm_mi355_strerror,
    sgemm_mi355_strided_batched, sgemm_mi355_strided_batched_with_config, sgemm_mi355_tile_map,
    sgemm_mi355_valu, sgemm_mi355_validate, sgemm_mi355_validate_ex, sgemm_mi355_version,
    sgemm_mi355_with_config, strerror)
from ._fp8 import (  # noqa: F401
    BF16, ERR_ROUTE, ERR_TYPE, F16, F32, FP8_DENSE, FP8_EPILOGUE, FP8_EXPERTS, FP8_WGRAD, FP32_SUMS, gemm_fp8,
    gemm_fp8_experts, gemm_fp8_experts_wgrad, quantize_fp8, quantize_fp8_cols, sgemm_mi355_fp8_gemm,
    sgemm_mi355_fp8_gemm_experts, sgemm_mi355_fp8_gemm_experts_wgrad, sgemm_mi355_fp8_kernel_name,
    sgemm_mi355_fp8_quantize_cols, sgemm_mi355_fp8_quantize_rows, sgemm_mi355_fp8_quantize_tiles)
from ._experts import (  # noqa: F401
    EXPERTS_DGRAD, EXPERTS_FORWARD, EXPERTS_WGRAD, gemm_experts, gemm_experts_dgrad, gemm_experts_wgrad,
    sgemm_mi355_experts_gemm, sgemm_mi355_experts_gemm_dgrad, sgemm_mi355_experts_gemm_wgrad,
    sgemm_mi355_experts_kernel_name)
from ._layer import (  # noqa: F401
    GELU, GELU_TANH, MAX_NORM_COLS, NONE, RELU, SILU, epilogue_backward, gated, gated_backward, gated_fp8,
    gemm_fp8_epilogue, rms_norm, rms_norm_backward, rms_norm_fp8, sgemm_mi355_epilogue_backward,
    sgemm_mi355_epilogue_backward_workspace_size, sgemm_mi355_fp8_gemm_epilogue, sgemm_mi355_gated,
    sgemm_mi355_gated_backward, sgemm_mi355_rms_norm, sgemm_mi355_rms_norm_backward,
    sgemm_mi355_rms_norm_backward_workspace_size)
from ._route import (  # noqa: F401
    MAX_CHOICES, MAX_EXPERTS, SIGMOID, SOFTMAX, route, route_backward, route_combine, route_combine_backward,
    route_plan, sgemm_mi355_route, sgemm_mi355_route_backward, sgemm_mi355_route_combine,
    sgemm_mi355_route_combine_backward, sgemm_mi355_route_plan, sgemm_mi355_route_plan_workspace_size)

__all__ = [n for n in dir() if not n.startswith("_")]
