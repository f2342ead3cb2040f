"""GB300-native output-stationary tiled matrix multiply, C = A @ B.

Beside it, products of 8-bit matrices with a scale for each block of 128, their
quantisation, orthogonalisation by Newton-Schulz products, products whose rows
are grouped by expert, and low-rank adapters beside a shared projection.

The products run in the CUDA library `_build/libtiled_gemm.so` (hand-written
sm_103a kernels behind the C ABI of include/tiled_gemm.h); this package is
its ctypes binding plus the seeded input generator.  The library is loaded
on first use and there is no CPU fallback.
"""
from .binding import (  # noqa: F401
    BF16, E4M3, E5M2, F16, F32, Fp8Matrix, KERNEL_NAMES, KERNELS, GemmError, addmm, error_string,
    gemm, gemm_debug_config, gemm_device_status, gemm_error_string, gemm_ex, gemm_ex_host, gemm_ex_host_ws, gemm_ex_kernel,
    gemm_ex_ws, gemm_host_panel_rows,
    gemm_general, gemm_launch_count, gemm_traffic_model, gemm_workspace_size, matmul_ws,
    gemm_select_kernel, gemm_splitk, gemm_splitk_noalloc, gemm_splitk_workspace_size,
    gemm_ws_split_count,
    header_functions, library_path,
    load_library, matmul, matmul_splitk,
    gemm_fp8, gemm_fp8_quantize, gemm_fp8_quantize_pair, matmul_fp8, quantize_fp8,
    quantize_fp8_pair,
    NEWTON_SCHULZ_COEFFICIENTS, gemm_newton_schulz, gemm_newton_schulz_workspace_size,
    newton_schulz,
    gemm_grouped, gemm_grouped_wgrad, gemm_grouped_wgrad_workspace_size,
    gemm_grouped_workspace_size, matmul_grouped, matmul_grouped_wgrad,
    LoraAdapters, gemm_lora, gemm_lora_backward, gemm_lora_backward_workspace_size,
    gemm_lora_workspace_size, matmul_lora, matmul_lora_backward,
)
