"""Register-tiled dense product C = A.B for one GB300 (sm_103a).

Two CUDA paths behind a C ABI (include/gemm.h, libgemm_gb300.so):

  gemm_f32      fp32 SIMT kernel: global C tiles, cp.async-staged shared K
                slices, an 8 x 8 fp32 register micro-tile per thread.
  gemm_bf16f32  tcgen05 kernel: TMA-staged bf16 K slices, fp32 accumulators
                in tensor memory, persistent warp-specialised CTAs.

  gemm_bf16w4f32, gemm_q8tbf16f32
                products with an operand held in fewer bits: 4-bit weights
                with group scales, activations saved in 8 bits.

  gemm_f8w8f32, gemm_f8w8tf32, gemm_f8tf8f32
                products of 8-bit floating-point operands with a scale for each
                block of 128, forward and backward.
  gemm_route, gemm_f8w8f32_experts, gemm_experts_join
                a layer of experts on them: routing, the experts' products and
                their sum, each with its backward pass.

This package is the thin Python binding (torch is used only for device
memory and streams) plus the in-tree build step.
"""

from .native_build import build, ptxas_report  # noqa: F401
from .binding import (  # noqa: F401
    LADDER,
    STATUS,
    GemmError,
    gemm_bf16f32,
    gemm_bf16f32_workspace_bytes,
    gemm_bf16f32_ws,
    gemm_bf16w4f32,
    gemm_bf16w4f32_selftest_timeout,
    gemm_f16f32,
    gemm_f16f32_ws,
    gemm_f16w4f32,
    gemm_bf16f32_selftest_timeout,
    gemm_f32,
    gemm_f32_ladder,
    gemm_f32_selftest_timeout,
    gemm_f32_schedule,
    gemm_f32_workspace_bytes,
    gemm_q8_dequantize,
    gemm_q8_quantize,
    gemm_q8t_workspace_bytes,
    gemm_q8tbf16f32,
    gemm_q8tbf16f32_selftest_timeout,
    gemm_q8tf16f32,
    gemm_w4_dequantize,
    gemm_w4_pack,
    gemm_w4_quantize,
    gemm_w4_workspace_bytes,
    F32_KINDS,
    Q8_ROWS,
    W4_BLOCK,
    W4_GROUPS,
    fp32_pipe_peak,
    gemm_f32_ws,
    get_device_error,
    header_symbols,
    library_path,
    load_library,
    status_string,
)
from .f8 import (  # noqa: F401
    F8_BLOCK,
    F8_KINDS,
    gemm_experts_join,
    gemm_experts_join_backward,
    gemm_f8_dequantize,
    gemm_f8_quantize,
    gemm_f8_quantize_tiles,
    gemm_f8tf8f32,
    gemm_f8tf8f32_experts,
    gemm_f8w8f32,
    gemm_f8w8f32_experts,
    gemm_f8w8f32_selftest_timeout,
    gemm_f8w8tf32,
    gemm_f8w8tf32_experts,
    gemm_route,
    gemm_route_backward,
    gemm_route_rows,
)
