"""Arguments of the low-bit entry points that are no tensors are refused like tensors of the
wrong kind, with ValueError."""

import numpy as np
import pytest
import torch

import register_tiled_matrix_gb300 as rtm

NO_TENSORS = [None, 3, [[1.0]], np.ones((1, 64), dtype=np.float32)]


@pytest.mark.cpu
@pytest.mark.parametrize("bad", NO_TENSORS, ids=lambda v: type(v).__name__)
def test_conversions(bad):
    codes, codes8 = torch.zeros(64, 64, dtype=torch.uint8), torch.zeros(64, 64, dtype=torch.int8)
    scales, scales8 = torch.ones(1, 64, dtype=torch.bfloat16), torch.ones(1, 64)
    for call in (lambda: rtm.gemm_w4_quantize(bad), lambda: rtm.gemm_w4_pack(bad),
                 lambda: rtm.gemm_w4_dequantize(codes, bad, None, 128),
                 lambda: rtm.gemm_w4_dequantize(bad, scales, None, 128),
                 lambda: rtm.gemm_q8_quantize(bad),
                 lambda: rtm.gemm_q8_dequantize(codes8, bad, 64, 64),
                 lambda: rtm.gemm_q8_dequantize(bad, scales8, 64, 64)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", NO_TENSORS, ids=lambda v: type(v).__name__)
def test_on_the_gpu(bad):
    rtm.build()
    W = torch.zeros(128, 64, dtype=torch.bfloat16, device="cuda:0")
    x = torch.zeros(20, 128, dtype=torch.bfloat16, device="cuda:0")
    codes, s, z = rtm.gemm_w4_quantize(W)
    codes8, s8 = rtm.gemm_q8_quantize(x)
    dy = x[:, :64].contiguous()
    calls = [lambda: rtm.gemm_w4_dequantize(codes, bad, z, 128),
             lambda: rtm.gemm_w4_dequantize(bad, s, z, 128),
             lambda: rtm.gemm_bf16w4f32(bad, codes, s, z),
             lambda: rtm.gemm_bf16w4f32(x, bad, s, z),
             lambda: rtm.gemm_bf16w4f32(x, codes, bad, z),
             lambda: rtm.gemm_q8_dequantize(codes8, bad, 20, 128),
             lambda: rtm.gemm_q8_dequantize(bad, s8, 20, 128),
             lambda: rtm.gemm_q8tbf16f32(bad, s8, dy), lambda: rtm.gemm_q8tbf16f32(codes8, bad, dy),
             lambda: rtm.gemm_q8tbf16f32(codes8, s8, bad)]
    if bad is not None:  # None is a choice here
        calls += [lambda: rtm.gemm_w4_dequantize(codes, s, bad, 128),
                  lambda: rtm.gemm_bf16w4f32(x, codes, s, bad),
                  lambda: rtm.gemm_bf16w4f32(x, codes, s, z, out=bad),
                  lambda: rtm.gemm_bf16w4f32(x, codes, s, z, workspace=bad),
                  lambda: rtm.gemm_q8tbf16f32(codes8, s8, dy, workspace=bad),
                  lambda: rtm.gemm_w4_dequantize(codes, s, z, 128, out=bad)]
    for call in calls:
        with pytest.raises(ValueError):
            call()
