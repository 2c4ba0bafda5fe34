"""A wait that gives up in a large low-bit product: the call comes back soon after the
limit, however much of the product was still to do, and the next one is right."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LIMIT_MS = 20
# A wait under way ends at the limit, or within 64 polls of another role that gave up;
# one begun later looks at the flag at once. The CTAs of a pair keep their own flags: two
# limits. A poll lasts a millisecond at the very most; the rest is instructions.
BOUND_MS = 250


def timed(call):
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    call()
    end.record()
    assert rtm.STATUS[rtm.get_device_error()] == "GEMM_ERR_TIMEOUT"
    return begin.elapsed_time(end)


# Many tiles a CTA, many groups a tile: pairs, and single CTAs of 32, 64 and 128 columns.
@pytest.mark.parametrize("M,N,K", [(8192, 8192, 8192), (24, 60000, 8192), (48, 60000, 8192),
                                   (100, 60000, 8192)])
def test_w4_returns_soon(M, N, K):
    rtm.build()
    gen = torch.Generator(DEV).manual_seed(M)
    W = torch.randn(K, N, generator=gen, device=DEV).to(torch.bfloat16)
    A = torch.randn(M, K, generator=gen, device=DEV).to(torch.bfloat16)
    codes, s, z = rtm.gemm_w4_quantize(W, 32)
    want = rtm.gemm_bf16w4f32(A, codes, s, z, 32)
    out = torch.empty_like(want)
    ms = timed(lambda: rtm.gemm_bf16w4f32_selftest_timeout(A, codes, s, z, 32, out,
                                                           LIMIT_MS * 1_000_000))
    print(f"back after {ms:.1f} ms")
    assert ms < BOUND_MS
    assert torch.equal(rtm.gemm_bf16w4f32(A, codes, s, z, 32), want)
    assert rtm.get_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(8192, 8192, 8192), (8192, 64, 60000), (8192, 128, 60000)])
def test_q8_returns_soon(M, N, K):
    rtm.build()
    gen = torch.Generator(DEV).manual_seed(N)
    codes, s = rtm.gemm_q8_quantize(torch.randn(M, K, generator=gen, device=DEV).to(torch.bfloat16))
    dY = torch.randn(M, N, generator=gen, device=DEV).to(torch.bfloat16)
    want = rtm.gemm_q8tbf16f32(codes, s, dY)
    out = torch.empty_like(want)
    ms = timed(lambda: rtm.gemm_q8tbf16f32_selftest_timeout(codes, s, dY, out,
                                                            LIMIT_MS * 1_000_000))
    print(f"back after {ms:.1f} ms")
    assert ms < BOUND_MS
    assert torch.equal(rtm.gemm_q8tbf16f32(codes, s, dY), want)
    assert rtm.get_device_error() == 0
