"""CPU tests of the low-bit entry points: argument errors are reported before any
CUDA call, and the host reference packs and quantises as the layout says."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import lowbit_reference as ref

pytestmark = pytest.mark.cpu
A, B, C, D, E, W = (0x10000000 * i for i in range(1, 7))


@pytest.fixture(scope="module")
def lib():
    rtm.build()
    return rtm.load_library()


def test_code_sizes(lib):
    assert lib.gemm_w4_codes_bytes(128, 10) == 640
    assert lib.gemm_w4_codes_bytes(129, 10) == 1280
    assert lib.gemm_w4_codes_bytes(0, 10) == 0
    assert lib.gemm_w4_codes_bytes(-1, 10) == -1
    assert lib.gemm_w4_codes_bytes(1 << 30, 1 << 20) == -1  # over 2^40 weights
    assert lib.gemm_q8_codes_bytes(5, 17) == 160
    assert lib.gemm_q8_codes_bytes(5, 1 << 31) == -1


@pytest.mark.parametrize("fn", ["gemm_bf16w4f32", "gemm_f16w4f32"])
def test_w4_product_arguments(lib, fn):
    f = getattr(lib, fn)
    assert f(-1, 8, 8, A, B, C, D, 128, E, 0, 0, None) == -1
    assert f(8, 8, 1 << 31, A, B, C, D, 128, E, 0, 0, None) == -1
    assert f(8, 8, (1 << 31) - 255, A, B, C, D, 128, E, 0, 0, None) == -1
    for group in (0, 16, 96, 256):
        assert f(8, 8, 256, A, B, C, D, group, E, 0, 0, None) == -1
    assert f(0, 8, 8, 0, 0, 0, 0, 128, 0, 0, 0, None) == 0
    assert f(8, 0, 8, 0, 0, 0, 0, 128, 0, 0, 0, None) == 0
    assert f(8, 8, 8, A, B, C, D, 128, 0, 0, 0, None) == -1      # no C
    assert f(8, 8, 8, 0, B, C, D, 128, E, 0, 0, None) == -1      # no A
    assert f(8, 8, 8, A, 0, C, D, 128, E, 0, 0, None) == -1      # no codes
    assert f(8, 8, 8, A, B, 0, D, 128, E, 0, 0, None) == -1      # no scales
    assert f(8, 8, 8, A, B, C, D, 128, E, 0, 64, None) == -1     # a size without a workspace
    assert f(8, 8, 8, A, B, C, D, 128, E, W, -1, None) == -1
    assert f(64, 64, 256, A, B, C, D, 128, A + 16, 0, 0, None) == -1  # C over A
    assert f(64, 64, 256, A, B, C, D, 128, B + 64, 0, 0, None) == -1  # C over codes
    assert f(64, 64, 256, A, B, C, D, 128, C, 0, 0, None) == -1       # C over scales
    assert f(64, 64, 256, A, B, C, D, 128, D, 0, 0, None) == -1       # C over zero points
    assert f(8, 8, 8, A + 1, B, C, D, 128, E, 0, 0, None) == -2
    assert f(8, 8, 8, A, B + 8, C, D, 128, E, 0, 0, None) == -2
    assert f(8, 8, 8, A, B, C + 1, D, 128, E, 0, 0, None) == -2
    assert f(8, 8, 8, A, B, C, D, 128, E + 2, 0, 0, None) == -2


@pytest.mark.parametrize("fn", ["gemm_q8tbf16f32", "gemm_q8tf16f32"])
def test_q8t_arguments(lib, fn):
    f = getattr(lib, fn)
    assert f(8, -1, 8, A, B, C, E, 0, 0, None) == -1
    assert f(8, 0, 8, 0, 0, 0, 0, 0, 0, None) == 0
    assert f(8, 8, 0, 0, 0, 0, 0, 0, 0, None) == 0
    for null in range(4):
        p = [A, B, C, E]
        p[null] = 0
        assert f(8, 8, 8, *p, 0, 0, None) == -1
    assert f(64, 64, 64, A, B, C, A + 32, 0, 0, None) == -1
    assert f(64, 64, 64, A, B, C, B, 0, 0, None) == -1
    assert f(64, 64, 64, A, B, C, C + 64, 0, 0, None) == -1
    assert f(8, 8, 8, A + 8, B, C, E, 0, 0, None) == -2
    assert f(8, 8, 8, A, B + 2, C, E, 0, 0, None) == -2
    assert f(8, 8, 8, A, B, C + 1, E, 0, 0, None) == -2
    assert f(8, 8, 8, A, B, C, E + 1, 0, 0, None) == -2


def test_conversion_arguments(lib):
    q = lib.gemm_bf16_w4_quantize
    assert q(-1, 8, 128, A, B, C, D, None) == -1 and q(8, 8, 100, A, B, C, D, None) == -1
    assert q(0, 8, 128, 0, 0, 0, 0, None) == 0 and q(8, 8, 128, 0, B, C, D, None) == -1
    assert q(8, 8, 128, A, A + 16, C, D, None) == -1    # codes over W
    assert q(256, 8, 128, A, B, B + 64, D, None) == -1  # scales over codes
    assert q(8, 8, 128, A, B + 4, C, D, None) == -2 and q(8, 8, 128, A + 1, B, C, D, None) == -2
    d = lib.gemm_f16_w4_dequantize
    assert d(8, 8, 0, A, B, C, D, None) == -1 and d(8, 8, 128, A, B, C, A + 16, None) == -1
    assert d(8, 8, 128, A + 2, B, C, D, None) == -2
    p = lib.gemm_w4_pack
    assert p(8, 8, 0, B, None) == -1 and p(8, 8, A, A, None) == -1 and p(8, 8, A, B + 1, None) == -2
    s = lib.gemm_bf16_q8_quantize
    assert s(8, -1, A, B, C, None) == -1 and s(8, 8, A, B, B, None) == -1
    assert s(8, 8, A, B + 8, C, None) == -2 and s(0, 8, 0, 0, 0, None) == 0
    r = lib.gemm_f16_q8_dequantize
    assert r(8, 8, A, B, A, None) == -1 and r(8, 8, A, B + 2, C, None) == -2


def test_cpu_tensors_are_refused():
    x = torch.zeros(8, 128, dtype=torch.bfloat16)
    codes, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.bfloat16)
    for call in (lambda: rtm.gemm_bf16w4f32(x, codes, s), lambda: rtm.gemm_w4_quantize(x),
                 lambda: rtm.gemm_q8_quantize(x), lambda: rtm.gemm_w4_pack(codes)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("K", [1, 100, 128, 300])
def test_reference_packs_and_unpacks(K):
    q = torch.randint(0, 16, (K, 5), dtype=torch.uint8)
    codes = ref.w4_pack(q)
    assert codes.shape == (5, (K + 127) // 128 * 64)
    assert torch.equal(ref.w4_unpack(codes, K), q)


def test_selftest_arguments(lib):
    f = lib.gemm_bf16w4f32_selftest_timeout
    assert f(64, 64, 256, A, B, C, D, 128, E, 10, None) == -1            # limit too short
    assert f(16, 64, 256, A, B, C, D, 128, E, 10 ** 8, None) == -1       # another kernel
    assert f(64, 64, 250, A, B, C, D, 128, E, 10 ** 8, None) == -1       # rows off 16 bytes
    g = lib.gemm_q8tbf16f32_selftest_timeout
    assert g(64, 64, 64, A, B, C, E, 10 ** 11, None) == -1
    assert g(64, 60, 64, A, B, C, E, 10 ** 8, None) == -1
