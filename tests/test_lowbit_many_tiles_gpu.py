"""Low-bit products with more tiles than the GPU has SMs, so that every block of threads
computes several, and the 32-column kernels for few rows and wide weights. Operands
are small integers with scales of powers of two: every sum is exact, and outputs
have to be equal."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rtm.build()
    rtm.load_library()


def integers(gen, rows, cols, high, dtype):
    return torch.randint(-high, high + 1, (rows, cols), generator=gen, device=DEV).to(dtype)


def powers(gen, rows, cols, dtype):
    """1/4, 1/2, 1 or 2."""
    return torch.ldexp(torch.ones((), device=DEV),
                       torch.randint(-2, 2, (rows, cols), generator=gen, device=DEV)).to(dtype)


def check_w4(M, N, K, group, zeros, dtype, calls=3):
    # |sum| <= K * 2 * 15 * 2 < 2^22 quarters for K <= 1000
    gen = torch.Generator(DEV).manual_seed(M + 3 * N + 5 * K + group)
    G = -(-K // group)
    q = torch.randint(0, 16, (K, N), generator=gen, device=DEV, dtype=torch.uint8)
    s = powers(gen, G, N, dtype)
    z = torch.randint(0, 16, (G, N), generator=gen, device=DEV, dtype=torch.uint8) if zeros else None
    A = integers(gen, M, K, 2, dtype)
    g = torch.arange(K, device=DEV) // group
    zero = 8.0 if z is None else z.double()[g]
    want = A.double() @ ((q.double() - zero) * s.double()[g])
    codes = rtm.gemm_w4_pack(q)
    product = rtm.gemm_bf16w4f32 if dtype == torch.bfloat16 else rtm.gemm_f16w4f32
    for _ in range(calls):
        guard = torch.full((M * N + 64,), 7.0, device=DEV)
        C = product(A, codes, s, z, group, out=guard[:M * N].view(M, N))
        assert torch.equal(C.double(), want) and (guard[M * N:] == 7.0).all()
    assert rtm.get_device_error() == 0


# One stage of depth; an odd number of stages; of 128-deep blocks; both even.
DEPTHS = [60, 72, 136, 184, 200, 330, 512]


@pytest.mark.parametrize("K", DEPTHS)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N", [(20, 40001), (48, 40000), (100, 40001), (300, 40001), (2100, 4201)])
def test_w4(M, N, K, group):
    for dtype in TYPES:
        for zeros in (True, False):
            check_w4(M, N, K, group, zeros, dtype)


@pytest.mark.parametrize("M", [60, 100, 130, 200, 330, 512])
@pytest.mark.parametrize("N", [40, 64, 100, 300])
@pytest.mark.parametrize("dtype", TYPES)
def test_q8t(M, N, dtype):
    # |sum| <= 512 * 127 * 2 * 2 < 2^20 quarters
    K = 40001
    gen = torch.Generator(DEV).manual_seed(M + 3 * N)
    codes = integers(gen, M, -(-K // 16) * 16, 127, torch.int8)
    s = powers(gen, -(-M // 128), K, torch.float32)
    dY = integers(gen, M, N, 2, dtype)
    x = codes[:, :K].double() * s.double()[torch.arange(M, device=DEV) // 128]
    want = x.t() @ dY.double()
    gradient = rtm.gemm_q8tbf16f32 if dtype == torch.bfloat16 else rtm.gemm_q8tf16f32
    for _ in range(3):
        guard = torch.full((K * N + 64,), 7.0, device=DEV)
        dW = gradient(codes, s, dY, out=guard[:K * N].view(K, N))
        assert torch.equal(dW.double(), want) and (guard[K * N:] == 7.0).all()
    assert rtm.get_device_error() == 0


# 32-column strips are taken for groups of 128 and M <= 4 where they give every SM two
# blocks: N beyond 64 columns for each of 152 SMs.
@pytest.mark.parametrize("K", [1, 264, 266, 333, 4608])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("N", [10001, 12800])
def test_w4_wide_strips(M, N, K):
    # K = 4608: |sum| <= 4608 * 2 * 15 * 2 < 2^21 quarters
    for dtype in TYPES:
        for zeros in (True, False):
            check_w4(M, N, K, 128, zeros, dtype)
