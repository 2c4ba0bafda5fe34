"""Low-bit operands whose offsets or sizes pass 32 bits: matrices of more than 2^31
elements, and one dimension at its limit of 2^31 - 256. Operands are small integers with
scales of powers of two, so outputs have to be equal; the longest sums have a few
terms that are not zero, at seeded places and at both ends."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LONGEST = 2 ** 31 - 256


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rtm.build()
    rtm.load_library()


@pytest.fixture(autouse=True)
def _room():
    yield
    torch.cuda.empty_cache()


def places(n, count, gen):
    """Seeded indices below n, both ends among them."""
    i = torch.randint(0, n, (count,), generator=gen, device=DEV)
    i[:2] = torch.tensor([0, n - 1], device=DEV)
    return torch.unique(i)


def integers(gen, rows, cols, high, dtype):
    return torch.randint(-high, high + 1, (rows, cols), generator=gen, device=DEV,
                         dtype=torch.int8).to(dtype)


# Pairs; 128, 64 and 32 columns on one CTA; few rows.
@pytest.mark.parametrize("M,N", [(46341, 46344), (100, 21474840), (60, 35791400), (20, 107374192),
                                 (16, 134217736)])
def test_w4_output(M, N):
    K = 24
    assert M * N > 2 ** 31
    gen = torch.Generator(DEV).manual_seed(M)
    q = torch.randint(0, 16, (K, N), generator=gen, device=DEV, dtype=torch.uint8)
    s = torch.full((1, N), 0.5, dtype=torch.bfloat16, device=DEV)
    s[:, ::3] = 2.0
    z = torch.randint(0, 16, (1, N), generator=gen, device=DEV, dtype=torch.uint8)
    A = integers(gen, M, K, 2, torch.bfloat16)
    C = rtm.gemm_bf16w4f32(A, rtm.gemm_w4_pack(q), s, z)
    rows, cols = places(M, 300, gen), places(N, 3000, gen)
    w = (q[:, cols].double() - z[:, cols].double()) * s[:, cols].double()
    assert torch.equal(C[rows][:, cols].double(), A[rows].double() @ w)
    assert torch.equal(C[-1].double(), (A[-1:].double() @ ((q.double() - z.double()) * s.double()))[0])
    assert rtm.get_device_error() == 0


@pytest.mark.parametrize("M", [1, 17])
def test_w4_longest_sum(M):
    K, N = LONGEST, 2
    gen = torch.Generator(DEV).manual_seed(M)
    codes = torch.randint(0, 256, (N, K // 128 * 64), generator=gen, device=DEV, dtype=torch.uint8)
    s = torch.full((K // 128, N), 0.5, dtype=torch.bfloat16, device=DEV)
    s[::3] = 2.0
    k = places(K, 4000, gen)
    A = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    A[:, k] = integers(gen, M, len(k), 2, torch.bfloat16)
    r = k % 128
    bit = 4 * (r % 8 // 2) + 16 * (r % 2)
    byte = k // 128 * 64 + r % 32 // 8 * 16 + r // 32 * 4 + bit // 8
    q = (codes[:, byte].int() >> (bit % 8)) & 15  # N x places
    w = (q.double() - 8).t() * s[k // 128].double()
    C = rtm.gemm_bf16w4f32(A, codes, s)
    assert torch.equal(C.double(), A[:, k].double() @ w)
    assert rtm.get_device_error() == 0


@pytest.mark.parametrize("K,N", [(46352, 46344), (46339, 46351), (16, 134217800)])
def test_w4_conversions(K, N):
    assert K * N > 2 ** 31
    gen = torch.Generator(DEV).manual_seed(K)
    W = torch.empty(K, N, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    codes, s, z = rtm.gemm_w4_quantize(W, 64)
    back = rtm.gemm_w4_dequantize(codes, s, z, K, 64)
    # Any one column is what the same column gives by itself.
    cols = places(N, 200, gen)
    c1, s1, z1 = rtm.gemm_w4_quantize(W[:, cols].contiguous(), 64)
    assert torch.equal(codes[cols], c1) and torch.equal(s[:, cols], s1)
    assert torch.equal(z[:, cols], z1)
    assert torch.equal(back[:, cols], rtm.gemm_w4_dequantize(c1, s1, z1, K, 64))


@pytest.mark.parametrize("M,K", [(46341, 46352), (46341, 46351), (LONGEST, 1), (7, 306783400)])
def test_q8_conversions(M, K):
    gen = torch.Generator(DEV).manual_seed(K % 1000)
    X = torch.empty(M, K, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    codes, s = rtm.gemm_q8_quantize(X)
    back = rtm.gemm_q8_dequantize(codes, s, M, K)
    cols = places(K, 200, gen)
    m0 = (M - 1) // 128 * 128  # the last block of rows, and the first
    for rows in (slice(0, 128), slice(m0, M)):
        part = X[rows][:, cols].contiguous()
        c1, s1 = rtm.gemm_q8_quantize(part)
        assert torch.equal(codes[rows][:, cols], c1[:, :len(cols)])
        assert torch.equal(s[rows.start // 128, cols], s1[0])
        assert torch.equal(back[rows][:, cols], rtm.gemm_q8_dequantize(c1, s1, *part.shape))


@pytest.mark.parametrize("K,N", [(46352, 46344), (53687100, 40), (21474900, 100)])
def test_q8t_output(K, N):
    M = 20
    assert K * N > 2 ** 31
    gen = torch.Generator(DEV).manual_seed(N)
    codes = integers(gen, M, -(-K // 16) * 16, 127, torch.int8)
    s = torch.full((1, K), 0.5, device=DEV)
    s[:, ::3] = 2.0
    dY = integers(gen, M, N, 2, torch.bfloat16)
    dW = rtm.gemm_q8tbf16f32(codes, s, dY)
    rows, cols = places(K, 3000, gen), places(N, 300, gen)
    x = codes[:, rows].double() * s[:, rows].double()
    assert torch.equal(dW[rows][:, cols].double(), x.t() @ dY[:, cols].double())
    assert rtm.get_device_error() == 0


def test_q8t_longest_sum():
    M, N, K = LONGEST, 8, 5
    gen = torch.Generator(DEV).manual_seed(3)
    codes = torch.full((M, 16), 3, dtype=torch.int8, device=DEV)
    codes[:, 1] = -5
    s = torch.full((M // 128, K), 0.5, device=DEV)
    s[::3] = 2.0
    m = places(M, 4000, gen)
    codes[m] = integers(gen, len(m), 16, 127, torch.int8)
    dY = torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)
    dY[m] = integers(gen, len(m), N, 2, torch.bfloat16)
    dW = rtm.gemm_q8tbf16f32(codes, s, dY)
    x = codes[m, :K].double() * s[m // 128].double()
    assert torch.equal(dW.double(), x.t() @ dY[m].double())
    assert rtm.get_device_error() == 0
