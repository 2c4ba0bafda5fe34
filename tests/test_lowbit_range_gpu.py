"""Values at the ends of the types' ranges in the low-bit formats and products."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import lowbit_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rtm.build()
    rtm.load_library()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N", [16, 65])
def test_w4_range_beyond_fp32(N, group):
    """Finite weights whose hi - lo overflows fp32 keep a finite scale, hi / 15 - lo / 15, and
    read back within a step."""
    gen = torch.Generator().manual_seed(N)
    W = ((torch.rand(256, N, generator=gen, dtype=torch.float64) - 0.5) * 4.8e38).to(torch.bfloat16)
    W[::16] = 2.4e38
    W[1::16] = -2.4e38
    codes, s, z = rtm.gemm_w4_quantize(W.to(DEV), group)
    fifteenth = torch.tensor(1 / 15)
    g = W.float().view(-1, group, N)
    hi, lo = g.amax(1), g.amin(1)
    assert torch.isfinite(W).all() and torch.isinf(hi - lo).all()
    want_s = (hi * fifteenth - lo * fifteenth).to(torch.bfloat16)
    inv = torch.ones_like(hi) / want_s.float()
    want_z = torch.round(-lo * inv).clamp(0, 15)
    want_q = (torch.round(g * inv[:, None]) + want_z[:, None]).clamp(0, 15).view(256, N)
    assert torch.equal(s.cpu(), want_s) and torch.equal(z.cpu(), want_z.to(torch.uint8))
    q = ref.w4_unpack(codes.cpu(), 256)
    assert torch.equal(q, want_q.to(torch.uint8))
    back = rtm.gemm_w4_dequantize(codes, s, z, 256, group).cpu().double()
    step = want_s.double()[torch.arange(256) // group]
    # a step at the clamped ends, and bf16 rounds what is read back
    assert ((back - W.double()).abs() <= step * (1 + 15 * 2.0 ** -8)).all()


@pytest.mark.parametrize("M", [1, 12, 40, 100, 300])
@pytest.mark.parametrize("dtype,largest", [(torch.bfloat16, 2.0 ** 117), (torch.float16, 65504.0)])
def test_w4_largest_operands(M, dtype, largest):
    """Up to |A| = 2^117 (any fp16 value) the sums of unscaled codes stay finite: here every
    code is 15 above its zero point and every product has one sign."""
    K, N = 384, 72
    codes = rtm.gemm_w4_pack(torch.full((K, N), 15, dtype=torch.uint8, device=DEV))
    s = torch.full((K // 128, N), 2.0 ** -20, dtype=dtype, device=DEV)
    z = torch.zeros(K // 128, N, dtype=torch.uint8, device=DEV)
    A = torch.full((M, K), largest, dtype=dtype, device=DEV)
    A[-1] = -A[-1]
    product = rtm.gemm_bf16w4f32 if dtype == torch.bfloat16 else rtm.gemm_f16w4f32
    C = product(A, codes, s, z).double().cpu()
    want = torch.full((M, N), K * 15 * 2.0 ** -20 * largest, dtype=torch.float64)
    want[-1] = -want[-1]
    a, w = torch.full((M, K), largest, dtype=torch.float64), torch.full((K, N), 15 * 2.0 ** -20).double()
    ref.assert_within(C, want, ref.product_bound(K, a, w))


@pytest.mark.parametrize("N", [40, 100, 300])
@pytest.mark.parametrize("dtype,largest", [(torch.bfloat16, 2.0 ** 113), (torch.float16, 65504.0)])
def test_q8t_largest_operands(N, dtype, largest):
    """Up to |dY| = 2^113 with the largest code, -128."""
    M, K = 300, 72
    codes = torch.full((M, 80), -128, dtype=torch.int8, device=DEV)
    s = torch.full((3, K), 2.0 ** -20, device=DEV)
    dY = torch.full((M, N), largest, dtype=dtype, device=DEV)
    gradient = rtm.gemm_q8tbf16f32 if dtype == torch.bfloat16 else rtm.gemm_q8tf16f32
    dW = gradient(codes, s, dY).double().cpu()
    x, d = torch.full((K, M), -2.0 ** -13).double(), torch.full((M, N), largest).double()
    ref.assert_within(dW, x @ d, ref.product_bound(M, x, d))


@pytest.mark.parametrize("M", [1, 12, 40, 100, 300])
def test_w4_infinite_scale(M):
    """An infinite scale multiplies its group's sum: infinite where the sum is not zero, also
    with codes at the zero point among them, and NaN where it is."""
    K, N = 256, 24
    q = torch.full((K, N), 5, dtype=torch.uint8)
    q[128, :8] = 9        # sum 4 a
    q[130, 8:16] = 1      # sum -4 a
    s = torch.ones(2, N, dtype=torch.bfloat16)
    s[1] = float("inf")
    z = torch.full((2, N), 5, dtype=torch.uint8)
    A = torch.ones(M, K, dtype=torch.bfloat16)
    C = rtm.gemm_bf16w4f32(A.to(DEV), rtm.gemm_w4_pack(q.to(DEV)), s.to(DEV), z.to(DEV)).cpu()
    inf = float("inf")
    assert (C[:, :8] == inf).all() and (C[:, 8:16] == -inf).all() and torch.isnan(C[:, 16:]).all()
