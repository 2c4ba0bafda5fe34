"""GPU tests of the low-bit conversions: 4-bit weights and 8-bit activations
against their definition in fp32 steps on the host, bit for bit."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import lowbit_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rtm.build()
    rtm.load_library()


def bits(t):
    return t.cpu().contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(got, want):
    """Equal bit for bit, NaNs of any payload alike."""
    got, want = got.cpu(), want.cpu()
    assert got.dtype == want.dtype and got.shape == want.shape
    if got.is_floating_point():
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        keep = ~torch.isnan(want)
        got, want = got[keep], want[keep]
    assert torch.equal(bits(got), bits(want))


def weights(K, N, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(K, N, generator=gen) * 0.02).to(dtype)


def check_w4(W, group, zeros, on_gpu=None):
    K, N = W.shape
    codes, s, z = rtm.gemm_w4_quantize(W.to(DEV) if on_gpu is None else on_gpu, group, zeros=zeros)
    q0, s0, z0 = ref.w4_quantize(W, group, zeros)
    same(s, s0)
    assert (z is None) == (z0 is None)
    if zeros:
        same(z, z0)
    assert codes.shape == (N, (K + 127) // 128 * 64)
    q = ref.w4_unpack(codes.cpu(), K)
    same(q, q0)
    back = rtm.gemm_w4_dequantize(codes, s, z, K, group)
    g = torch.arange(K) // group
    zz = 8.0 if z0 is None else z0.float()[g]
    same(back, ((q0.float() - zz) * s0.float()[g]).to(W.dtype))
    return codes, s, z


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K,N", [(1, 1), (33, 65), (128, 64), (129, 72), (515, 130), (1000, 200)])
def test_w4_quantize(K, N, dtype, zeros, group):
    check_w4(weights(K, N, dtype, K * 7 + N), group, zeros)


@pytest.mark.parametrize("dtype", TYPES)
def test_w4_quantize_offset_pointer(dtype):
    """Rows of a width that fits 16-byte loads on a base that does not."""
    W = weights(130, 64, dtype, 5)
    room = torch.empty(130 * 64 + 1, dtype=dtype, device=DEV)
    view = room[1:].view(130, 64)
    view.copy_(W)
    check_w4(W, 64, True, on_gpu=view)
    codes, s, z = rtm.gemm_w4_quantize(view, 64)
    out = torch.zeros(130 * 64 + 2, dtype=dtype, device=DEV)
    got = rtm.gemm_w4_dequantize(codes, s, z, 130, 64, out=out[1:-1].view(130, 64))
    same(got, rtm.gemm_w4_dequantize(codes, s, z, 130, 64))
    assert out[0] == 0 and out[-1] == 0


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
def test_w4_unusual_groups(dtype, zeros):
    """Groups of zeros, of one sign, of the smallest values, with infinities and NaN."""
    W = weights(256, 16, dtype, 9)
    W[:128, 0] = 0
    W[:128, 1] = W[:128, 1].abs() + 0.01
    W[:128, 2] = -W[:128, 2].abs() - 0.01
    W[:128, 3] = torch.finfo(dtype).tiny / 64
    W[5, 4] = float("inf")
    W[200, 5] = float("nan")
    W[7, 6] = -float("inf")
    W[:128, 7] = torch.finfo(dtype).max / 4
    W[3, 8] = torch.finfo(dtype).max
    W[:, 9] = -0.0
    codes, s, z = check_w4(W, 128, zeros)
    back = rtm.gemm_w4_dequantize(codes, s, z, 256, 128).cpu()
    assert torch.isnan(back[:128, 4]).all() and torch.isnan(back[128:, 5]).all()
    assert torch.isfinite(back[128:, 4]).all() and (back[:, 9] == 0).all()


def test_w4_error_is_half_a_step():
    """Each weight comes back within half a step, and half a step more at the
    ends, where rounding the zero point and the scale may cut the range."""
    W = weights(384, 96, torch.bfloat16, 3)
    codes, s, z = rtm.gemm_w4_quantize(W.to(DEV), 128)
    q = ref.w4_unpack(codes.cpu(), 384)
    err = (ref.w4_values(q, s.cpu(), z.cpu(), 128) - W.double()).abs()
    step = s.cpu().double()[torch.arange(384) // 128]
    assert (err <= step * (1 + 15 * 2.0 ** -8)).all()
    inner = (q > 0) & (q < 15)
    assert (err[inner] <= (step * (0.5 + 2.0 ** -16))[inner]).all()


@pytest.mark.parametrize("K,N", [(1, 3), (128, 64), (300, 70)])
def test_w4_pack(K, N):
    gen = torch.Generator().manual_seed(K)
    q = torch.randint(0, 256, (K, N), generator=gen, dtype=torch.uint8)  # high bits ignored
    codes = rtm.gemm_w4_pack(q.to(DEV))
    same(codes, ref.w4_pack(q))


def activations(M, K, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=gen)
    x[:, ::17] *= 16
    return x.to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (127, 15), (128, 128), (129, 136), (300, 257), (513, 72)])
def test_q8_roundtrip(M, K, dtype):
    X = activations(M, K, dtype, M + K)
    codes, s = rtm.gemm_q8_quantize(X.to(DEV))
    q0, s0 = ref.q8_quantize(X)
    same(s, s0)
    same(codes, ref.q8_pad(q0))
    back = rtm.gemm_q8_dequantize(codes, s, M, K, dtype)
    same(back, (q0.float() * s0[torch.arange(M) // 128]).to(dtype))
    err = (q0.double() * s0.double()[torch.arange(M) // 128] - X.double()).abs()
    assert (err <= s0.double()[torch.arange(M) // 128] * (0.5 + 2.0 ** -14)).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_q8_unusual_columns(dtype):
    X = activations(200, 24, dtype, 4)
    X[:, 0] = 0
    X[3, 1] = float("inf")
    X[150, 2] = float("nan")
    X[:, 3] = torch.finfo(dtype).tiny / 4
    X[:, 4] = torch.finfo(dtype).max
    X[9, 5] = -float("inf")
    codes, s = rtm.gemm_q8_quantize(X.to(DEV))
    q0, s0 = ref.q8_quantize(X)
    same(s, s0)
    same(codes, ref.q8_pad(q0))
    back = rtm.gemm_q8_dequantize(codes, s, 200, 24, dtype).cpu()
    assert torch.isnan(back[:128, 1]).all() and torch.isfinite(back[128:, 1]).all()
    assert torch.isnan(back[128:, 2]).all() and (back[:, 0] == 0).all()


def test_q8_offset_pointer():
    X = activations(140, 64, torch.bfloat16, 8)
    room = torch.empty(140 * 64 + 1, dtype=X.dtype, device=DEV)
    view = room[1:].view(140, 64)
    view.copy_(X)
    codes, s = rtm.gemm_q8_quantize(view)
    want_codes, want_s = rtm.gemm_q8_quantize(X.to(DEV))
    same(codes, want_codes)
    same(s, want_s)
    out = torch.zeros(140 * 64 + 2, dtype=X.dtype, device=DEV)
    got = rtm.gemm_q8_dequantize(codes, s, 140, 64, out=out[1:-1].view(140, 64))
    same(got, rtm.gemm_q8_dequantize(codes, s, 140, 64))
    assert out[0] == 0 and out[-1] == 0


def test_empty():
    for K, N in [(0, 8), (8, 0), (0, 0)]:
        W = torch.empty(K, N, dtype=torch.bfloat16, device=DEV)
        codes, s, z = rtm.gemm_w4_quantize(W)
        assert rtm.gemm_w4_dequantize(codes, s, z, K).shape == (K, N)
        c8, s8 = rtm.gemm_q8_quantize(W)
        assert rtm.gemm_q8_dequantize(c8, s8, K, N).shape == (K, N)
    torch.cuda.synchronize()


def test_side_stream():
    """A call on another stream sees that stream's inputs and orders its outputs after them."""
    side = torch.cuda.Stream()
    W = weights(512, 512, torch.bfloat16, 1)
    want = rtm.gemm_w4_dequantize(*rtm.gemm_w4_quantize(W.to(DEV)), 512)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        w = torch.zeros(512, 512, dtype=torch.bfloat16, device=DEV)
        torch.cuda._sleep(2_000_000)
        w.copy_(W)
    codes, s, z = rtm.gemm_w4_quantize(w, stream=side)
    got = rtm.gemm_w4_dequantize(codes, s, z, 512, stream=side)
    side.synchronize()
    same(got, want)


def test_refusals():
    W = torch.zeros(128, 64, dtype=torch.bfloat16, device=DEV)
    codes, s, z = rtm.gemm_w4_quantize(W)
    for bad in (lambda: rtm.gemm_w4_quantize(W, 48), lambda: rtm.gemm_w4_quantize(W.float()),
                lambda: rtm.gemm_w4_quantize(W.t()), lambda: rtm.gemm_w4_quantize(W.cpu()),
                lambda: rtm.gemm_w4_dequantize(codes, s, z, 300),
                lambda: rtm.gemm_w4_dequantize(codes, s[:, :8], z, 128),
                lambda: rtm.gemm_w4_dequantize(codes, s.float(), z, 128),
                lambda: rtm.gemm_w4_dequantize(codes, s, z.int(), 128),
                lambda: rtm.gemm_w4_pack(W), lambda: rtm.gemm_q8_quantize(W[:, ::2]),
                lambda: rtm.gemm_q8_dequantize(codes, s, 128, 64),
                lambda: rtm.gemm_w4_dequantize(codes, s, z, 128, out=W.float())):
        with pytest.raises(ValueError):
            bad()
