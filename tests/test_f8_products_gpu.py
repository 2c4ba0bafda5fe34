"""Products of 8-bit floating-point operands and their gradients against 64-bit products of the
values that the codes stand for; the tolerance is derived in f8_reference.close."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import f8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    rtm.build()
    yield
    torch.cuda.synchronize()
    assert rtm.get_device_error() == 0


def codes(M, K, seed, pitch=None):
    """Any codes but NaN, rows `pitch` bytes apart; what lies between the rows is NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pitch = pitch or (K + 15) // 16 * 16
    held = torch.full((M, pitch), 0x7F, dtype=torch.uint8, device=DEV)
    v = (torch.randn(M, K, generator=g, device=DEV) * 60).clamp(-448, 448).to(F8)
    held[:, :K] = v.view(torch.uint8)
    return held.view(F8)[:, :K]


def scales(*shape, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.exp2(torch.randn(shape, generator=g, device=DEV) * 3) * 0.01


def blocks(n):
    return (n + 127) // 128


def operands(direction, M, N, K, seed=0, pitches=(None, None)):
    """(A, its scales, B, its scales, A's values, B's values as the product's right side)."""
    if direction == "forward":
        a, s = codes(M, K, seed, pitches[0]), scales(M, blocks(K), seed=seed)
        w, t = codes(K, N, seed + 1, pitches[1]), scales(blocks(K), blocks(N), seed=seed + 1)
        return a, s, w, t, ref.values(a, s, "rows"), ref.values(w, t, "tiles")
    if direction == "input":
        a, s = codes(M, N, seed, pitches[0]), scales(M, blocks(N), seed=seed)
        w, t = codes(K, N, seed + 1, pitches[1]), scales(blocks(K), blocks(N), seed=seed + 1)
        return a, s, w, t, ref.values(a, s, "rows"), ref.values(w, t, "tiles").t()
    a, s = codes(M, K, seed, pitches[0]), scales(blocks(M), K, seed=seed)
    b, t = codes(M, N, seed + 1, pitches[1]), scales(blocks(M), N, seed=seed + 1)
    return a, s, b, t, ref.values(a, s, "columns").t(), ref.values(b, t, "columns")


CALLS = {"forward": rtm.gemm_f8w8f32, "input": rtm.gemm_f8w8tf32, "weight": rtm.gemm_f8tf8f32}


def check(direction, M, N, K, seed=0, **more):
    a, s, b, t, left, right = operands(direction, M, N, K, seed, **more)
    got = CALLS[direction](a, s, b, t)
    assert got.shape == (left.shape[0], right.shape[1]) and got.dtype == torch.float32
    ref.close(got, left @ right, left.abs() @ right.abs(), blocks(left.shape[1]))
    assert torch.equal(got, CALLS[direction](a, s, b, t)), "results repeat exactly"


ROWS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500]


@pytest.mark.parametrize("direction", ["forward", "input"])
@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("N,K", [(128, 128), (259, 300), (1, 1), (1000, 16), (130, 2100)])
def test_every_number_of_rows(direction, M, N, K):
    check(direction, M, N, K, seed=M)


@pytest.mark.parametrize("M", [1, 127, 128, 129, 1000, 4097])
@pytest.mark.parametrize("N,K", [(128, 128), (259, 300), (1, 1), (500, 129), (40, 1030)])
def test_weight_gradients(M, N, K):
    check("weight", M, N, K, seed=M)


@pytest.mark.parametrize("direction", CALLS)
@pytest.mark.parametrize("M,N,K", [(2000, 4100, 520), (520, 2000, 4100), (4100, 520, 2000),
                                   (2048, 2048, 2048), (3001, 1023, 515), (1025, 5000, 1041)])
def test_large_tiles(direction, M, N, K):
    check(direction, M, N, K, seed=7)


@pytest.mark.parametrize("direction", CALLS)
@pytest.mark.parametrize("M", [3, 100, 2200])
def test_strided_rows(direction, M):
    N, K = 200, 600
    if direction == "input":
        N, K = K, N
    check(direction, M, N, K, seed=5, pitches=(1024, 848))


def test_views_of_one_buffer():
    """Operands that start inside another tensor's rows, on 16-byte boundaries."""
    whole = codes(300, 1024, 3, 1024)
    a, s = whole[16:116, 128:528], scales(100, 4)
    w, t = codes(400, 256, 4), scales(4, 2)
    left, right = ref.values(a, s, "rows"), ref.values(w, t, "tiles")
    ref.close(rtm.gemm_f8w8f32(a, s, w, t), left @ right, left.abs() @ right.abs(), 4)


def test_contiguous_codes_and_a_given_result():
    a, w = codes(200, 256, 1, 256).contiguous(), codes(256, 64, 2, 64).contiguous()
    s, t = scales(200, 2), scales(2, 1)
    whole = torch.full((202, 64), 7.0, device=DEV)
    out = whole[1:201]
    assert rtm.gemm_f8w8f32(a, s, w, t, out=out) is out
    assert torch.equal(out, rtm.gemm_f8w8f32(a, s, w, t))
    assert (whole[0] == 7).all() and (whole[201] == 7).all(), "beside the result nothing is written"
    odd = torch.full((200 * 64 + 1,), 7.0, device=DEV)[1:].view(200, 64)  # off 16 bytes
    assert torch.equal(rtm.gemm_f8w8f32(a, s, w, t, out=odd), out)


@pytest.mark.parametrize("direction", CALLS)
@pytest.mark.parametrize("M,N,K", [(2030, 2004, 2012), (2030, 2002, 2010), (2031, 2001, 2009)])
def test_large_results_at_every_alignment(direction, M, N, K):
    """Rows of 16, 8 and 4 bytes' multiples, from 0, 4, 8 and 12 bytes behind a boundary."""
    a, s, b, t, left, right = operands(direction, M, N, K)
    rows, cols = left.shape[0], right.shape[1]
    want = CALLS[direction](a, s, b, t)
    ref.close(want, left @ right, left.abs() @ right.abs(), blocks(left.shape[1]))
    for shift in range(4):
        whole = torch.full((rows * cols + 64,), 7.0, device=DEV)
        out = whole[32 + shift:32 + shift + rows * cols].view(rows, cols)
        CALLS[direction](a, s, b, t, out=out)
        assert torch.equal(out, want)
        assert (whole[:32 + shift] == 7).all() and (whole[32 + shift + rows * cols:] == 7).all()


@pytest.mark.parametrize("M", [5, 100, 600])
def test_not_a_number_stays_in_its_row_and_column(M):
    K, N = 300, 400
    a, s, w, t, left, right = operands("forward", M, N, K)
    s[M // 2, 1] = torch.nan
    t[2, 3] = torch.inf
    a.view(torch.uint8)[0, 7] = 0x7F  # a NaN code
    got = rtm.gemm_f8w8f32(a, s, w, t)
    bad = torch.zeros(M, N, dtype=torch.bool, device=DEV)
    bad[0], bad[M // 2], bad[:, 384:] = True, True, True
    assert torch.equal(~got.isfinite(), bad)


def test_not_a_number_in_the_weight_gradient():
    M, K, N = 500, 300, 600
    x, s, y, t, left, right = operands("weight", M, N, K)
    s[2, 17], t[3, 500] = torch.nan, torch.nan
    got = rtm.gemm_f8tf8f32(x, s, y, t)
    bad = torch.zeros(K, N, dtype=torch.bool, device=DEV)
    bad[17], bad[:, 500] = True, True
    assert torch.equal(got.isnan(), bad)


@pytest.mark.parametrize("M,N,K", [(0, 5, 7), (5, 0, 7), (5, 7, 0), (200, 300, 0), (0, 0, 0)])
def test_empty_sizes(M, N, K):
    f8 = lambda r, c: torch.zeros(r, c, dtype=torch.uint8, device=DEV).view(F8)  # noqa: E731
    for name, a, b, s, t in (
            ("forward", f8(M, K), f8(K, N), (M, blocks(K)), (blocks(K), blocks(N))),
            ("input", f8(M, N), f8(K, N), (M, blocks(N)), (blocks(K), blocks(N))),
            ("weight", f8(M, K), f8(M, N), (blocks(M), K), (blocks(M), N))):
        if a.numel() or b.numel():  # rows of the operand that is there on 16 bytes
            a = torch.zeros(a.shape[0], (a.shape[1] + 15) // 16 * 16, dtype=torch.uint8,
                            device=DEV).view(F8)[:, :a.shape[1]]
            b = torch.zeros(b.shape[0], (b.shape[1] + 15) // 16 * 16, dtype=torch.uint8,
                            device=DEV).view(F8)[:, :b.shape[1]]
        out = CALLS[name](a, torch.ones(s, device=DEV), b, torch.ones(t, device=DEV))
        assert out.shape == {"forward": (M, N), "input": (M, K), "weight": (K, N)}[name]
        assert not out.any()


def test_extreme_scales():
    """Products whose scales' product is near the ends of fp32's range keep their accuracy."""
    a, w = codes(40, 256, 1), codes(256, 128, 2)
    for e in (-70, 55):
        s = torch.full((40, 2), 2.0 ** e, device=DEV)
        t = torch.full((2, 1), 2.0 ** (e // 2), device=DEV)
        left, right = ref.values(a, s, "rows"), ref.values(w, t, "tiles")
        ref.close(rtm.gemm_f8w8f32(a, s, w, t), left @ right, left.abs() @ right.abs(), 2)


def test_another_stream():
    a, s, w, t, left, right = operands("forward", 300, 700, 900)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rtm.gemm_f8w8f32(a, s, w, t, stream=side)
    q = rtm.gemm_f8_quantize(torch.ones(64, 64, device=DEV), stream=side)
    side.synchronize()
    assert torch.equal(got, rtm.gemm_f8w8f32(a, s, w, t)) and len(q) == 2


def test_refusals():
    a, s, w, t, _, _ = operands("forward", 20, 40, 300)
    far = torch.zeros(300, 320, dtype=torch.uint8, device=DEV).view(F8)
    calls = [lambda: rtm.gemm_f8w8f32(a, s, w.t(), t), lambda: rtm.gemm_f8w8f32(a[:, :200], s, w, t),
             lambda: rtm.gemm_f8w8f32(a, s[:, :2], w, t), lambda: rtm.gemm_f8w8f32(a, s.half(), w, t),
             lambda: rtm.gemm_f8w8f32(a, s, w, t.t()), lambda: rtm.gemm_f8w8f32(a.cpu(), s, w, t),
             lambda: rtm.gemm_f8w8f32(a, s.cpu(), w, t), lambda: rtm.gemm_f8w8f32(a.float(), s, w, t),
             lambda: rtm.gemm_f8w8f32(a[:, 8:], s, w[8:], t),  # rows off 16 bytes
             lambda: rtm.gemm_f8w8f32(far[:20, ::2][:, :300], s, w, t),
             lambda: rtm.gemm_f8w8f32(a, s, w, t, out=torch.empty(20, 41, device=DEV)),
             lambda: rtm.gemm_f8w8f32(a, s, w, t, out=torch.empty(20, 40, device=DEV).half()),
             lambda: rtm.gemm_f8w8f32(a.view(torch.uint8), s, w, t),
             lambda: rtm.gemm_f8tf8f32(a, s, w, t), lambda: rtm.gemm_f8w8tf32(a, s, w, t)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(rtm.GemmError):  # the result over an operand
        out = w.as_strided((300, 48), (48, 1)).view(torch.uint8).flatten()[:20 * 40 * 4]
        rtm.gemm_f8w8f32(a, s, w, t, out=out.view(torch.float32).view(20, 40))


def test_codes_past_32_bits():
    """A weight of more than 2^31 codes: the last columns and rows against their own product."""
    K, N = 16400, 133000
    g = torch.Generator(device=DEV).manual_seed(2)
    held = torch.randint(0, 0x70, (K, (N + 15) // 16 * 16), generator=g, device=DEV,
                         dtype=torch.uint8)
    w = held.view(F8)[:, :N]
    t = scales(blocks(K), blocks(N), seed=3)
    for M in (3, 300):
        a, s = codes(M, K, 1), scales(M, blocks(K), seed=1)
        got = rtm.gemm_f8w8f32(a, s, w, t)
        first = (blocks(N) - 2) * 128
        left = ref.values(a, s, "rows")
        right = ref.values(w[:, first:], t[:, blocks(N) - 2:], "tiles")
        ref.close(got[:, first:], left @ right, left.abs() @ right.abs(), blocks(K))
