"""Conversions to e4m3 codes with block scales and back, against the definition in 64 bits: a
power-of-two scale makes every step but the code's rounding exact, so codes and scales are equal
to the last bit."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import f8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    rtm.build()


def values(M, K, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(M, K, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-6, 7, (M, K), generator=g, device=DEV).float())
    return x.to(dtype)


def check(codes, scales, x, kind):
    want, s = ref.quantize(x, kind)
    assert codes.shape == x.shape and codes.dtype == torch.float8_e4m3fn
    assert torch.equal(scales.double().nan_to_num(nan=-1.0), s.nan_to_num(nan=-1.0))
    assert torch.equal(codes.double(), want)
    if codes.numel():
        K = x.shape[1]
        padded = codes.view(torch.uint8).as_strided((x.shape[0], codes.stride(0) if x.shape[0] > 1
                                                     else (K + 15) // 16 * 16),
                                                    (codes.stride(0), 1))
        assert not padded[:, K:].any(), "bytes past a row are 0"


SIZES = [(1, 1), (1, 128), (3, 7), (16, 129), (127, 128), (128, 127), (129, 260), (300, 1023),
         (257, 16), (1000, 384)]


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,K", SIZES)
def test_all_kinds(M, K, type_):
    x = values(M, K, TYPES[type_], seed=M + K)
    rows, columns = rtm.gemm_f8_quantize(x, "rows"), rtm.gemm_f8_quantize(x, "columns")
    both, tiles = rtm.gemm_f8_quantize(x, "both"), rtm.gemm_f8_quantize_tiles(x)
    torch.cuda.synchronize()
    for got, kind in ((rows, "rows"), (columns, "columns"), (both[:2], "rows"),
                      (both[2:], "columns"), (tiles, "tiles")):
        check(*got, x, kind)
        for dtype in TYPES.values():
            # code * scale is exact in 32 bits, and rounded once to 16
            want = ref.values(*got, kind).to(dtype)
            assert torch.equal(rtm.gemm_f8_dequantize(*got, kind, dtype), want)


@pytest.mark.parametrize("E,K,N", [(1, 130, 70), (3, 128, 128), (5, 200, 333)])
def test_several_matrices(E, K, N):
    w = values(E * K, N, torch.bfloat16, seed=E).view(E, K, N)
    codes, scales = rtm.gemm_f8_quantize_tiles(w)
    back = rtm.gemm_f8_dequantize(codes, scales, "tiles", torch.float32)
    for e in range(E):
        want, s = ref.quantize(w[e], "tiles")
        assert torch.equal(codes[e].double(), want) and torch.equal(scales[e].double(), s)
        assert torch.equal(back[e], ref.values(codes[e], scales[e], "tiles").float())


def test_any_scales_come_back_rounded_once():
    codes = values(130, 200, torch.float32).clamp(-400, 400).to(torch.float8_e4m3fn)
    held = torch.zeros(130, 208, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)[:, :200]
    held.view(torch.uint8).copy_(codes.view(torch.uint8))
    for kind, shape in (("rows", (130, 2)), ("columns", (2, 200)), ("tiles", (2, 2))):
        s = torch.rand(shape, device=DEV) + 0.3
        want = ref.values(held, s, kind).float()  # 28 bits, once to 24 (and then once to 8)
        assert torch.equal(rtm.gemm_f8_dequantize(held, s, kind, torch.float32), want)
        assert torch.equal(rtm.gemm_f8_dequantize(held, s, kind, torch.bfloat16), want.bfloat16())


@pytest.mark.parametrize("kind", ["rows", "columns", "tiles"])
def test_special_blocks(kind):
    x = torch.ones(384, 384, device=DEV)
    x[5, 5], x[200, 5], x[5, 200] = torch.nan, torch.inf, -torch.inf
    x[130:256, 130:256] = 0
    x[256:, :128] = 2.0 ** -101           # below the least scale
    x[256:, 128:256] = 2.0 ** -100
    x[256:, 256:] = 3.4e38
    x[300, 300] = -3.4028234663852886e38  # the largest value
    x[128:256, 256:] = torch.tensor([1.75, 1.75 + 2.0 ** -23], device=DEV).repeat(64)  # 448 * 2^-8
    got = rtm.gemm_f8_quantize_tiles(x) if kind == "tiles" else rtm.gemm_f8_quantize(x, kind)
    check(*got, x, kind)
    back = rtm.gemm_f8_dequantize(*got, kind, torch.float32)
    bad = ref.spread(got[1].isnan(), *ref.blocks_of(kind), 384, 384)
    assert bad.any() and torch.equal(back.isnan(), bad)


def test_halves_go_to_even():
    # 1 + i / 16 between the codes 1 + j / 8, and the subnormals' steps of 2^-9
    x = torch.zeros(1, 128, device=DEV)
    x[0, 0] = 448
    x[0, 1:17] = 1 + torch.arange(16, device=DEV) / 16
    x[0, 17:49] = torch.arange(32, device=DEV) * 2.0 ** -10
    x[0, 49:81] = -x[0, 17:49]
    check(*rtm.gemm_f8_quantize(x, "rows"), x, "rows")


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("kind", ["rows", "columns", "both"])
@pytest.mark.parametrize("M,K,fan", [(7, 130, 1), (50, 64, 3), (300, 259, 4)])
def test_gathered(M, K, fan, kind, type_):
    x = values(M, K, TYPES[type_], seed=M)
    g = torch.Generator(device=DEV).manual_seed(1)
    rows = torch.randint(-1, M * fan, (M * fan + 40,), generator=g, device=DEV, dtype=torch.int32)
    rows[3], rows[9], rows[11] = M * fan, 2 ** 31 - 1, -2 ** 31  # none of them a slot
    factors = torch.randn(M, fan, generator=g, device=DEV)
    for f in (None, factors):
        want = ref.gathered(x, rows, fan, f)
        got = rtm.gemm_f8_quantize(x, kind, gather=rows, fan=fan, factors=f)
        pairs = {"rows": [(got[:2], "rows")], "columns": [(got[:2], "columns")],
                 "both": [(got[:2], "rows"), (got[2:], "columns")]}[kind]
        for pair, one in pairs:
            check(*pair, want, one)


def test_unaligned_rows_of_the_input():
    flat = values(1, 64 * 128 + 1, torch.bfloat16)[0]
    x = flat[1:].view(64, 128)  # 2 bytes off a 16-byte boundary
    check(*rtm.gemm_f8_quantize(x, "rows"), x, "rows")
    check(*rtm.gemm_f8_quantize(x, "columns"), x, "columns")


def test_empty():
    for M, K in ((0, 16), (5, 0), (0, 0)):
        x = torch.empty(M, K, device=DEV)
        for got in (rtm.gemm_f8_quantize(x, "both"), rtm.gemm_f8_quantize_tiles(x)):
            assert got[0].shape == (M, K)
        assert rtm.gemm_f8_dequantize(*rtm.gemm_f8_quantize(x), "rows").shape == (M, K)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert rtm.gemm_f8_quantize(torch.ones(3, 20, device=DEV), gather=none)[0].shape == (0, 20)
    # rows gathered from nothing are zeros
    codes, s = rtm.gemm_f8_quantize(torch.empty(0, 20, device=DEV),
                                    gather=torch.zeros(4, dtype=torch.int32, device=DEV))
    assert not codes.double().any() and not s.any()


def test_refusals():
    x = torch.ones(8, 32, device=DEV)
    q, s = rtm.gemm_f8_quantize(x)
    rows = torch.zeros(8, dtype=torch.int32, device=DEV)
    calls = [lambda: rtm.gemm_f8_quantize(x.double()), lambda: rtm.gemm_f8_quantize(x.t()),
             lambda: rtm.gemm_f8_quantize(x, "tiles"), lambda: rtm.gemm_f8_quantize(x[0]),
             lambda: rtm.gemm_f8_quantize(x, fan=2), lambda: rtm.gemm_f8_quantize(x, gather=rows.long()),
             lambda: rtm.gemm_f8_quantize(x, gather=rows, fan=0),
             lambda: rtm.gemm_f8_quantize(x, gather=rows, fan=True),
             lambda: rtm.gemm_f8_quantize(x, gather=rows, factors=torch.ones(7, device=DEV)),
             lambda: rtm.gemm_f8_quantize(x, gather=rows, factors=torch.ones(8)),
             lambda: rtm.gemm_f8_quantize(x, factors=torch.ones(8, device=DEV)),
             lambda: rtm.gemm_f8_quantize(x, gather=rows, factors=torch.ones(8, device=DEV).half()),
             lambda: rtm.gemm_f8_quantize_tiles(x.int()),
             lambda: rtm.gemm_f8_dequantize(q, s, "rows", torch.float64),
             lambda: rtm.gemm_f8_dequantize(q, s, "blocks"), lambda: rtm.gemm_f8_dequantize(q, s.half()),
             lambda: rtm.gemm_f8_dequantize(q, s, "columns"), lambda: rtm.gemm_f8_dequantize(x, s),
             lambda: rtm.gemm_f8_dequantize(q.t(), s), lambda: rtm.gemm_f8_dequantize(q[:, 1:], s),
             lambda: rtm.gemm_f8_dequantize(q, s, out=torch.empty(8, 32, device=DEV))]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")


def test_rows_past_32_bits():
    """More than 2^31 values: the last rows come out as they do alone."""
    M, K = 262200, 8208
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)
    tail = values(200, K, torch.bfloat16)
    x[-200:] = tail
    q, s, qc, sc = rtm.gemm_f8_quantize(x, "both")
    want, ws = ref.quantize(tail, "rows")
    assert torch.equal(q[-200:].double(), want) and torch.equal(s[-200:].double(), ws)
    first = M - M % 128  # the last block of columns holds rows of the tail alone
    want, ws = ref.quantize(x[first:], "columns")
    assert torch.equal(qc[first:].double(), want) and torch.equal(sc[-1:].double(), ws)
    back = rtm.gemm_f8_dequantize(q, s, "rows", torch.bfloat16)
    assert torch.equal(back[-200:], ref.values(q[-200:], s[-200:], "rows").bfloat16())


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,K", [(4100, 4096), (2600, 6416), (140000, 16), (127, 131200)])
def test_rows_alone_of_whole_sixteens(M, K, type_):
    """The kernel of large conversions along rows, plain and gathered with factors."""
    x = values(M, K, TYPES[type_], seed=K)
    x[5, 3], x[M - 1, K - 1], x[7] = torch.nan, torch.inf, 0
    check(*rtm.gemm_f8_quantize(x, "rows"), x, "rows")
    g = torch.Generator(device=DEV).manual_seed(2)
    rows = torch.randint(-1, 2 * M, (M,), generator=g, device=DEV, dtype=torch.int32)
    rows[3] = 2 * M
    factors = torch.randn(M, 2, generator=g, device=DEV)
    got = rtm.gemm_f8_quantize(x, "rows", gather=rows, fan=2, factors=factors)
    check(*got, ref.gathered(x, rows, 2, factors), "rows")
    whole = torch.empty(M * K + 8, dtype=x.dtype, device=DEV)
    odd = whole[8:].view(M, K)  # 16 bytes (fp32: 32) on: another kernel
    odd.copy_(x)
    for a, b in zip(rtm.gemm_f8_quantize(odd, "rows"), rtm.gemm_f8_quantize(x, "rows")):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,K", [(1, 16), (129, 48), (257, 1024), (100, 144), (1000, 2000)])
def test_scales_that_span_rows_of_whole_sixteens(M, K, type_):
    """The kernels of such rows, and the one of rows off 16 bytes: the same codes."""
    x = values(M, K, TYPES[type_], seed=K)
    x[M // 2, K - 3], x[M - 1, 1], x[0] = torch.nan, -torch.inf, 0
    x[:, 2] = 2.0 ** -20 if type_ == "f16" else 2.0 ** -110
    whole = torch.empty(M * K + 1, dtype=x.dtype, device=DEV)
    odd = whole[1:].view(M, K)
    odd.copy_(x)
    for one in (x, odd):
        both = rtm.gemm_f8_quantize(one, "both")
        check(*both[:2], x, "rows")
        check(*both[2:], x, "columns")
        check(*rtm.gemm_f8_quantize(one, "columns"), x, "columns")
        check(*rtm.gemm_f8_quantize_tiles(one), x, "tiles")
    g = torch.Generator(device=DEV).manual_seed(3)
    rows = torch.randint(-1, 3 * M + 1, (M + 77,), generator=g, device=DEV, dtype=torch.int32)
    factors = torch.randn(M, 3, generator=g, device=DEV)
    for f in (None, factors):
        want = ref.gathered(x, rows, 3, f)
        both = rtm.gemm_f8_quantize(x, "both", gather=rows, fan=3, factors=f)
        check(*both[:2], want, "rows")
        check(*both[2:], want, "columns")
        check(*rtm.gemm_f8_quantize(x, "columns", gather=rows, fan=3, factors=f), want, "columns")


def test_matrices_of_whole_sixteens():
    for dtype in TYPES.values():
        w = values(3 * 200, 144, dtype, seed=4).view(3, 200, 144)
        codes, scales = rtm.gemm_f8_quantize_tiles(w)
        for e in range(3):
            want, s = ref.quantize(w[e], "tiles")
            assert torch.equal(codes[e].double(), want) and torch.equal(scales[e].double(), s)


@pytest.mark.parametrize("kind", ["rows", "columns", "tiles"])
def test_back_at_every_alignment(kind):
    """Scales off 16 bytes, results off 32: the same values."""
    M, K = 260, 648
    x = values(M, K, torch.float32)
    codes, s = rtm.gemm_f8_quantize_tiles(x) if kind == "tiles" else rtm.gemm_f8_quantize(x, kind)
    shifted = torch.empty(s.numel() + 1, device=DEV)[1:].view(s.shape)
    shifted.copy_(s)
    for dtype in TYPES.values():
        want = ref.values(codes, s, kind).to(dtype)
        for scales in (s, shifted):
            for off in (0, 1, 4, 8):
                whole = torch.full((M * K + 32,), 7.0, dtype=dtype, device=DEV)
                out = whole[off:off + M * K].view(M, K)
                assert torch.equal(rtm.gemm_f8_dequantize(codes, scales, kind, dtype, out=out), want)
                assert (whole[:off] == 7).all() and (whole[off + M * K:] == 7).all()
