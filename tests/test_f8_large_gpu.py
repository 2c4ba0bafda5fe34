"""8-bit floating-point products whose offsets pass 32 bits. Scales are powers of two; sums of one
term have to be equal."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    rtm.build()
    yield
    torch.cuda.synchronize()
    assert rtm.get_device_error() == 0


@pytest.fixture(autouse=True)
def room():
    yield
    torch.cuda.empty_cache()


def codes(rows, cols, gen):
    """Any codes but NaN, rows padded to 16 bytes."""
    held = torch.randint(0, 0x7f, (rows, (cols + 15) // 16 * 16), generator=gen, device=DEV,
                         dtype=torch.uint8)
    return held.view(F8)[:, :cols]


def scales(rows, cols, gen):
    return torch.exp2(torch.randint(-3, 4, (rows, cols), generator=gen, device=DEV).float())


@pytest.mark.parametrize("N", [2 ** 30 + 1, 2 ** 30 + 4])
def test_weight_gradient_with_rows_of_more_than_4_gb(N):
    """Two rows of the result are 2^31 values apart; rows off 16 bytes and on them."""
    K, gen = 3, torch.Generator(DEV).manual_seed(1)
    x, s = codes(1, K, gen), scales(1, K, gen)
    y, t = codes(1, N, gen), scales(1, N, gen)
    whole = torch.full((K * N + 64,), 7.0, device=DEV)
    out = whole[32:-32].view(K, N)
    rtm.gemm_f8tf8f32(x, s, y, t, out=out)
    assert (whole[:32] == 7).all() and (whole[-32:] == 7).all()
    left = (x.float() * s)[0]
    for c in range(0, N, 1 << 26):
        right = y[0, c:c + (1 << 26)].float() * t[0, c:c + (1 << 26)]
        for k in range(K):
            assert torch.equal(out[k, c:c + (1 << 26)], left[k] * right), (k, c)


@pytest.mark.parametrize("per", [10, 70, 200])
def test_a_stack_of_experts_past_32_bits(per):
    """More than 2^31 codes of W and values of its gradient: the first and last experts' parts
    against their own products."""
    E, K, N = 41, 4096, 13000
    assert E * K * N > 2 ** 31
    gen = torch.Generator(DEV).manual_seed(per)
    w = codes(E * K, N, gen).unflatten(0, (E, K))
    t = scales(E * 32, 102, gen).view(E, 32, 102)
    starts = [e * per for e in range(E + 1)]
    R, offsets = starts[-1], torch.tensor(starts, dtype=torch.int32, device=DEV)

    def few(rows, cols):
        """Eight values of a row that are not 0, at places of its own, in -4 .. 4."""
        held = torch.zeros(rows, (cols + 15) // 16 * 16, device=DEV)
        at = torch.randint(0, cols, (rows, 8), generator=gen, device=DEV)
        held.scatter_(1, at, torch.randint(-4, 5, (rows, 8), generator=gen, device=DEV).float())
        return held.to(F8)[:, :cols]

    def tiles(e):
        full = t[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return w[e].double() * full[:K, :N]

    a, s = few(R, K), torch.ones(R, 32, device=DEV)
    y = rtm.gemm_f8w8f32_experts(a, s, w, t, offsets)
    d, u = few(R, N), torch.ones(R, 102, device=DEV)
    dx = rtm.gemm_f8w8tf32_experts(d, u, w, t, offsets)
    for e in (0, 1, E // 2, E - 1):
        part, right = slice(e * per, (e + 1) * per), tiles(e)
        # eight terms that are not 0: a block's sum, and the total, take at most eight additions
        # each, off by at most a truncated step, 2^-23 of the terms' magnitudes; the scales are exact
        for got, left, b in ((y, a, right), (dx, d, right.t())):
            want, size = left[part].double() @ b, left[part].double().abs() @ b.abs()
            assert ((got[part].double() - want).abs() <= 2.0 ** -19 * size).all(), e


def test_gradients_of_a_stack_of_experts_past_32_bits():
    E, K, N = 41, 4096, 13000
    gen = torch.Generator(DEV).manual_seed(7)
    starts = [128 * e for e in range(E + 1)]
    offsets = torch.tensor(starts, dtype=torch.int32, device=DEV)
    # one row of an expert's 128 is not 0, so that each value is one product
    x, d = (torch.zeros(starts[-1], n, dtype=torch.uint8, device=DEV) for n in (K, 13008))
    x[5::128] = codes(E, K, gen).view(torch.uint8)
    d[5::128, :N] = codes(E, N, gen).view(torch.uint8)
    x, d = x.view(F8), d.view(F8)[:, :N]
    s, u = scales(E, K, gen), scales(E, N, gen)
    got = rtm.gemm_f8tf8f32_experts(x, s, d, u, offsets)
    for e in (0, 1, E // 2, E - 1):
        left, right = x[128 * e + 5].float() * s[e], d[128 * e + 5].float() * u[e]
        assert torch.equal(got[e], left[:, None] * right[None, :]), e
