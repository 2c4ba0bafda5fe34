"""8-bit floating-point products whose offsets pass 32 bits. Scales are powers of two and sums have
one term or few, so outputs have to be equal."""

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
