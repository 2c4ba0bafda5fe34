"""8-bit floating-point products of whole numbers whose sums of magnitudes stay below 2^24: every
partial sum, in whatever order, is a whole number that fp32 holds, so results have to be equal. A
sum that is kept in fewer than 24 bits anywhere would show."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests.test_f8_products_gpu import CALLS, blocks

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    rtm.build()
    yield
    torch.cuda.synchronize()
    assert rtm.get_device_error() == 0


def whole(rows, cols, high, gen, signed):
    """e4m3 whole numbers up to `high`."""
    v = torch.arange(high + 1, device=DEV).float()
    v = v[v.to(F8).float() == v]
    x = v[torch.randint(0, len(v), (rows, cols), generator=gen, device=DEV)]
    if signed:
        x = x * (2.0 * torch.randint(0, 2, (rows, cols), generator=gen, device=DEV) - 1)
    held = torch.zeros(rows, (cols + 15) // 16 * 16, device=DEV)
    held[:, :cols] = x
    return held.to(F8)[:, :cols]


@pytest.mark.parametrize("direction", CALLS)
@pytest.mark.parametrize("M,N,K", [(1, 500, 1000), (16, 300, 1000), (33, 700, 520), (64, 256, 1000),
                                   (100, 400, 1000), (300, 200, 1000), (2000, 2100, 1000),
                                   (1000, 130, 2100), (900, 4000, 3900)])
@pytest.mark.parametrize("signed", [False, True])
def test_whole_numbers(M, N, K, signed, direction):
    gen = torch.Generator(DEV).manual_seed(M + N)
    shapes = {"forward": ((M, K), (K, N)), "input": ((M, N), (K, N)), "weight": ((M, K), (M, N))}
    a, b = shapes[direction]
    depth = {"forward": K, "input": N, "weight": M}[direction]
    high = int(((2 ** 24 - 1) / depth) ** 0.5)
    high = min(high, 448)
    assert depth * high * high < 2 ** 24
    A, B = whole(*a, high, gen, signed), whole(*b, high, gen, signed)
    ones = {"forward": ((M, blocks(K)), (blocks(K), blocks(N))),
            "input": ((M, blocks(N)), (blocks(K), blocks(N))),
            "weight": ((blocks(M), K), (blocks(M), N))}[direction]
    got = CALLS[direction](A, torch.ones(ones[0], device=DEV), B, torch.ones(ones[1], device=DEV))
    left, right = A.double(), B.double()
    want = {"forward": lambda: left @ right, "input": lambda: left @ right.t(),
            "weight": lambda: left.t() @ right}[direction]()
    assert torch.equal(got.double(), want)
