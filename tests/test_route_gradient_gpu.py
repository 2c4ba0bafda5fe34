"""The gradient of routing where a score is close to 1, or the weights hardly move: dlogits are
within fp32's rounding of what they are, however small, against the formula in 64 bits (written
without differences of nearly equal numbers) and against differences."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import f8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    rtm.build()


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def uniform(low, high, *shape, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return low + (high - low) * torch.rand(*shape, generator=gen, device=DEV)


# ---- a sigmoid's s * (1 - s)
# s and 1 - s each: exp within 2 units in the last place (2^-22), a rounding of 1 + exp (2^-24) and
# a division within 2 units (2^-22); then three products: 2 * (2^-21 + 2^-24) + 3 * 2^-24 < 2^-19.
@pytest.mark.parametrize("type_", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("low,high", [(10, 20), (-20, -10), (-80, 80), (-4, 4)])
def test_sigmoids_near_0_and_1(low, high, type_):
    z, dw = uniform(low, high, 300, 64, seed=1).to(type_), normal(300, 6, seed=2)
    experts = rtm.gemm_route(z, 6, score="sigmoid")[0]
    got = rtm.gemm_route_backward(z, experts, dw, score="sigmoid", renormalise=False, scale=1.5)
    x = z.double().gather(1, experts.long())
    want = 1.5 * dw.double() * torch.sigmoid(x) * torch.sigmoid(-x)
    off = (got.double().gather(1, experts.long()) - want).abs()
    assert (off <= 2.0 ** -19 * want.abs() + 1e-37).all(), float((off / want.abs()).max())
    assert int((got != 0).sum()) <= experts.numel()  # and nothing elsewhere


def test_sigmoids_near_1_against_differences():
    """Central differences of sum(weights * dw) by each logit: a step of 2^-6 is exact, the error of
    the difference step^2 / 6 (of a derivative as large as the gradient) and 2^-52 of s / step."""
    z = uniform(6, 14, 40, 8, seed=5)
    dw = torch.ones(40, 1, device=DEV)
    experts = rtm.gemm_route(z, 1, score="sigmoid")[0]
    got = rtm.gemm_route_backward(z, experts, dw, score="sigmoid", renormalise=False)
    x, h = z.double().gather(1, experts.long()), 2.0 ** -6
    # 1 - s is a sigmoid too, and keeps its digits
    slope = (torch.sigmoid(-(x - h)) - torch.sigmoid(-(x + h))) / (2 * h)
    off = (got.double().gather(1, experts.long()) - slope).abs()
    assert (off <= (h * h / 6 + 2.0 ** -18) * slope + 2.0 ** -50 / h * torch.sigmoid(-x)).all()
