"""Routing by groups with biases of large magnitude and mixed sign: the choice is the one of 64-bit
scores, although such biases cancel in a group's sum and their roundings do not."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import f8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    rtm.build()


def check(z, k, bias, score, groups, top):
    got = rtm.gemm_route(z, k, bias, score=score, groups=groups, top_groups=top, align=1)
    want = ref.route(z, k, bias, score=score, groups=groups, top_groups=top, align=1)
    wrong = (got[0] != want[0]).any(1)
    assert not wrong.any(), f"{int(wrong.sum())} of {len(z)} tokens"
    for a, b in zip(got[2:], want[2:]):
        assert torch.equal(a, b)


def test_opposite_biases_of_one_group():
    """The sums are 0.8751469 and 0.8751490; 32 bits have 0.8751526 for the first."""
    z = torch.tensor([[-0.59536892, 0.07901291, 1.37114227, -2.47562957]], device=DEV)
    bias = torch.tensor([64.0, -64.0, 0.0, 0.0], device=DEV)
    check(z, 2, bias, "sigmoid", 2, 1)
    assert rtm.gemm_route(z, 2, bias, score="sigmoid", groups=2)[0].tolist() == [[2, 3]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B", [1.0, 16.0, 64.0, 1000.0])
@pytest.mark.parametrize("groups,size,top", [(2, 2, 1), (8, 2, 4), (4, 4, 2), (32, 8, 5)])
def test_sums_nearer_than_their_members_round(groups, size, top, B, score):
    """A group's two best have a bias of B and of -B (odd groups: of 0), its others one that keeps
    them out; all groups' sums lie within some units of 32 bits' rounding at 64."""
    T, gen = 3000, torch.Generator(device=DEV).manual_seed(groups + size)

    def uniform(low, high, *shape):
        return low + (high - low) * torch.rand(*shape, generator=gen, device=DEV, dtype=torch.float64)

    one, two = uniform(0.3, 0.6, T, 1), uniform(0.3, 0.6, T, 1)
    shift, off = uniform(-0.1, 0.1, T, groups), uniform(-2e-5, 2e-5, T, groups)
    s = uniform(0.05, 0.1, T, groups, size)
    s[..., 0], s[..., 1] = one + shift, two - shift + off
    s = s.view(T, -1)
    z = (s.log() if score == "softmax" else (s / (1 - s)).log()).float()
    bias = torch.zeros(groups, size, device=DEV)
    bias[::2, 0], bias[::2, 1], bias[:, 2:] = B, -B, -4 * B
    check(z, 2, bias.flatten(), score, groups, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("B", [16.0, 1000.0])
def test_random_biases(B, score):
    gen = torch.Generator(device=DEV).manual_seed(int(B))
    for E, groups, top, k in ((16, 8, 3, 3), (64, 16, 4, 6), (256, 8, 4, 8), (24, 12, 6, 4)):
        z = torch.randn(2000, E, generator=gen, device=DEV)
        bias = torch.randn(E, generator=gen, device=DEV) * B
        check(z, k, bias, score, groups, top)
