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


# ---- renormalised weights
def renormalised(z, experts, dw, score, scale):
    """(dlogits, what its terms' magnitudes add up to) in 64 bits, all but NIL sums of differences."""
    at, dw = experts.long(), dw.double()
    s = ref.scores(z, score)
    p = s.gather(1, at)
    total = p.sum(1, keepdim=True) + ref.NIL
    between = dw[:, :, None] - dw[:, None, :]
    g = ((p[:, None, :] * between).sum(2) + ref.NIL * dw) * scale / total ** 2
    size = ((p[:, None, :] * between.abs()).sum(2) + ref.NIL * dw.abs()) * scale / total ** 2
    if score == "sigmoid":
        slope = p * torch.sigmoid(-z.double().gather(1, at))
        zero = torch.zeros_like(s)
        return zero.scatter(1, at, g * slope), zero.scatter(1, at, size * slope)
    inner = scale * ref.NIL * (p * dw).sum(1, keepdim=True) / total ** 2
    bound = scale * ref.NIL * (p * dw.abs()).sum(1, keepdim=True) / total ** 2
    return (s * (torch.zeros_like(s).scatter(1, at, g) - inner),
            s * (torch.zeros_like(s).scatter(1, at, size) + bound))


# A score is within 2^-18 of itself: the exponent's rounding, 2^-24 of the at most 32 between two
# logits (2^-19; a sigmoid's is 2^-21), exp's 2^-22, and of a softmax the sum of 2 additions in a
# lane, 5 across lanes and a division, 8 * 2^-24. dlogits has it four times (its own, that of the
# sum, twice that of S). The sum of differences may be made of differences from one dw, that of the
# largest score: these are at most 2 k + 1 times the terms, with 8 roundings each; and 12 more.
def tolerance(k):
    return 2.0 ** -16 + (8 * (2 * k + 1) + 12) * 2.0 ** -24


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 2, 8, 32])
@pytest.mark.parametrize("spread", [1, 4])
@pytest.mark.parametrize("alike", [False, True])
def test_renormalised(alike, spread, k, score):
    """`alike`: all of a token's dweights are equal, so that only NIL moves its weights."""
    z = normal(400, 64, seed=k) * spread
    dw = normal(400, 1, seed=3).expand(400, k).contiguous() if alike else normal(400, k, seed=3)
    experts = rtm.gemm_route(z, k, score=score)[0]
    got = rtm.gemm_route_backward(z, experts, dw, score=score, scale=1.5).double()
    want, size = renormalised(z, experts, dw, score, 1.5)
    assert ((got - want).abs() <= tolerance(k) * size + 1e-37).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_renormalised_scores_as_small_as_what_keeps_them_from_0(score):
    """Chosen scores of 1e-16 to 1e-24 (one expert, that is not chosen, has the softmax): S is
    1e-20 and they together, and the gradient is not small."""
    z = uniform(-55, -37, 200, 16, seed=4)
    z[:, 0] = 0.0
    experts = torch.tensor([[3, 9, 5]], dtype=torch.int32, device=DEV).expand(200, 3).contiguous()
    dw = normal(200, 3, seed=6)
    got = rtm.gemm_route_backward(z, experts, dw, score=score).double()
    want, size = renormalised(z, experts, dw, score, 1.0)
    assert ((got - want).abs() <= 2 * tolerance(3) * size + 1e-37).all()  # the exponents are twice as large
    assert float(want.abs().max()) > 1e-3


# ---- softmax without renormalisation, where one score is nearly 1
def plain_softmax(z, experts, dw, scale):
    """(dlogits, what its terms' magnitudes add up to) in 64 bits, as sums of differences."""
    at = experts.long()
    s = ref.scores(z, "softmax")
    g = torch.zeros_like(s).scatter_add(1, at, scale * dw.double())
    between = g.gather(1, at)[:, :, None] - g[:, None, :]  # an expert's g less each other's
    p = s.gather(1, at)
    inner = (s * g).sum(1, keepdim=True)
    bound = (s * torch.zeros_like(s).scatter_add(1, at, scale * dw.double().abs())).sum(1, keepdim=True)
    return ((-s * inner).scatter(1, at, p * (s[:, None, :] * between).sum(2)),
            (s * bound).scatter(1, at, p * (s[:, None, :] * between.abs()).sum(2)))


# Two scores have 2 * 2^-18, as above; differences from one g are at most 2 k + 3 times the terms
# (the experts that are not chosen count as one), with 8 roundings each: below tolerance(k).
@pytest.mark.parametrize("k", [1, 2, 8, 32])
@pytest.mark.parametrize("lead", [0, 8, 15])
def test_a_softmax_score_near_1(lead, k):
    z, dw = normal(300, 100, seed=k), normal(300, k, seed=lead)
    z[torch.arange(300, device=DEV), torch.arange(300, device=DEV) % 100] += lead
    experts = rtm.gemm_route(z, k)[0]
    got = rtm.gemm_route_backward(z, experts, dw, renormalise=False, scale=1.5).double()
    want, size = plain_softmax(z, experts, dw, 1.5)
    off = (got - want).abs() - tolerance(k) * size
    assert (off <= 1e-37).all()


def test_named_twice_and_outside_beside_a_score_near_1():
    z, dw = normal(100, 8, seed=1), normal(100, 4, seed=2)
    z[:, 1] += 14
    experts = torch.tensor([[1, 1, 2, 8]], dtype=torch.int32, device=DEV).expand(100, 4).contiguous()
    got = rtm.gemm_route_backward(z, experts, dw, renormalise=False).double()
    want, size = plain_softmax(z, experts[:, :3], dw[:, :3], 1.0)
    assert ((got - want).abs() <= tolerance(3) * size + 1e-37).all()


def test_a_softmax_score_near_1_against_differences():
    """One expert chosen: its weight's slope by its own logit is that of the others' scores, which
    keep their digits. A step of 2^-6: the error is step^2 / 6 and 2^-50 of the scores."""
    z = normal(60, 16, seed=8)
    z[:, 4] += 12
    experts = rtm.gemm_route(z, 1)[0]
    assert (experts == 4).all()
    got = rtm.gemm_route_backward(z, experts, torch.ones(60, 1, device=DEV), renormalise=False)
    h, step = 2.0 ** -6, torch.zeros(16, device=DEV, dtype=torch.float64)
    step[4] = h
    others = [None, None]
    for i, x in enumerate((z.double() - step, z.double() + step)):
        s = torch.softmax(x, 1)
        others[i] = torch.cat((s[:, :4], s[:, 5:]), 1).sum(1)
    slope = (others[0] - others[1]) / (2 * h)
    off = (got[:, 4].double() - slope).abs()
    assert (off <= (h * h / 6 + 2.0 ** -16 + 2.0 ** -50 / h) * slope).all()
