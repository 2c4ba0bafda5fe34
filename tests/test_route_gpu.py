"""Routing to experts and its gradient, against 64-bit scores: the choice, the order by expert and
the rows that no slot takes are equal, weights and gradients within fp32's rounding."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import f8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# Scores: exp of a difference of logits (2^-24 of at most 40 between them, here), the sum of at
# most 1024 of them, a division: under 64 * 2^-24 in all; renormalised twice that.
REL = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def built():
    rtm.build()


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


def check(z, k, bias=None, align=1, **more):
    got = rtm.gemm_route(z, k, bias, align=align, **more)
    want = ref.route(z, k, bias, align=align, **more)
    for name, i in (("experts", 0), ("slots", 2), ("rows", 3), ("offsets", 4)):
        assert torch.equal(got[i], want[i]), name
    w = want[1]
    assert torch.equal(got[1].isnan(), w.isnan())
    off = (got[1].double() - w).abs().nan_to_num(0)
    assert (off <= REL * w.abs().nan_to_num(0) + 1e-37).all()
    return got


CASES = [(8, 2, 1, 1), (8, 8, 1, 1), (1, 1, 1, 1), (33, 5, 1, 1), (64, 6, 8, 3), (64, 32, 2, 2),
         (128, 8, 1, 1), (256, 8, 8, 4), (320, 8, 32, 6), (512, 10, 16, 1), (1000, 8, 8, 2),
         (1024, 32, 32, 32), (12, 3, 12, 3), (96, 4, 3, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,k,groups,top", CASES)
def test_choice_and_order(E, k, groups, top, biased, score):
    for T in (1, 37, 128, 129, 700):
        z = normal(T, E, seed=T + E)
        bias = normal(E, seed=E) * 0.05 if biased else None
        check(z, k, bias, score=score, groups=groups, top_groups=top, align=(1, 16, 128)[T % 3],
              renormalise=T % 2 == 0, scale=2.5 if T > 100 else 1.0)


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("groups,top,biased", [(1, 1, False), (4, 2, False), (1, 1, True)])
def test_types_and_equal_logits(type_, groups, top, biased):
    """16-bit logits collide often: the lower index goes first."""
    z = normal(300, 256, seed=3).to(TYPES[type_])
    bias = torch.zeros(256, device=DEV) if biased else None
    for score in ("softmax", "sigmoid"):
        check(z, 8, bias, score=score, groups=groups, top_groups=top)


def test_all_logits_equal():
    z = torch.zeros(200, 64, device=DEV)
    for more in ({}, {"groups": 8, "top_groups": 2}, {"bias": torch.zeros(64, device=DEV)}):
        experts = check(z, 6, align=128, **more)[0]
        assert torch.equal(experts, torch.arange(6, dtype=torch.int32, device=DEV).expand(200, 6))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_neighbours_that_32_bits_cannot_tell(score):
    """Scores + bias that lie nearer than fp32 resolves are ordered by 64 bits."""
    T, E = 400, 64
    z = normal(T, E, seed=9)
    s = ref.scores(z, score)
    # The bias of each expert (from token 0) brings all its sums next to each other.
    bias = (1.0 - s[0]).float()
    check(z[:1].contiguous(), 16, bias, score=score)
    check(z[:1].expand(200, E).contiguous(), 16, bias, score=score)
    check(z, 16, bias, score=score, groups=8, top_groups=3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(score):
    z = normal(260, 40, seed=1)
    z[0] = -torch.inf
    z[1, :38] = -torch.inf          # fewer left than are chosen
    z[2, 5] = torch.nan
    z[3] = torch.nan
    z[4] *= 60
    z[5, :] = torch.finfo(torch.float32).min
    z[6, :20] = torch.finfo(torch.float32).min
    z[130:, 7] = -torch.inf
    for more in ({}, {"groups": 4, "top_groups": 2}, {"bias": normal(40) * 0.1}):
        got = check(z, 4, score=score, **more)
        if score == "softmax":
            assert (got[1][0] == 0).all() and got[1][2].isnan().all() and got[1][3].isnan().all()


def test_bias_of_infinities():
    """An expert's bias of -inf takes it out, one of inf brings it in; weights stay the scores'."""
    z, bias = normal(150, 16, seed=2), torch.zeros(16, device=DEV)
    bias[3], bias[11] = -torch.inf, torch.inf
    experts, weights = check(z, 4, bias)[:2]
    assert not (experts == 3).any() and (experts[:, 0] == 11).all() and weights.isfinite().all()


def test_one_expert_takes_all_and_others_none():
    z = torch.zeros(1000, 32, device=DEV)
    z[:, 17] = 9
    got = check(z, 1, align=128)
    assert got[4][17] == 0 and got[4][18] == 1024 and (got[3][1000:] == -1).all()


def test_many_tokens():
    check(normal(40000, 60, seed=4), 4, align=128)
    check(normal(20011, 256, seed=5), 8, normal(256) * 0.05, score="sigmoid", groups=8,
          top_groups=4)


def test_no_tokens():
    experts, weights, slots, rows, offsets = rtm.gemm_route(torch.empty(0, 16, device=DEV), 2)
    assert experts.shape == weights.shape == slots.shape == (0, 2) and rows.numel() == 0
    assert offsets.shape == (17,) and not offsets.any()
    assert rtm.gemm_route_backward(torch.empty(0, 16, device=DEV), experts, weights).shape == (0, 16)


def test_a_logits_view_and_another_stream():
    z = normal(501, 64, seed=6)[1:]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rtm.gemm_route(z, 4, stream=side)
    side.synchronize()
    for a, b in zip(got, rtm.gemm_route(z, 4)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (40, 8), (128, 8), (500, 32), (1024, 7)])
def test_gradient(E, k, renormalise, score):
    for T, type_ in ((1, "f32"), (300, "f32"), (77, "bf16"), (77, "f16")):
        z, dw = normal(T, E, seed=E).to(TYPES[type_]), normal(T, k, seed=k)
        experts = rtm.gemm_route(z, k, score=score)[0]
        got = rtm.gemm_route_backward(z, experts, dw, score=score, renormalise=renormalise, scale=1.5)
        want = ref.route_backward(z, experts, dw, score, renormalise, 1.5)
        # dp_j is a difference of terms as large as dw and its weighted mean over the sum of the
        # chosen scores; each is off by at most REL, a few roundings and k additions.
        s = ref.scores(z, score)
        total = s.gather(1, experts.long()).sum(1, keepdim=True) if renormalise else 1.0
        size = 1.5 * dw.abs().double().amax(1, keepdim=True) / total
        tol = (3 * REL + k * 2.0 ** -23) * size * 2 * s
        assert ((got.double() - want).abs() <= tol + 1e-37).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(score):
    """The gradient of sum(weights * dw) along a direction, by central differences of the 64-bit
    definition: their error is h^2 / 6 of a third derivative of order 1."""
    z, dw, d = normal(20, 16, seed=1), normal(20, 3, seed=2), normal(20, 16, seed=3).double()
    experts = rtm.gemm_route(z, 3, score=score)[0]

    def loss(x):
        p = ref.scores(x, score).gather(1, experts.long())
        return (p / (p.sum(1, keepdim=True) + ref.NIL) * dw.double()).sum()

    h = 1e-4
    slope = (loss(z.double() + h * d) - loss(z.double() - h * d)) / (2 * h)
    got = (rtm.gemm_route_backward(z, experts, dw, score=score).double() * d).sum()
    assert abs(float(got - slope)) <= 1e-5 * float(dw.abs().sum() * d.abs().max())


def test_gradient_of_named_twice_outside_and_masked():
    z, dw = normal(4, 8, seed=1), normal(4, 3, seed=2)
    z[3] = -torch.inf
    experts = torch.tensor([[1, 1, 2], [0, 8, 3], [-1, 5, 6], [0, 1, 2]], dtype=torch.int32,
                           device=DEV)
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            got = rtm.gemm_route_backward(z, experts, dw, score=score, renormalise=renormalise)
            for t, used in enumerate(([0, 1, 2], [0, 2], [1, 2])):
                want = ref.route_backward(z[t:t + 1], experts[t:t + 1, used], dw[t:t + 1, used],
                                          score, renormalise)
                assert torch.allclose(got[t:t + 1].double(), want, rtol=1e-4, atol=1e-6)
            assert not got[3].any()


def test_refusals():
    z = normal(10, 16)
    experts, weights = rtm.gemm_route(z, 2)[:2]
    calls = [lambda: rtm.gemm_route(z, 0), lambda: rtm.gemm_route(z, 2.0), lambda: rtm.gemm_route(z, 33),
             lambda: rtm.gemm_route(z, True), lambda: rtm.gemm_route(z.double(), 2),
             lambda: rtm.gemm_route(z.t(), 2), lambda: rtm.gemm_route(z, 2, torch.zeros(15, device=DEV)),
             lambda: rtm.gemm_route(z, 2, torch.zeros(16, device=DEV).half()),
             lambda: rtm.gemm_route(z, 2, torch.zeros(16)), lambda: rtm.gemm_route(z, 2, score="tanh"),
             lambda: rtm.gemm_route(z, 2, align=0), lambda: rtm.gemm_route(z, 2, groups=33),
             lambda: rtm.gemm_route_backward(z, experts.long(), weights),
             lambda: rtm.gemm_route_backward(z, experts, weights.half()),
             lambda: rtm.gemm_route_backward(z, experts[:9], weights),
             lambda: rtm.gemm_route_backward(z, experts, weights, out=torch.empty(10, 15, device=DEV))]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    for call in (lambda: rtm.gemm_route(z, 17), lambda: rtm.gemm_route(z, 2, groups=3),
                 lambda: rtm.gemm_route(z, 2, groups=4, top_groups=5),
                 lambda: rtm.gemm_route(z, 5, groups=4, top_groups=1)):
        with pytest.raises(rtm.GemmError):
            call()
