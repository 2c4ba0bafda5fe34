"""The example of a layer of experts: it runs, and its gradients are those of the values that its
operands are held as, by autograd in 64 bits."""

import os
import sys

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import f8_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import f8_experts  # noqa: E402

pytestmark = pytest.mark.gpu


def test_runs():
    losses, token = f8_experts.main(steps=3, T=200, K=96, N=80)
    assert len(losses) == 3 and torch.tensor(losses).isfinite().all()
    assert token.shape == (1, 80) and token.isfinite().all()


def test_gradients():
    rtm.build()
    T, K, N, E, k = 150, 130, 70, 6, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    router = torch.randn(K, E, generator=g, device="cuda") * 0.2
    experts = torch.randn(E, K, N, generator=g, device="cuda") * 0.1
    dy = torch.randn(T, N, generator=g, device="cuda")
    y, saved = f8_experts.forward(x, router, experts, k)
    d_router, d_experts, dx = f8_experts.backward(dy, saved)

    # The layer in 64 bits at the same choice of experts.
    chosen = saved[2].long()
    xs, rs, es = (t.double().requires_grad_(True) for t in (x, router.bfloat16(), experts))
    s = torch.softmax(xs @ rs, 1).gather(1, chosen)
    w = s / s.sum(1, keepdim=True)
    parts = torch.einsum("tk,tjkn->tjn", xs, es[chosen])
    want = (w[..., None] * parts).sum(1)
    got = torch.autograd.grad((want * dy.double()).sum(), (rs, es))
    dx_want = torch.einsum("tj,tn,tjkn->tk", w, dy.double(), es[chosen]).detach()

    # Each operand is off by half a step of its codes, 2^-4 of a value, or where it is far below
    # its block's largest by half the least step, 2^-10 of 2^-8 to 2^-7 of that: 2 * 2^-4 and a
    # bit of the sums of magnitudes covers two such operands.
    def near(a, b, size):
        assert (a.double() - b).abs().le(0.14 * size + 1e-3 * size.max()).all()

    ax, ae, ad = xs.detach().abs(), es.detach().abs(), dy.double().abs()
    wd = w.detach()
    near(y, want.detach(), torch.einsum("tj,tk,tjkn->tn", wd, ax, ae[chosen]))
    near(dx, dx_want, torch.einsum("tj,tn,tjkn->tk", wd, ad, ae[chosen]))
    size = torch.zeros_like(ae)
    for j in range(k):
        size.index_add_(0, chosen[:, j], wd[:, j, None, None] * ax[:, :, None] * ad[:, None, :])
    near(d_experts, got[1], size)
    # The router's gradient goes through the products as they were rounded.
    dw = (dy.double()[:, None] * saved[11].double()[saved[4].long()]).sum(-1)
    dz = ref.route_backward(saved[1], saved[2], dw)
    assert torch.allclose(d_router.double(), x.double().t() @ dz, rtol=1e-4,
                          atol=1e-4 * float(dz.abs().sum(0).max()))
