"""A layer of experts with 8-bit floating-point operands, trained and served.

Each token goes to `k` of `E` experts, a matrix each: the router's logits choose them
(gemm_route), the tokens' rows are gathered into the experts' order as they are taken to 8 bits
(gemm_f8_quantize), each expert multiplies its rows (gemm_f8w8f32_experts), and a token's parts
are summed by their weights (gemm_experts_join). The backward pass runs the same way: the
gradient is gathered, weighted and taken to 8 bits along both axes at once, and feeds both the
input's and the weights' gradients. Master weights stay in fp32 and are taken to 8 bits each step.

    python examples/f8_experts.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import register_tiled_matrix_gb300 as rtm  # noqa: E402


def forward(x, router, experts, k, align=128):
    """y (T x N) of tokens x (T x K, bf16); router K x E and experts E x K x N in fp32. Returns y
    and what the backward pass needs. A serving program passes align=1: the shortest order."""
    logits = rtm.gemm_bf16f32(x, router.bfloat16())
    chosen, weights, slots, rows, offsets = rtm.gemm_route(logits, k, align=align)
    a, a_scales, columns, column_scales = rtm.gemm_f8_quantize(x, "both", gather=rows, fan=k)
    w, w_scales = rtm.gemm_f8_quantize_tiles(experts)
    parts = rtm.gemm_f8w8f32_experts(a, a_scales, w, w_scales, offsets)
    y = rtm.gemm_experts_join(parts, slots, weights)
    return y, (x, logits, chosen, weights, slots, rows, offsets, columns, column_scales, w,
               w_scales, parts, k)


def backward(dy, saved):
    """(d router, d experts, dx) of the gradient dy (T x N, fp32)."""
    (x, logits, chosen, weights, slots, rows, offsets, columns, column_scales, w, w_scales, parts,
     k) = saved
    d, d_scales, dc, dc_scales = rtm.gemm_f8_quantize(dy, "both", gather=rows, fan=k,
                                                      factors=weights)
    d_experts = rtm.gemm_f8tf8f32_experts(columns, column_scales, dc, dc_scales, offsets)
    dx = rtm.gemm_experts_join(rtm.gemm_f8w8tf32_experts(d, d_scales, w, w_scales, offsets), slots)
    d_weights = rtm.gemm_experts_join_backward(dy, parts, slots)
    d_logits = rtm.gemm_route_backward(logits, chosen, d_weights)
    d_router = rtm.gemm_f32(x.float().t().contiguous(), d_logits)
    return d_router, d_experts, dx


def main(steps=20, T=1024, K=256, N=256, E=8, k=2, seed=0):
    """Trains the layer towards a fixed linear map; returns the losses and a decoded token's y."""
    rtm.build()
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    target, router = normal(K, N) / K ** 0.5, normal(K, E) * 0.1
    experts, losses = normal(E, K, N) * 0.02, []
    for _ in range(steps):
        x = normal(T, K).bfloat16()
        y, saved = forward(x, router, experts, k)
        off = y - rtm.gemm_f32(x.float(), target)
        losses.append(off.square().mean())
        d_router, d_experts, _ = backward(off * (2 / off.numel()), saved)
        router -= 20.0 * d_router
        experts -= 200.0 * d_experts
    token = forward(normal(1, K).bfloat16(), router, experts, k, align=1)[0]
    return [float(v) for v in losses], token


if __name__ == "__main__":
    losses, token = main()
    for i, v in enumerate(losses):
        print(f"step {i}: loss {v:.4f}")
    print(f"one token: {token.shape[1]} values, finite: {bool(token.isfinite().all())}")
