"""A linear layer through its life with low-bit operands.

Training: Y = X.W in bf16 (gemm_bf16f32); the input is kept for the backward pass
in 8 bits (gemm_q8_quantize: half of what bf16 takes) and the weight gradient is
formed straight from it (gemm_q8tbf16f32). Serving: the trained weight is held in 4
bits (gemm_w4_quantize) and multiplies a prompt and then single tokens
(gemm_bf16w4f32).

    python examples/low_bit_linear.py [tokens inputs outputs steps]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import register_tiled_matrix_gb300 as rtm  # noqa: E402


class LowBitLinear:
    def __init__(self, inputs, outputs, device, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.master = torch.randn(inputs, outputs, generator=gen, device=device) * inputs ** -0.5
        self.saved = None
        self.served = None

    def forward(self, x):
        self.saved = rtm.gemm_q8_quantize(x)  # x itself need not outlive this call
        return rtm.gemm_bf16f32(x, self.master.to(torch.bfloat16))

    def backward(self, dy):
        """The weight's gradient (and the input's, which needs no saved activation)."""
        dw = rtm.gemm_q8tbf16f32(*self.saved, dy)
        dx = rtm.gemm_bf16f32(dy, self.master.to(torch.bfloat16).t().contiguous())
        self.saved = None
        return dx, dw

    def quantize(self, group=128):
        self.served = (*rtm.gemm_w4_quantize(self.master.to(torch.bfloat16), group), group)

    def serve(self, x):
        return rtm.gemm_bf16w4f32(x, *self.served)


def main(tokens=2048, inputs=1024, outputs=512, steps=30, device="cuda:0"):
    rtm.build()
    gen = torch.Generator(device=device).manual_seed(1)
    target = torch.randn(inputs, outputs, generator=gen, device=device) * inputs ** -0.5
    layer = LowBitLinear(inputs, outputs, device)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, inputs, generator=gen, device=device).to(torch.bfloat16)
        y = layer.forward(x)
        error = y - x.float() @ target
        losses.append(float(error.square().mean()))
        _, dw = layer.backward((error / tokens).to(torch.bfloat16))
        layer.master -= 0.5 * dw
    layer.quantize()
    prompt = torch.randn(100, inputs, generator=gen, device=device).to(torch.bfloat16)
    answer = layer.serve(prompt)
    token = layer.serve(prompt[-1:].contiguous())
    dense = prompt.float() @ layer.master
    away = float((answer - dense).norm() / dense.norm())
    apart = float((token - answer[-1:]).abs().max() / answer.abs().max())
    if rtm.get_device_error() != 0:
        raise RuntimeError("a bounded wait gave up")
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.6f}; served in 4 bits {away:.3f} from the dense layer; "
          f"token by token {apart:.1e} from the prompt's row")
    return losses, away, apart


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:]))
