"""The feed-forward half of an FP8 serving step whose layer is split into experts,
from the attention block's output to the next layer's FP8 input, with this
library's operators:

    fp8_residual_norm_quant  attention's output joined with the residual stream, norm
    fp8_moe_route            each token's experts, rows sorted by expert
    fp8_grouped_linear       gate and values of each expert's rows, gated activation
    fp8_grouped_linear       the experts' second product
    fp8_residual_norm_quant  rows of a token summed by weight, joined, the next norm, codes

One layer at the 8B widths (4096 in, 14336 inside) with eight experts by default.

    python examples/expert_block.py [--tokens T] [--experts E] [--top K] [--steps S]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_w8a8_quantized_gb300 as fp8  # noqa: E402


class ExpertBlock:
    """One layer's router, experts and norms."""

    def __init__(self, hidden=4096, inner=14336, experts=8, top=2, post_norm=False, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(torch.bfloat16)

        def expert_weights(rows, width):
            wq = torch.empty(experts, rows, width, dtype=torch.uint8, device=device)
            s_w = torch.empty(experts, rows, device=device)
            for e in range(experts):
                fp8.fp8_quant_per_channel_weights(normal(rows, width, scale=width ** -0.5), wq=wq[e], s_w=s_w[e])
            return wq, s_w

        self.top = top
        self.router = normal(experts, hidden, scale=hidden ** -0.5)
        self.w_in, self.s_in = expert_weights(2 * inner, hidden)  # the gate's rows, then the values'
        self.w_out, self.s_out = expert_weights(hidden, inner)
        self.gamma = normal(hidden, scale=0.1) + 1
        self.gamma_next = normal(hidden, scale=0.1) + 1
        self.gamma_post = normal(hidden, scale=0.1) + 1 if post_norm else None

    def experts(self, z):
        """The experts' rows of tokens z [T, hidden], and where each token's lie."""
        ids, weights, offsets, row_token, token_row = fp8.fp8_moe_route(z @ self.router.t(), self.top)
        inner = fp8.fp8_grouped_linear(z, self.w_in, self.s_in, offsets, row_token=row_token, swiglu=True)
        return fp8.fp8_grouped_linear(inner, self.w_out, self.s_out, offsets), token_row, weights

    def forward(self, h, attended):
        """(residual stream, the next layer's codes, their scales) of the stream h and
        the attention block's output."""
        h, z, _, _ = fp8.fp8_residual_norm_quant(h, attended, self.gamma, codes=False)
        rows, token_row, weights = self.experts(z)
        h, _, codes, scales = fp8.fp8_residual_norm_quant(h, rows, self.gamma_next, gamma_post=self.gamma_post,
                                                          token_row=token_row, weights=weights, rows=False)
        return h, codes, scales


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--top", type=int, default=2)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    block = ExpertBlock(experts=a.experts, top=a.top)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        h = torch.randn(a.tokens, 4096, device="cuda").to(torch.bfloat16)
        attended = torch.randn(a.tokens, 4096, device="cuda").to(torch.bfloat16)
        begin.record()
        h, codes, scales = block.forward(h, attended)
        end.record()
        torch.cuda.synchronize()
        print(f"step {i}: {a.tokens} tokens, stream rms {h.float().square().mean().sqrt():.3f}, "
              f"{begin.elapsed_time(end) * 1e3:.0f} us")
    assert fp8.fp8_device_status() == fp8.FP8_OK


if __name__ == "__main__":
    main()
