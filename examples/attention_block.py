"""The attention block of an FP8 serving step, from the residual stream to the
residual stream, with this library's operators:

    fp8_linear_rmsnorm     norm + QKV projection
    fp8_kv_slots           pages and slots of the step's new tokens
    fp8_qk_norm_rope       norms and rotation of queries and keys, FP8 cache write
    fp8_attention_prompt   whole prompts, packed
    fp8_attention_decode   one new token a request over the paged cache, a shared
                           prefix read once
    fp8_linear             O projection

One layer at the 8B shapes (32 query heads on 8 key heads of 128) by default:
a system prompt is computed once, requests share its pages, and every request
gets a few new tokens.

    python examples/attention_block.py [--requests N] [--system T] [--steps S]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_w8a8_quantized_gb300 as fp8  # noqa: E402


class AttentionBlock:
    """One layer's weights, its part of the cache and the page pool."""

    def __init__(self, hidden=4096, q_heads=32, kv_heads=8, dim=128, pages=4096, page_size=16,
                 requests=64, table_width=256, norm=True, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device=device) * scale).to(torch.bfloat16)

        self.q_heads, self.kv_heads, self.dim, self.page_size = q_heads, kv_heads, dim, page_size
        self.gamma = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        qkv = normal((q_heads + 2 * kv_heads) * dim, hidden, scale=hidden ** -0.5)
        self.wqkv, self.s_qkv = fp8.fp8_quant_per_channel_weights(qkv)
        self.wo, self.s_o = fp8.fp8_quant_per_channel_weights(
            normal(hidden, q_heads * dim, scale=(q_heads * dim) ** -0.5))
        self.gamma_q = normal(dim, scale=0.1) + 1 if norm else None
        self.gamma_k = normal(dim, scale=0.1) + 1 if norm else None
        self.turns = fp8.fp8_rope_turns(rot_dim=dim, device=device)
        # scales of the cache: calibrated in earnest; here keys and values are of order 1
        self.k_scale = torch.full((kv_heads,), 8.0 / 448.0, device=device)
        self.v_scale = torch.full((kv_heads,), 8.0 / 448.0, device=device)
        shape = (pages * page_size, kv_heads, dim)
        self.k_cache = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.v_cache = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.free = torch.arange(pages, dtype=torch.int32, device=device)
        self.table = torch.full((requests, table_width), -1, dtype=torch.int32, device=device)
        self.ctx = torch.zeros(requests, dtype=torch.int32, device=device)

    def place(self, new_lens, tokens, rows=slice(None)):
        """Pages and slots for new_lens[b] new tokens of each request."""
        slots, positions, cu, lens, used = fp8.fp8_kv_slots(
            self.ctx[rows], new_lens, self.free, self.page_size, self.table[rows], tokens)
        taken = int(used)  # (pages come from the front of `free`: the host waits for their number)
        if taken > self.free.numel():
            raise RuntimeError(f"{taken} pages wanted, {self.free.numel()} free")
        self.free = self.free[taken:]
        self.ctx[rows] = lens
        return slots, positions, cu, lens

    def project(self, x, positions, slots, cache_only):
        """Norm, QKV projection, rotation and cache write: (q, k or None, v)."""
        qkv = fp8.fp8_linear_rmsnorm(x, self.gamma, 1e-6, self.wqkv, self.s_qkv)
        heads = qkv.view(x.shape[0], self.q_heads + 2 * self.kv_heads, self.dim)
        q, k, v = heads.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
        q, k = fp8.fp8_qk_norm_rope(
            q, k, positions, self.turns, gamma_q=self.gamma_q, gamma_k=self.gamma_k, v=v,
            k_scale=self.k_scale, v_scale=self.v_scale, slot_mapping=slots, k_cache=self.k_cache,
            v_cache=self.v_cache, cache_only=cache_only)
        return q, k, v

    def output(self, x, attended):
        return x + fp8.fp8_linear(attended.reshape(x.shape[0], -1), self.wo, self.s_o)

    def prompt(self, x, new_lens, rows=slice(None)):
        """Whole prompts x [T, hidden], packed, of requests without a context."""
        slots, positions, cu, _ = self.place(new_lens, x.shape[0], rows)
        q, k, v = self.project(x, positions, slots, cache_only=False)
        return self.output(x, fp8.fp8_attention_prompt(q, k, v, cu))

    def step(self, x, prefix_len=0):
        """One new token of each request, x [requests, hidden]."""
        one = torch.ones_like(self.ctx)
        slots, positions, _, lens = self.place(one, x.shape[0])
        q, _, _ = self.project(x, positions, slots, cache_only=True)
        attended = fp8.fp8_attention_decode(q, self.k_cache, self.v_cache, self.k_scale, self.v_scale,
                                            self.table, lens, self.page_size, prefix_len=prefix_len)
        return self.output(x, attended)

    def share(self, tokens):
        """Gives every request the pages of request 0's first `tokens` tokens
        (whole pages) as its own beginning; returns how many that are."""
        pages = tokens // self.page_size
        self.table[1:, :pages] = self.table[:1, :pages]
        self.table[:, pages:] = -1
        self.ctx.fill_(pages * self.page_size)
        return pages * self.page_size


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--system", type=int, default=2048, help="tokens of the shared system prompt")
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    width = (a.system + a.steps) // 16 + 2
    block = AttentionBlock(requests=a.requests, pages=a.system // 16 + a.requests * (a.steps // 16 + 2) + 8,
                           table_width=width)
    x = torch.randn(a.system, 4096, device="cuda").to(torch.bfloat16)
    y = block.prompt(x, torch.tensor([a.system], dtype=torch.int32, device="cuda"), slice(0, 1))
    shared = block.share(a.system)
    print(f"system prompt: {a.system} tokens, output rms {y.float().square().mean().sqrt():.3f}, "
          f"{shared} of them shared by {a.requests} requests")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        x = torch.randn(a.requests, 4096, device="cuda").to(torch.bfloat16)
        begin.record()
        y = block.step(x, prefix_len=shared)
        end.record()
        torch.cuda.synchronize()
        print(f"step {i}: {a.requests} tokens, context {int(block.ctx[0])}, "
              f"output rms {y.float().square().mean().sqrt():.3f}, {begin.elapsed_time(end) * 1e3:.0f} us")
    assert fp8.fp8_device_status() == fp8.FP8_OK


if __name__ == "__main__":
    main()
