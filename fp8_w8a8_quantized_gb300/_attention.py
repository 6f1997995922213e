"""Binding of the attention block's calls (include/fp8w8a8.h): slot maps, norms
and rotation of queries and keys, prompt attention and decode attention over
the paged FP8 cache.  Checks of arguments (ValueError) and allocations are the
extension module's (csrc/attention_binding.cpp, built beside the library); a
status of the library becomes Fp8Error.  Without the module the calls raise."""
from __future__ import annotations

import importlib.machinery
import importlib.util
import math
import os

import torch

from ._binding import _HERE, Fp8Error, _lock, lib

MODULE_PATH = os.path.join(_HERE, "_build", "fp8_attention_binding"
                           + importlib.machinery.EXTENSION_SUFFIXES[0])
_module = None


def _native():
    """The loaded extension module."""
    global _module
    if _module is None:
        lib()  # the library that the module links to
        if not os.path.exists(MODULE_PATH):
            raise RuntimeError(f"binding module not built ({MODULE_PATH}); run "
                               "`python -m fp8_w8a8_quantized_gb300.build`")
        with _lock:
            if _module is None:
                spec = importlib.util.spec_from_file_location("fp8_attention_binding", MODULE_PATH)
                module = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(module)
                _module = module
    return _module


def _handle(stream):
    """None, or the raw handle of a given stream."""
    return getattr(stream, "cuda_stream", stream)


def _result(r, what: str):
    if type(r) is int:
        raise Fp8Error(r, what)
    return r


def fp8_kv_slots(ctx_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                 page_size: int, block_table: torch.Tensor, max_tokens: int,
                 slot_mapping: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                 cu_seqlens: torch.Tensor | None = None, seq_lens: torch.Tensor | None = None,
                 pages_used: torch.Tensor | None = None, stream=None):
    """Gives the new tokens of each request their pages and slots: takes pages
    from the front of free_pages (int32) into block_table (int32 [B, width],
    in place) and returns (slot_mapping int64 [max_tokens], positions int32
    [max_tokens], cu_seqlens int32 [B + 1], seq_lens int32 [B], pages_used
    int32 [1]); where none of them is given, the five share one allocation."""
    return _result((_module or _native()).kv_slots(
        ctx_lens, new_lens, free_pages, page_size, block_table, max_tokens, slot_mapping, positions,
        cu_seqlens, seq_lens, pages_used, _handle(stream)), "fp8_kv_slots")


def fp8_rope_turns(theta: float = 500000.0, rot_dim: int = 128, inv_freq=None,
                   device="cuda") -> torch.Tensor:
    """The rotation's plan for fp8_qk_norm_rope: the frequency of each of the
    rot_dim / 2 pairs as a 64-bit fraction of a turn per position (int64 bits).
    Frequencies are theta^(-2 i / rot_dim) radians, or `inv_freq`'s."""
    if inv_freq is None:
        inv_freq = [theta ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    turns = []
    for f in (inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else inv_freq):
        n = int(math.fmod(float(f) / (2.0 * math.pi), 1.0) * 2.0 ** 64) % (1 << 64)
        turns.append(n - (1 << 64) if n >= 1 << 63 else n)
    return torch.tensor(turns, dtype=torch.int64, device=device)


def fp8_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor,
                     turns: torch.Tensor, gamma_q: torch.Tensor | None = None,
                     gamma_k: torch.Tensor | None = None, eps: float = 1e-6,
                     interleaved: bool = False, q_out: torch.Tensor | None = None,
                     k_out: torch.Tensor | None = None, v: torch.Tensor | None = None,
                     k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                     slot_mapping: torch.Tensor | None = None,
                     k_cache: torch.Tensor | None = None, v_cache: torch.Tensor | None = None,
                     cache_only: bool = False, stream=None):
    """Norm (where a gamma is given) and rotation of each head of q [T, Hq, D]
    and k [T, Hkv, D] (bf16, views into a fused projection will do); with
    caches also the FP8 cache write of the rotated keys and of v.  turns:
    fp8_rope_turns().  Returns (q_out, k_out); q_out=q, k_out=k work in place;
    cache_only leaves k_out out (None)."""
    return _result((_module or _native()).qk_norm_rope(
        q, k, positions, turns, gamma_q, gamma_k, eps, interleaved, q_out, k_out, v, k_scale, v_scale,
        slot_mapping, k_cache, v_cache, cache_only, _handle(stream)), "fp8_qk_norm_rope")


def fp8_attention_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         cu_seqlens: torch.Tensor, scale: float | None = None,
                         out: torch.Tensor | None = None, stream=None):
    """Causal attention over prompts packed one after the other: q [T, Hq, D],
    k and v [T, Hkv, D] bf16 (views into a fused projection will do), sequence
    s in tokens cu_seqlens[s] .. cu_seqlens[s + 1] - 1 -> bf16 [T, Hq, D].
    Tokens outside every sequence get no output.  scale: 1 / sqrt(D) unless
    given."""
    return _result((_module or _native()).attention_prompt(q, k, v, cu_seqlens, scale, out,
                                                           _handle(stream)), "fp8_attention_prompt")


def fp8_attention_decode_workspace_size(B: int, Hq: int, Hkv: int, D: int, table_width: int,
                                        page_size: int, prefix_len: int = 0) -> int:
    return int(lib().fp8_attention_decode_workspace_size(B, Hq, Hkv, D, table_width, page_size,
                                                         prefix_len))


def fp8_attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         k_scale: torch.Tensor, v_scale: torch.Tensor, block_table: torch.Tensor,
                         seq_lens: torch.Tensor, page_size: int, prefix_len: int = 0,
                         scale: float | None = None, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None):
    """Attention of one new token per request, q [B, Hq, D] bf16, over the paged
    FP8 cache (codes uint8 [slots, Hkv, D]; scales fp32, one a head or one in
    all): request b's token j lies in slot block_table[b, j // page_size] *
    page_size + j % page_size, j < seq_lens[b].  The first prefix_len tokens,
    which all requests share, are read once, from the pages of table row 0.
    Returns bf16 [B, Hq, D], zeros for a request without tokens."""
    return _result((_module or _native()).attention_decode(
        q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, page_size, prefix_len, scale, out,
        workspace, _handle(stream)), "fp8_attention_decode")
