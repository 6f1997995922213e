"""ctypes binding of the attention block's calls (include/fp8w8a8.h): slot
maps, norms and rotation of queries and keys, prompt attention and decode
attention over the paged FP8 cache.  As in the layer's binding every tensor's
device, dtype, shape and layout is checked before the C call (ValueError), and
the library checks the rest (Fp8Error)."""
from __future__ import annotations

import math

import torch

from ._binding import _check, _expect, _ptr, _stream, _workspace, lib


def _tokens(t, name: str, shape=None):
    """The token stride of a bf16 [tokens, heads, D] CUDA tensor whose heads
    are contiguous within a token (a view into a wider projection will do)."""
    if (not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda
            or t.dim() != 3 or (shape is not None and tuple(t.shape) != shape)):
        got = (f"{t.dtype} {tuple(t.shape)} on {t.device}" if isinstance(t, torch.Tensor)
               else type(t).__name__)
        raise ValueError(f"{name} must be a CUDA torch.bfloat16 tensor of shape "
                         f"{shape or '[tokens, heads, D]'}; got {got}")
    n, h, d = t.shape
    ld, sh, sd = t.stride()
    if t.numel() and ((d > 1 and sd != 1) or (h > 1 and sh != d)):
        raise ValueError(f"{name} must have the heads of a token contiguous; got strides {t.stride()}")
    return ld if n > 1 else h * d


def _empty(shape, dtype, device, stream):
    """A new tensor in the memory of the stream that the call runs on: where
    the caller lets go of it, nothing but later work of that stream gets it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _fresh(t, name: str, shape, like, stream):
    """`t` or a new contiguous tensor of that shape, and its token stride."""
    if t is None:
        return _empty(shape, torch.bfloat16, like.device, stream), shape[1] * shape[2]
    return t, _tokens(t, name, shape)


def _scales(t, name: str, heads: int) -> int:
    """The scale stride: 1 for one scale a head, 0 for one in all."""
    if isinstance(t, torch.Tensor) and t.numel() == 1:
        _expect(t, name, t.shape, torch.float32)
        return 0
    _expect(t, name, (heads,), torch.float32)
    return 1


def _cache(k_cache, v_cache, heads: int, dim: int) -> int:
    slots = k_cache.shape[0] if isinstance(k_cache, torch.Tensor) and k_cache.dim() == 3 else 0
    _expect(k_cache, "k_cache", (slots, heads, dim), torch.uint8)
    _expect(v_cache, "v_cache", (slots, heads, dim), torch.uint8)
    return slots


def _table(t, rows: int):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("block_table must be a 2-D CUDA int32 tensor")
    _expect(t, "block_table", (rows, t.shape[1]), torch.int32, contiguous=False)
    return t.shape[1], (t.stride(0) if rows > 1 else t.shape[1])


def fp8_kv_slots(ctx_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                 page_size: int, block_table: torch.Tensor, max_tokens: int,
                 slot_mapping: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                 cu_seqlens: torch.Tensor | None = None, seq_lens: torch.Tensor | None = None,
                 pages_used: torch.Tensor | None = None, stream=None):
    """Gives the new tokens of each request their pages and slots: takes pages
    from the front of free_pages (int32) into block_table (int32 [B, width],
    in place) and returns (slot_mapping int64 [max_tokens], positions int32
    [max_tokens], cu_seqlens int32 [B + 1], seq_lens int32 [B], pages_used
    int32 [1])."""
    B = ctx_lens.shape[0]
    _expect(ctx_lens, "ctx_lens", (B,), torch.int32)
    _expect(new_lens, "new_lens", (B,), torch.int32)
    _expect(free_pages, "free_pages", (free_pages.numel(),), torch.int32)
    width, ld = _table(block_table, B)
    dev = ctx_lens.device
    if slot_mapping is None:
        slot_mapping = _empty((max_tokens,), torch.int64, dev, stream)
    if positions is None:
        positions = _empty((max_tokens,), torch.int32, dev, stream)
    if cu_seqlens is None:
        cu_seqlens = _empty((B + 1,), torch.int32, dev, stream)
    if seq_lens is None:
        seq_lens = _empty((B,), torch.int32, dev, stream)
    if pages_used is None:
        pages_used = _empty((1,), torch.int32, dev, stream)
    _expect(slot_mapping, "slot_mapping", (max_tokens,), torch.int64)
    _expect(positions, "positions", (max_tokens,), torch.int32)
    _expect(cu_seqlens, "cu_seqlens", (B + 1,), torch.int32)
    _expect(seq_lens, "seq_lens", (B,), torch.int32)
    _expect(pages_used, "pages_used", (1,), torch.int32)
    _check(lib().fp8_kv_slots(_ptr(ctx_lens), _ptr(new_lens), B, _ptr(free_pages),
                              free_pages.numel(), page_size, _ptr(block_table), width, ld,
                              max_tokens, _ptr(slot_mapping), _ptr(positions), _ptr(cu_seqlens),
                              _ptr(seq_lens), _ptr(pages_used), _stream(stream)), "fp8_kv_slots")
    return slot_mapping, positions, cu_seqlens, seq_lens, pages_used


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
    ldq, ldk = _tokens(q, "q"), _tokens(k, "k")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if k.shape[0] != T or k.shape[2] != D:
        raise ValueError(f"k must be [{T}, heads, {D}]; got {tuple(k.shape)}")
    _expect(positions, "positions", (T,), torch.int32)
    _expect(turns, "turns", (turns.numel(),), torch.int64)
    for g, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")):
        if g is not None:
            _expect(g, name, (D,), torch.bfloat16)
    q_out, ldqo = _fresh(q_out, "q_out", (T, Hq, D), q, stream)
    ldko = ldv = stride = slots = 0
    cached = k_cache is not None or v_cache is not None
    if cached:
        ldv = _tokens(v, "v", (T, Hkv, D))
        slots = _cache(k_cache, v_cache, Hkv, D)
        stride = _scales(k_scale, "k_scale", Hkv)
        if _scales(v_scale, "v_scale", Hkv) != stride:
            raise ValueError("k_scale and v_scale must both be per head or both single")
        if slot_mapping is not None:
            _expect(slot_mapping, "slot_mapping", (T,), torch.int64)
    if not (cached and cache_only):
        k_out, ldko = _fresh(k_out, "k_out", (T, Hkv, D), k, stream)
    _check(lib().fp8_qk_norm_rope(
        _ptr(q), ldq, _ptr(k), ldk, _ptr(v), ldv, T, Hq, Hkv, D, _ptr(gamma_q), _ptr(gamma_k), eps,
        _ptr(positions), _ptr(turns), 2 * turns.numel(), int(interleaved), _ptr(q_out), ldqo,
        _ptr(k_out), ldko, _ptr(k_scale), _ptr(v_scale), stride, _ptr(slot_mapping),
        _ptr(k_cache), _ptr(v_cache), slots, _stream(stream)), "fp8_qk_norm_rope")
    return q_out, k_out


def fp8_attention_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         cu_seqlens: torch.Tensor, scale: float | None = None,
                         out: torch.Tensor | None = None, stream=None):
    """Causal attention over prompts packed one after the other: q [T, Hq, D],
    k and v [T, Hkv, D] bf16 (views into a fused projection will do), sequence
    s in tokens cu_seqlens[s] .. cu_seqlens[s + 1] - 1 -> bf16 [T, Hq, D].
    Tokens outside every sequence get no output.  scale: 1 / sqrt(D) unless
    given."""
    ldq, ldk, ldv = _tokens(q, "q"), _tokens(k, "k"), _tokens(v, "v")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    if k.shape != (T, Hkv, D) or v.shape != (T, Hkv, D):
        raise ValueError(f"k and v must be [{T}, heads, {D}]; got {tuple(k.shape)}, {tuple(v.shape)}")
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold the sequences' bounds")
    _expect(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32)
    out, ldo = _fresh(out, "out", (T, Hq, D), q, stream)
    _check(lib().fp8_attention_prompt(
        _ptr(q), ldq, _ptr(k), ldk, _ptr(v), ldv, T, Hq, Hkv, D, _ptr(cu_seqlens),
        cu_seqlens.numel() - 1, D ** -0.5 if scale is None and D else scale or 0.0, _ptr(out), ldo,
        _stream(stream)), "fp8_attention_prompt")
    return out


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
    ldq = _tokens(q, "q")
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1] if isinstance(k_cache, torch.Tensor) and k_cache.dim() == 3 else 0
    slots = _cache(k_cache, v_cache, Hkv, D)
    stride = _scales(k_scale, "k_scale", Hkv)
    if _scales(v_scale, "v_scale", Hkv) != stride:
        raise ValueError("k_scale and v_scale must both be per head or both single")
    width, ld = _table(block_table, B)
    _expect(seq_lens, "seq_lens", (B,), torch.int32)
    out, ldo = _fresh(out, "out", (B, Hq, D), q, stream)
    if workspace is None:  # (a given workspace is size-checked by the library)
        need = lib().fp8_attention_decode_workspace_size(B, Hq, Hkv, D, width, page_size, prefix_len)
        workspace = _empty((max(need, 1),), torch.uint8, q.device, stream)
    _workspace(workspace)
    _check(lib().fp8_attention_decode(
        _ptr(q), ldq, B, Hq, Hkv, D, _ptr(k_cache), _ptr(v_cache), slots, _ptr(k_scale),
        _ptr(v_scale), stride, _ptr(block_table), width, ld, page_size, _ptr(seq_lens), prefix_len,
        D ** -0.5 if scale is None and D else scale or 0.0, _ptr(out), ldo, _ptr(workspace),
        workspace.numel(), _stream(stream)), "fp8_attention_decode")
    return out
