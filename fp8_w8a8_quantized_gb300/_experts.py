"""Binding of the expert block's calls (include/fp8w8a8.h): routing, products
grouped by expert, and the join with the residual stream.  Checks of arguments
(ValueError) and allocations are the extension module's
(csrc/experts_binding.cpp, built beside the library); a status of the library
becomes Fp8Error.  Without the module the calls raise."""
from __future__ import annotations

import torch

from ._attention import _handle, _load, _result
from ._binding import lib

_module = None


def _native():
    """The loaded extension module."""
    global _module
    if _module is None:
        _module = _load("fp8_experts_binding")
    return _module


def fp8_moe_route_workspace_size(T: int, E: int, top_k: int) -> int:
    return int(lib().fp8_moe_route_workspace_size(T, E, top_k))


def fp8_moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True, scale: float = 1.0,
                  expert_ids: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                  offsets: torch.Tensor | None = None, row_token: torch.Tensor | None = None,
                  token_row: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                  stream=None):
    """Each token's top_k experts by the softmax of logits [T, E] (fp32 or bf16; -inf or
    NaN switches an expert off) and the rows that they make, sorted by expert.
    Returns (expert_ids int32 [T, top_k], weights fp32 [T, top_k], offsets int32
    [E + 1], row_token int32 [T * top_k], token_row int32 [T, top_k]); where none
    of them is given, all share one allocation."""
    return _result((_module or _native()).moe_route(
        logits, top_k, renormalize, scale, expert_ids, weights, offsets, row_token, token_row, workspace,
        _handle(stream)), "fp8_moe_route")


def fp8_grouped_gemm_workspace_size(E: int, R: int, N: int, K: int) -> int:
    return int(lib().fp8_grouped_gemm_workspace_size(E, R, N, K))


def fp8_grouped_gemm(xq: torch.Tensor, s_tok: torch.Tensor, wq: torch.Tensor, s_w: torch.Tensor,
                     offsets: torch.Tensor, swiglu: bool = False, y: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rows offsets[e] .. offsets[e + 1] - 1 of the codes xq [R, K] times the codes
    wq[e] [N, K], with both scales, as bf16 [R, N]; with swiglu silu(first half)
    * second half, [R, N / 2].  Rows outside the offsets stay as they are (in a new
    y: anything)."""
    return _result((_module or _native()).grouped_gemm(xq, s_tok, wq, s_w, offsets, swiglu, y, workspace,
                                                       _handle(stream)), "fp8_grouped_gemm")


def fp8_grouped_linear_workspace_size(E: int, R: int, N: int, K: int) -> int:
    return int(lib().fp8_grouped_linear_workspace_size(E, R, N, K))


def fp8_grouped_linear(x: torch.Tensor, wq: torch.Tensor, s_w: torch.Tensor, offsets: torch.Tensor,
                       row_token: torch.Tensor | None = None, swiglu: bool = False,
                       y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """An expert layer: row r is token row_token[r] of x (bf16 [T, K]), or row r of
    x itself, quantized with a scale of its own; then fp8_grouped_gemm.  Expert
    weights wq [E, N, K], s_w [E, N]: fp8_quant_per_channel_weights of the
    [E * N, K] rows."""
    return _result((_module or _native()).grouped_linear(x, wq, s_w, offsets, row_token, swiglu, y, workspace,
                                                         _handle(stream)), "fp8_grouped_linear")


def fp8_residual_norm_quant(h: torch.Tensor, y: torch.Tensor, gamma: torch.Tensor | None, eps: float = 1e-6,
                            gamma_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                            residual_scale: float = 1.0, branch_scale: float = 1.0,
                            token_row: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                            rows: bool = True, codes: bool = True, h_out: torch.Tensor | None = None,
                            z: torch.Tensor | None = None, xq: torch.Tensor | None = None,
                            s_tok: torch.Tensor | None = None, stream=None):
    """The end of a block and the start of the next: the branch y [T, K] (or, with
    token_row [T, top_k], the rows of y that belong to a token, by weight), normed
    (gamma_post), gated (gate [K] or [T, K]) and scaled, is added to the residual
    stream h [T, K]; the sum's norm (gamma) is the next layer's input.  Returns
    (h_out, z, xq, s_tok): the new stream, the normed rows in bf16 (rows=False:
    None) and as E4M3 codes with a scale a token (codes=False: None).  h_out=h
    works in place."""
    return _result((_module or _native()).residual_norm_quant(
        h, y, gamma, eps, gamma_post, gate, residual_scale, branch_scale, token_row, weights, rows, codes, h_out,
        z, xq, s_tok, _handle(stream)), "fp8_residual_norm_quant")
