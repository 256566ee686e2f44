"""A cache of keys and values in pages, and differential attention over it (include/paged.h).

For histories that grow: the keys and values of B sequences lie in pages of a
shared pool, and page_table says which pages are whose.

    q = paged_append(k, v, k_cache, v_cache, page_table, lengths, q=q, frequencies=turns, k_weight=w, q_weight=w)
    out = paged_attention(q, k_cache, v_cache, lam, page_table, lengths + k.shape[1])

The first normalises and rotates the new tokens' keys (and queries) as
qkr_forward does and stores keys and values; the second is dattn_forward of the
new tokens over the cache: one token each, the next part of prompts, or trees of
drafted tokens. The functions only marshal arguments; the arithmetic runs in the
library's CUDA kernels and there is no fallback.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _binding, _on_stream

__all__ = ["paged_append", "paged_attention", "paged_path"]


def paged_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                 lengths: torch.Tensor, counts: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                 frequencies: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 eps: Optional[float] = 1e-6, interleaved: bool = False, magnitude: float = 1.0,
                 out_q: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Stores new tokens into the cache on the current (or given) CUDA stream;
    returns their queries, normalised and rotated, or None without q.

    k [B, T, Hkv, 2, D] and q [B, T, H, 2, D] become qkr_forward's, with the same
    options; v [B, T, Hkv, Dv] is stored as it is. k_cache [pages, page_size,
    Hkv, 2, D] and v_cache [pages, page_size, Hkv, Dv] are written in place.
    Token t of sequence b goes to place lengths[b] + t, which page
    page_table[b, place // page_size] holds; lengths int32 [B] are the cache's
    before the call, and are not changed. counts int32 [B]: sequence b has only
    its first counts[b] tokens. positions int32 [B, T] of the rotation, default
    the places. Tokens whose place no page holds (a number outside the pool, a
    place past the table) are not stored. Any strides with a contiguous last
    dimension."""
    args = (q, k, frequencies, q_weight, k_weight, None if q is None else positions, positions, eps, interleaved, magnitude, v,
            k_cache, v_cache, page_table, lengths, counts, out_q)
    if stream is None:
        return _binding().append(*args)
    with _on_stream(stream, k.device):
        return _binding().append(*args)


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, lam: torch.Tensor, page_table: torch.Tensor,
                    key_lengths: torch.Tensor, counts: Optional[torch.Tensor] = None, tree: Optional[torch.Tensor] = None,
                    bias_table: Optional[torch.Tensor] = None, bucket_map: Optional[torch.Tensor] = None,
                    pos_q: Optional[torch.Tensor] = None, pos_k: Optional[torch.Tensor] = None,
                    key_mask: Optional[torch.Tensor] = None, causal: bool = True, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Differential attention (dattn_forward) of new tokens over a paged cache
    that holds them already, on the current (or given) CUDA stream; returns out
    [B, T, H, Dv] in q's type.

    q [B, T, H, 2, D]; k_cache, v_cache and page_table as in paged_append, of any
    strides with a contiguous last dimension; key_lengths int32 [B] with the new
    tokens; lam fp32 [H]. Sequence b has counts[b] new tokens (default T), the
    last of its keys; the rows past them give 0. Query i sees the keys up to its
    own place (causal; all with causal=False), or with tree bool [B, T, T] all
    keys before the new ones and new token j where tree[b, i, j]. bias_table and
    bucket_map as in dattn_forward; pos_q int32 [B, T] and pos_k int32 [B, L],
    L = page_table.shape[1] * page_size, default the places; key_mask bool
    [B, L]. A query that sees no key gives 0. scale defaults to D ** -0.5."""
    args = (q, k_cache, v_cache, page_table, key_lengths, counts, lam, tree, bias_table, bucket_map, pos_q, pos_k, key_mask, causal,
            scale, out)
    if stream is None:
        return _binding().attention(*args)
    with _on_stream(stream, q.device):
        return _binding().attention(*args)


def paged_path(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, lam: torch.Tensor, page_table: torch.Tensor,
               key_lengths: torch.Tensor, counts=None, tree=None, bias_table=None, bucket_map=None, pos_q=None, pos_k=None,
               key_mask=None, causal: bool = True, scale: Optional[float] = None) -> str:
    """Which kernels paged_attention takes for these arguments: "tensor" (the
    tensor cores) or "general" (fp32 units)."""
    return "tensor" if _binding().path(q, k_cache, v_cache, page_table, key_lengths, counts, lam, tree, bias_table, bucket_map,
                                       pos_q, pos_k, key_mask, causal, scale) else "general"
