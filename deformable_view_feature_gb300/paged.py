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

import ctypes
import struct
from typing import Optional

import torch

from . import _check, _dptr, _on_stream, load_library
from . import rotary as _rotary
from .attention import _DTYPES, _small, _strided

__all__ = ["paged_append", "paged_attention", "paged_path"]


class PgCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64 * 4), ("v_stride", ctypes.c_int64 * 3),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("table_pages", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("counts", ctypes.c_void_p)]


class PgProblem(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "num_tokens", "num_heads", "num_kv_heads", "width", "value_width",
                                               "dtype", "num_buckets", "reach", "causal")]
                + [("scale", ctypes.c_float), ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64 * 4), ("cache", PgCache)]
                + [(n, ctypes.c_void_p) for n in ("lam", "bias_table", "bucket_map", "pos_q", "pos_k", "key_mask", "tree")])


# The same as bytes, which take a fifth of the time to fill.
_CACHE = struct.Struct("@2P7q3i3P")
_PROBLEM = struct.Struct("@10ifP4q")
_REST = struct.Struct("@7P")
assert _CACHE.size == ctypes.sizeof(PgCache) and _PROBLEM.size + _CACHE.size + _REST.size == ctypes.sizeof(PgProblem)


def _cache(k_cache, v_cache, page_table, lengths, counts, B, at, dtype) -> bytes:
    """The pg_cache of these arguments, after the checks that only the tensors'
    shapes and types allow."""
    if k_cache.dim() != 5 or k_cache.shape[3] != 2:
        raise ValueError("k_cache must be [pages, page_size, Hkv, 2, D]")
    if v_cache.dim() != 4:
        raise ValueError("v_cache must be [pages, page_size, Hkv, Dv]")
    P, S, Hkv = k_cache.shape[:3]
    if v_cache.shape[:3] != (P, S, Hkv):
        raise ValueError("k_cache and v_cache disagree on pages, page_size or heads")
    if k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise TypeError("the cache must have the new tokens' type")
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B, pages of a sequence]")
    N = page_table.shape[1]
    small = [_small(t, name, shape, torch.int32, at)
             for t, name, shape in ((page_table, "page_table", (B, N)), (lengths, "lengths", (B,)), (counts, "counts", (B,)))]
    return _CACHE.pack(_strided(k_cache, "k_cache", at), _strided(v_cache, "v_cache", at), *k_cache.stride()[:4],
                       *v_cache.stride()[:3], P, S, N, *small)


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
    lib = load_library()
    if k.dim() != 5 or v.dim() != 4:
        raise ValueError("k must be [B, T, Hkv, 2, D] and v [B, T, Hkv, Dv]")
    if q is not None and q.shape[:2] != k.shape[:2]:
        raise ValueError("q and k disagree on batch or tokens")
    B, T, Hkv, _, D = k.shape
    if v.shape[:3] != (B, T, Hkv) or v.dtype != k.dtype:
        raise ValueError(f"v must be {k.dtype} [B, T, Hkv, Dv] of k's tokens and heads")
    if k_cache.dim() != 5 or k_cache.shape[2:] != (Hkv, 2, D) or v_cache.dim() != 4 or v_cache.shape[2:] != v.shape[2:]:
        raise ValueError("the cache must hold the new tokens' heads and widths")
    at = k.get_device()
    cache = _cache(k_cache, v_cache, page_table, lengths, counts, B, at, k.dtype)
    p = _rotary._problem(q, k, frequencies, q_weight, k_weight, None if q is None else positions, positions, eps, interleaved,
                         magnitude)
    with _on_stream(stream, k.device) as handle:
        out_q = _rotary._result(q, out_q, "out_q")
        _check(lib.pg_append(p, _strided(v, "v", at) or None, (ctypes.c_int64 * 3)(*v.stride()[:3]), v.shape[3], cache,
                             _dptr(out_q, at), handle))
    return out_q


def _attention(q, k_cache, v_cache, lam, page_table, key_lengths, counts, tree, bias_table, bucket_map, pos_q, pos_k, key_mask,
               causal, scale) -> bytes:
    """The pg_problem of these arguments, after the checks that only the
    tensors' shapes and types allow."""
    if q.dim() != 5 or q.shape[3] != 2:
        raise ValueError("q must be [B, T, H, 2, D]")
    B, T, H, _, D = q.shape
    if q.dtype not in _DTYPES:
        raise TypeError("q and the cache must be float32, bfloat16 or float16")
    if k_cache.shape[-1] != D:
        raise ValueError("q and k_cache disagree on width")
    if (bias_table is None) != (bucket_map is None):
        raise ValueError("bias_table and bucket_map go together")
    at = q.get_device()
    cache = _cache(k_cache, v_cache, page_table, key_lengths, counts, B, at, q.dtype)
    Hkv, Dv = v_cache.shape[2:]
    L = page_table.shape[1] * k_cache.shape[1]
    table = buckets = num_buckets = reach = 0
    if bias_table is not None:
        if bias_table.dim() != 2 or bucket_map.dim() != 1 or bucket_map.shape[0] % 2 != 1:
            raise ValueError("bias_table must be [num_buckets, H] and bucket_map [2 * reach + 1]")
        num_buckets, reach = bias_table.shape[0], bucket_map.shape[0] // 2
        table = _small(bias_table, "bias_table", (num_buckets, H), torch.float32, at)
        buckets = _small(bucket_map, "bucket_map", (2 * reach + 1,), torch.int32, at)
    return (_PROBLEM.pack(B, T, H, Hkv, D, Dv, _DTYPES[q.dtype], num_buckets, reach, 1 if causal else 0,
                          D ** -0.5 if scale is None else scale, _strided(q, "q", at), *q.stride()[:4]) + cache
            + _REST.pack(_small(lam, "lam", (H,), torch.float32, at), table, buckets,
                         _small(pos_q, "pos_q", (B, T), torch.int32, at), _small(pos_k, "pos_k", (B, L), torch.int32, at),
                         _small(key_mask, "key_mask", (B, L), torch.bool, at), _small(tree, "tree", (B, T, T), torch.bool, at)))


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
    lib = load_library()
    p = _attention(q, k_cache, v_cache, lam, page_table, key_lengths, counts, tree, bias_table, bucket_map, pos_q, pos_k,
                   key_mask, causal, scale)
    shape = (*q.shape[:3], v_cache.shape[3])
    if out is not None and (out.shape != shape or out.dtype != q.dtype):
        raise ValueError(f"out must be {q.dtype} {shape}")
    with _on_stream(stream, q.device) as handle:
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=q.device)
        to, n = _dptr(out, q.get_device()), ctypes.c_size_t(0)
        _check(lib.pg_workspace_size(p, ctypes.byref(n)))
        ws = torch.empty(n.value, dtype=torch.uint8, device=q.device) if n.value else None
        _check(lib.pg_attention(p, to, _dptr(ws), n.value, handle))
    return out


def paged_path(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, lam: torch.Tensor, page_table: torch.Tensor,
               key_lengths: torch.Tensor, counts=None, tree=None, bias_table=None, bucket_map=None, pos_q=None, pos_k=None,
               key_mask=None, causal: bool = True, scale: Optional[float] = None) -> str:
    """Which kernels paged_attention takes for these arguments: "tensor" (the
    tensor cores) or "general" (fp32 units)."""
    lib = load_library()
    p = _attention(q, k_cache, v_cache, lam, page_table, key_lengths, counts, tree, bias_table, bucket_map, pos_q, pos_k,
                   key_mask, causal, scale)
    _check(lib.pg_workspace_size(p, ctypes.byref(ctypes.c_size_t(0))))  # the status of an invalid problem
    return "tensor" if lib.pg_path(p) == 1 else "general"
