"""Differential attention with a learned relative position bias by buckets (include/dattn.h).

Each head has two query and two key vectors and one value; its output is the
difference of two softmax maps over the keys, weighted by a learned lam:

    out = (softmax(q0 k0 + bias) - lam * softmax(q1 k1 + bias)) v

    buckets = relative_buckets(32, 128).cuda()                    # once
    out = dattn_forward(q, k, v, lam, bias_table=table, bucket_map=buckets)
    out, saved = dattn_forward(..., keep_for_backward=True)
    grad_q, grad_k, grad_v, grad_lam, grad_table = dattn_backward(q, k, v, lam, out, saved, grad_out, ...)

``DifferentialAttentionFunction`` wraps the two as a torch autograd function.
The functions only marshal arguments; the arithmetic runs in the library's CUDA
kernels and there is no fallback.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import DA_BF16, DA_F16, DA_F32, _check, _dptr, _on_stream, load_library

__all__ = ["dattn_forward", "dattn_backward", "dattn_path", "relative_buckets", "DifferentialAttentionFunction"]

_DTYPES = {torch.float32: DA_F32, torch.bfloat16: DA_BF16, torch.float16: DA_F16}


class DattnProblem(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "num_queries", "num_keys", "num_heads", "num_kv_heads", "width",
                                               "value_width", "dtype", "num_buckets", "reach", "causal")]
                + [("scale", ctypes.c_float)] + [(n, ctypes.c_void_p) for n in ("q", "k", "v")]
                + [("q_stride", ctypes.c_int64 * 4), ("k_stride", ctypes.c_int64 * 4), ("v_stride", ctypes.c_int64 * 3)]
                + [(n, ctypes.c_void_p) for n in ("lam", "bias_table", "bucket_map", "pos_q", "pos_k", "key_mask",
                                                  "key_lengths")])


# The same as bytes, which take a fifth of the time to fill.
_PROBLEM = struct.Struct("@11if3P11q7P")
assert _PROBLEM.size == ctypes.sizeof(DattnProblem)


def relative_buckets(num_buckets: int, max_distance: int, bidirectional: bool = True) -> torch.Tensor:
    """Bucket of each relative position r = key - query in -max_distance ..
    max_distance, as int32 [2 * max_distance + 1] (a bucket_map for
    dattn_forward; farther positions take the ends' buckets).

    With bidirectional, one half of the buckets is for keys at or before the
    query and the other for keys after it; without, all are for keys at or
    before it and later keys share bucket 0. Half of each side's buckets hold
    one distance each; the others grow with the logarithm of the distance. The
    borders are decided in whole numbers: with e single-distance buckets and w
    others, distance n lies t or more buckets past e when
    n**w * e**t >= max_distance**t * e**w."""
    side = num_buckets // 2 if bidirectional else num_buckets
    if side < 1 or max_distance < 1:
        raise ValueError("relative_buckets needs a bucket per side and max_distance >= 1")
    e = max(side // 2, 1)
    w = side - e
    of = []
    for r in range(-max_distance, max_distance + 1):
        n = abs(r) if bidirectional else max(-r, 0)
        t = 0
        if n >= e:
            while t + 1 < w and n ** w * e ** (t + 1) >= max_distance ** (t + 1) * e ** w:
                t += 1
            n = e + t
        of.append(min(n, side - 1) + (side if bidirectional and r > 0 else 0))
    return torch.tensor(of, dtype=torch.int32)


def _strided(t: torch.Tensor, name: str, index: int) -> int:
    """Data pointer of a q, k or v whose last dimension is contiguous."""
    if t.numel() == 0:
        return 0
    if not t.is_cuda:
        raise ValueError("device tensors must live on a CUDA device")
    if t.get_device() != index:
        raise ValueError("tensors must all live on one CUDA device")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr()


def _small(t: Optional[torch.Tensor], name: str, shape, dtype, index: int) -> int:
    if t is None:
        return 0
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {shape}")
    return _dptr(t, index) or 0


def _problem(q, k, v, lam, bias_table, bucket_map, pos_q, pos_k, key_mask, key_lengths, causal, scale) -> bytes:
    """The dattn_problem of these arguments, after the checks that only the
    tensors' shapes and types allow."""
    if q.dim() != 5 or q.shape[3] != 2:
        raise ValueError("q must be [B, Lq, H, 2, D]")
    if k.dim() != 5 or k.shape[3] != 2:
        raise ValueError("k must be [B, Lk, Hkv, 2, D]")
    if v.dim() != 4:
        raise ValueError("v must be [B, Lk, Hkv, Dv]")
    B, Lq, H, _, D = q.shape
    Bk, Lk, Hkv, _, Dk = k.shape
    Bv, Lv, Hv, Dv = v.shape
    if Bk != B or Bv != B or Lv != Lk or Hv != Hkv or Dk != D:
        raise ValueError("q, k and v disagree on batch, keys, heads or width")
    dtype = q.dtype
    if dtype not in _DTYPES:
        raise TypeError("q, k and v must be float32, bfloat16 or float16")
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError("q, k and v must have one type")
    table = buckets = num_buckets = reach = 0
    at = q.get_device()
    if bias_table is not None or bucket_map is not None:
        if bias_table is None or bucket_map is None:
            raise ValueError("bias_table and bucket_map go together")
        if bias_table.dim() != 2 or bucket_map.dim() != 1 or bucket_map.shape[0] % 2 != 1:
            raise ValueError("bias_table must be [num_buckets, H] and bucket_map [2 * reach + 1]")
        num_buckets, reach = bias_table.shape[0], bucket_map.shape[0] // 2
        table = _small(bias_table, "bias_table", (num_buckets, H), torch.float32, at)
        buckets = _small(bucket_map, "bucket_map", (2 * reach + 1,), torch.int32, at)
    sq, sk, sv = q.stride(), k.stride(), v.stride()
    return _PROBLEM.pack(B, Lq, Lk, H, Hkv, D, Dv, _DTYPES[dtype], num_buckets, reach, 1 if causal else 0,
                         D ** -0.5 if scale is None else scale, _strided(q, "q", at), _strided(k, "k", at), _strided(v, "v", at),
                         sq[0], sq[1], sq[2], sq[3], sk[0], sk[1], sk[2], sk[3], sv[0], sv[1], sv[2],
                         _small(lam, "lam", (H,), torch.float32, at), table, buckets,
                         _small(pos_q, "pos_q", (B, Lq), torch.int32, at), _small(pos_k, "pos_k", (B, Lk), torch.int32, at),
                         _small(key_mask, "key_mask", (B, Lk), torch.bool, at),
                         _small(key_lengths, "key_lengths", (B,), torch.int32, at))


def _saved_shape(shape, dtype):
    """Shape of saved[0] (out1 of include/dattn.h) for an output of this shape."""
    return shape if dtype == torch.float32 else (*shape[:3], 3, shape[3])


def _scratch(lib, p, backward, device):
    n = ctypes.c_size_t(0)
    _check(lib.dattn_workspace_size(p, backward, ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device=device) if n.value else None, n.value


def dattn_path(q, k, v, lam, backward: bool = False, **options) -> str:
    """Which kernels dattn_forward (or dattn_backward) takes for these
    arguments: "tensor" (the tensor cores) or "general" (fp32 units)."""
    lib, p = load_library(), _options(q, k, v, lam, **options)
    _check(lib.dattn_workspace_size(p, int(backward), ctypes.byref(ctypes.c_size_t(0))))  # the status of an invalid problem
    return "tensor" if lib.dattn_path(p, int(backward)) == 1 else "general"


def _options(q, k, v, lam, bias_table=None, bucket_map=None, pos_q=None, pos_k=None, key_mask=None, key_lengths=None,
             causal=False, scale=None) -> bytes:
    return _problem(q, k, v, lam, bias_table, bucket_map, pos_q, pos_k, key_mask, key_lengths, causal, scale)


def dattn_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor,
                  bias_table: Optional[torch.Tensor] = None, bucket_map: Optional[torch.Tensor] = None,
                  pos_q: Optional[torch.Tensor] = None, pos_k: Optional[torch.Tensor] = None,
                  key_mask: Optional[torch.Tensor] = None, key_lengths: Optional[torch.Tensor] = None,
                  causal: bool = False, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  keep_for_backward: bool = False, stream=None):
    """Forward pass on the current (or given) CUDA stream; returns out
    [B, Lq, H, Dv] in q's type, with keep_for_backward (out, saved).

    q [B, Lq, H, 2, D], k [B, Lk, Hkv, 2, D], v [B, Lk, Hkv, Dv], H a multiple
    of Hkv, any strides with a contiguous last dimension; lam fp32 [H];
    bias_table fp32 [num_buckets, H] with bucket_map int32 [2 * reach + 1]
    (relative_buckets); pos_q, pos_k int32 [B, L], in (-2**30, 2**30), default
    the indices, the queries being the last; key_mask bool [B, Lk];
    key_lengths int32 [B]. A query that sees no key gives 0. scale defaults to
    D ** -0.5. What the call allocates belongs to the stream it runs on."""
    lib = load_library()
    p = _problem(q, k, v, lam, bias_table, bucket_map, pos_q, pos_k, key_mask, key_lengths, causal, scale)
    shape = (*q.shape[:3], v.shape[3])
    if out is not None and (out.shape != shape or out.dtype != q.dtype):
        raise ValueError(f"out must be {q.dtype} {shape}")
    with _on_stream(stream, q.device) as handle:
        if out is None:
            out = torch.empty(shape, dtype=q.dtype, device=q.device)
        out1 = lse = None
        if keep_for_backward:
            out1 = torch.empty(_saved_shape(shape, q.dtype), dtype=q.dtype, device=q.device)
            lse = torch.empty(shape[0], shape[2], 2, shape[1], dtype=torch.float32, device=q.device)
        ws, n = _scratch(lib, p, 0, q.device)
        _check(lib.dattn_forward(p, _dptr(out, q.get_device()), _dptr(out1), _dptr(lse), _dptr(ws), n, handle))
    return (out, (out1, lse)) if keep_for_backward else out


def dattn_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: torch.Tensor, out: torch.Tensor, saved,
                   grad_out: torch.Tensor, bias_table: Optional[torch.Tensor] = None,
                   bucket_map: Optional[torch.Tensor] = None, pos_q: Optional[torch.Tensor] = None,
                   pos_k: Optional[torch.Tensor] = None, key_mask: Optional[torch.Tensor] = None,
                   key_lengths: Optional[torch.Tensor] = None, causal: bool = False, scale: Optional[float] = None,
                   stream=None):
    """Backward pass of dattn_forward(..., keep_for_backward=True) with the
    same arguments; returns (grad_q, grad_k, grad_v contiguous in q's type,
    grad_lam fp32 [H], grad_table fp32 [num_buckets, H] or None)."""
    lib = load_library()
    p = _problem(q, k, v, lam, bias_table, bucket_map, pos_q, pos_k, key_mask, key_lengths, causal, scale)
    shape = (*q.shape[:3], v.shape[3])
    out1, lse = saved
    for name, t in (("out", out), ("grad_out", grad_out)):
        if t.shape != shape or t.dtype != q.dtype:
            raise ValueError(f"{name} must be {q.dtype} {shape}")
    if (out1.shape != _saved_shape(shape, q.dtype) or out1.dtype != q.dtype
            or lse.shape != (shape[0], shape[2], 2, shape[1]) or lse.dtype != torch.float32):
        raise ValueError("saved must be what dattn_forward returned")
    with _on_stream(stream, q.device) as handle:
        gq, gk, gv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        gl = torch.empty_like(lam)
        gt = torch.empty_like(bias_table) if bias_table is not None else None
        ws, n = _scratch(lib, p, 1, q.device)
        at = q.get_device()
        _check(lib.dattn_backward(p, _dptr(out, at), _dptr(out1, at), _dptr(lse, at), _dptr(grad_out, at), _dptr(gq),
                                  _dptr(gk), _dptr(gv), _dptr(gl), _dptr(gt), _dptr(ws), n, handle))
    return gq, gk, gv, gl, gt


class DifferentialAttentionFunction(torch.autograd.Function):
    """Autograd wrapper: apply(q, k, v, lam, bias_table, bucket_map, pos_q,
    pos_k, key_mask, key_lengths, causal, scale) -> out, with gradients for q,
    k, v, lam and bias_table. Without a gradient to come (torch.no_grad, or no
    argument that requires one) nothing is kept for it. It has no second
    derivative: asking for one raises RuntimeError."""

    @classmethod
    def apply(cls, q, k, v, lam, bias_table=None, *rest):
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (q, k, v, lam, bias_table)):
            return super().apply(q, k, v, lam, bias_table, *rest)
        return dattn_forward(*cls._contiguous(q, k, v, lam, bias_table), *rest)  # no backward pass: nothing kept for one

    @staticmethod
    def _contiguous(q, k, v, lam, bias_table):
        q, k, v = (t if t.shape[-1] == 1 or t.stride(-1) == 1 else t.contiguous() for t in (q, k, v))
        return q, k, v, lam.contiguous(), None if bias_table is None else bias_table.contiguous()

    @staticmethod
    def forward(ctx, q, k, v, lam, bias_table=None, bucket_map=None, pos_q=None, pos_k=None, key_mask=None,
                key_lengths=None, causal=False, scale=None):
        q, k, v, lam, bias_table = DifferentialAttentionFunction._contiguous(q, k, v, lam, bias_table)
        opt = dict(bias_table=bias_table, bucket_map=bucket_map, pos_q=pos_q, pos_k=pos_k, key_mask=key_mask,
                   key_lengths=key_lengths, causal=causal, scale=scale)
        out, saved = dattn_forward(q, k, v, lam, **opt, keep_for_backward=True)
        ctx.save_for_backward(q, k, v, lam, out, *saved, bias_table, bucket_map, pos_q, pos_k, key_mask, key_lengths)
        ctx.rest = (causal, scale)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_output):
        q, k, v, lam, out, out1, lse, *opt = ctx.saved_tensors
        names = ("bias_table", "bucket_map", "pos_q", "pos_k", "key_mask", "key_lengths")
        gq, gk, gv, gl, gt = dattn_backward(q, k, v, lam, out, (out1, lse), grad_output.to(q.dtype).contiguous(),
                                            **dict(zip(names, opt)), causal=ctx.rest[0], scale=ctx.rest[1])
        return gq, gk, gv, gl, gt, None, None, None, None, None, None, None
