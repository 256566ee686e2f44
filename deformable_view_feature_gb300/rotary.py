"""Norm of every head's queries and keys and their rotation by position (include/qkr.h).

What comes before dattn_forward: each of a head's vectors is normalised by its
root mean square, weighted, and rotated by its position, in one pass over
queries and keys.

    turns = rotary_frequencies(64).cuda()                         # once
    q, k = qkr_forward(q, k, turns, q_weight, k_weight)
    grad_q, grad_k, grad_q_weight, grad_k_weight = qkr_backward(q, k, grad_out_q, grad_out_k, turns, q_weight, k_weight)

``QkRotaryFunction`` wraps the two as a torch autograd function. The functions
only marshal arguments; the arithmetic runs in the library's CUDA kernels and
there is no fallback.
"""
from __future__ import annotations

import math
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _binding, _on_stream

__all__ = ["qkr_forward", "qkr_backward", "rotary_frequencies", "QkRotaryFunction"]

def rotary_frequencies(rotated: int, base: float = 10000.0, stretch: float = 1.0, method: str = "linear",
                       original_length: Optional[int] = None, fast: float = 32.0, slow: float = 1.0) -> torch.Tensor:
    """The angle of each of the rotated / 2 pairs for one position, as int64
    [rotated / 2] in units of 2^-64 of a turn (qkr_forward's frequencies): pair
    i turns by base ** (-2 i / rotated) radians.

    stretch > 1 is for contexts that much longer than those trained on:
      "linear"  every angle divided by stretch
      "base"    base times stretch ** (rotated / (rotated - 2)), which leaves the
                first pair and divides the last one's angle by stretch
      "parts"   pairs that turn more than `fast` times within original_length
                positions stay, those that turn less than `slow` times are
                divided by stretch, and in between by a linear mixture of the
                two (magnitude is then usually 0.1 * ln(stretch) + 1)"""
    if rotated < 2 or rotated % 2:
        raise ValueError("rotated must be even and at least 2")
    if not base > 0 or not stretch > 0 or not math.isfinite(base) or not math.isfinite(stretch):
        raise ValueError("base and stretch must be positive and finite")
    if method not in ("linear", "base", "parts"):
        raise ValueError('method must be "linear", "base" or "parts"')
    if method == "parts" and (original_length is None or original_length < 1 or not fast > slow):
        raise ValueError('method "parts" needs original_length >= 1 and fast > slow')
    if method == "base":
        if rotated == 2:
            raise ValueError('method "base" needs more than one pair')
        base = base * stretch ** (rotated / (rotated - 2))
    of = []
    for i in range(rotated // 2):
        f = base ** (-2 * i / rotated)
        if method == "linear":
            f /= stretch
        elif method == "parts":
            times = original_length * f / (2 * math.pi)
            keep = min(max((times - slow) / (fast - slow), 0.0), 1.0)
            f = f * keep + f / stretch * (1 - keep)
        turns = round(f / (2 * math.pi) * 2 ** 64) % 2 ** 64
        of.append(turns - 2 ** 64 if turns >= 2 ** 63 else turns)
    return torch.tensor(of, dtype=torch.int64)


def qkr_forward(q: Optional[torch.Tensor], k: Optional[torch.Tensor] = None, frequencies: Optional[torch.Tensor] = None,
                q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                pos_q: Optional[torch.Tensor] = None, pos_k: Optional[torch.Tensor] = None, eps: Optional[float] = 1e-6,
                interleaved: bool = False, magnitude: float = 1.0, out_q: Optional[torch.Tensor] = None,
                out_k: Optional[torch.Tensor] = None, stream=None):
    """Forward pass on the current (or given) CUDA stream; returns (q, k),
    contiguous in their type, None for one that is not given.

    q [B, Lq, H, 2, D], k [B, Lk, Hkv, 2, D], any strides with a contiguous last
    dimension; frequencies int64 [R / 2] (rotary_frequencies) rotates the first
    R channels, None none of them; weights fp32 [D], default 1; pos_q, pos_k
    int32 [B, L], default the indices, the queries being the last of the
    sequence. eps=None leaves out the norm. Pairs are (i, R/2 + i), or
    (2 i, 2 i + 1) with interleaved; magnitude multiplies the rotated channels.
    out_q and out_k may be q and k themselves where these are contiguous. What
    the call allocates belongs to the stream it runs on."""
    args = (q, k, frequencies, q_weight, k_weight, pos_q, pos_k, eps, interleaved, magnitude, out_q, out_k)
    if stream is None:
        return _binding().rotary_forward(*args)
    with _on_stream(stream, (k if q is None else q).device):
        return _binding().rotary_forward(*args)


def qkr_backward(q: Optional[torch.Tensor], k: Optional[torch.Tensor], grad_out_q: Optional[torch.Tensor],
                 grad_out_k: Optional[torch.Tensor], frequencies: Optional[torch.Tensor] = None,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                 pos_q: Optional[torch.Tensor] = None, pos_k: Optional[torch.Tensor] = None, eps: Optional[float] = 1e-6,
                 interleaved: bool = False, magnitude: float = 1.0, stream=None):
    """Backward pass of qkr_forward with the same arguments (q and k as they
    were before it); returns (grad_q, grad_k, grad_q_weight, grad_k_weight), the
    first two contiguous in q's type, the others fp32 [D], None where there is
    no such input."""
    args = (q, k, frequencies, q_weight, k_weight, pos_q, pos_k, eps, interleaved, magnitude, grad_out_q, grad_out_k)
    if stream is None:
        return _binding().rotary_backward(*args)
    with _on_stream(stream, (k if q is None else q).device):
        return _binding().rotary_backward(*args)


class QkRotaryFunction(torch.autograd.Function):
    """Autograd wrapper: apply(q, k, frequencies, q_weight, k_weight, pos_q,
    pos_k, eps, interleaved, magnitude) -> (q, k), with gradients for q, k and
    the weights; k may be None. It has no second derivative: asking for one
    raises RuntimeError."""

    @staticmethod
    def forward(ctx, q, k=None, frequencies=None, q_weight=None, k_weight=None, pos_q=None, pos_k=None, eps=1e-6,
                interleaved=False, magnitude=1.0):
        q, k = (t if t is None or t.shape[-1] == 1 or t.stride(-1) == 1 else t.contiguous() for t in (q, k))
        q_weight, k_weight = (None if w is None else w.contiguous() for w in (q_weight, k_weight))
        out = qkr_forward(q, k, frequencies, q_weight, k_weight, pos_q, pos_k, eps, interleaved, magnitude)
        ctx.save_for_backward(q, k, frequencies, q_weight, k_weight, pos_q, pos_k)
        ctx.rest = (eps, interleaved, magnitude)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_q, grad_k):
        q, k, *rest = ctx.saved_tensors
        # An output that nothing used comes back as None or as zeros of any stride.
        grads = [None if t is None else torch.zeros_like(t, memory_format=torch.contiguous_format) if g is None
                 else g.to(t.dtype).contiguous() for t, g in ((q, grad_q), (k, grad_k))]
        gq, gk, gwq, gwk = qkr_backward(q, k, *grads, *rest, *ctx.rest)
        return gq, gk, None, gwq, gwk, None, None, None, None, None
