"""Group norm with an activation over packed channels-last feature maps (include/gn.h).

The maps are those that da_forward samples: mc_ms_feat [B, rows, C] with the
host tables spatial_shape [K, S, 2] and level_start_index [K, S]. Every map of
every batch item is normalised on its own.

    out, stats = gn_forward(feat, spatial_shape, level_start_index, gamma, beta, num_groups, act="silu")
    grad_feat, grad_gamma, grad_beta = gn_backward(feat, spatial_shape, level_start_index, gamma, beta, stats,
                                                   grad_out, num_groups, act="silu")

``GroupNormActFunction`` wraps the two as a torch autograd function. As in the
rest of the package the functions only marshal arguments; the arithmetic runs
in the library's CUDA kernels and there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import DA_BF16, DA_F16, DA_F32, _check, _dptr, _host_i32, _on_stream, load_library

__all__ = ["gn_forward", "gn_backward", "GroupNormActFunction", "GN_ACTIVATIONS"]

GN_ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2}
_DTYPES = {torch.float32: DA_F32, torch.bfloat16: DA_BF16, torch.float16: DA_F16}


class GnDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_cams", ctypes.c_int32), ("num_scales", ctypes.c_int32),
                ("num_embeds", ctypes.c_int32), ("num_groups", ctypes.c_int32), ("feat_dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("affine_scales", ctypes.c_int32), ("num_feat_rows", ctypes.c_int64),
                ("eps", ctypes.c_float)]


def _gn_dims(feat, ss, ls, gamma, beta, num_groups, eps, act) -> GnDims:
    if feat.dim() != 3:
        raise ValueError("feat must be [B, rows, C]")
    B, rows, C = feat.shape
    if ss.dim() != 3 or ss.shape[2] != 2:
        raise ValueError("spatial_shape must be [K, S, 2]")
    K, S = ss.shape[:2]
    if tuple(ls.shape) != (K, S):
        raise ValueError("level_start_index must be [K, S]")
    if gamma.shape != beta.shape or tuple(gamma.shape) not in ((C,), (S, C)):
        raise ValueError("gamma and beta must both be [C] or [S, C]")
    if feat.dtype not in _DTYPES:
        raise TypeError("feat must be float32, bfloat16 or float16")
    if gamma.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("gamma and beta must be float32")
    if act not in GN_ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(GN_ACTIVATIONS)}")
    return GnDims(B, K, S, C, int(num_groups), _DTYPES[feat.dtype], GN_ACTIVATIONS[act], gamma.dim() - 1, rows, eps)


def _tables(spatial_shape, level_start_index):
    ss, ls = _host_i32(spatial_shape), _host_i32(level_start_index)
    return ss, ls, ss.data_ptr() if ss.numel() else None, ls.data_ptr() if ls.numel() else None


def _scratch(lib, d, ssp, lsp, backward, device):
    n = ctypes.c_size_t(0)
    _check(lib.gn_workspace_size(ctypes.byref(d), ssp, lsp, backward, ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device=device)


def _like(t: Optional[torch.Tensor], name: str, shape, dtype, device) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}")
    return t


def gn_forward(feat: torch.Tensor, spatial_shape, level_start_index, gamma: torch.Tensor, beta: torch.Tensor,
               num_groups: int, eps: float = 1e-5, act: str = "none", out: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Forward pass on the current (or given) CUDA stream.

    feat [B, rows, C] fp32, bf16 or fp16; gamma, beta fp32 [C], or [S, C] for
    scales with weights of their own. Returns (out like feat, stats fp32
    [B, K, S, G, 2]: mean and 1/sqrt(var + eps), which gn_backward takes).
    out may be feat itself. What the call allocates belongs to the stream it
    runs on."""
    lib = load_library()
    ss, ls, ssp, lsp = _tables(spatial_shape, level_start_index)
    d = _gn_dims(feat, ss, ls, gamma, beta, num_groups, eps, act)
    with _on_stream(stream, feat.device) as handle:
        out = _like(out, "out", feat.shape, feat.dtype, feat.device)
        stats = torch.empty(d.batch, d.num_cams, d.num_scales, d.num_groups, 2, dtype=torch.float32, device=feat.device)
        ws = _scratch(lib, d, ssp, lsp, 0, feat.device)
        at = feat.get_device()
        _check(lib.gn_forward(ctypes.byref(d), _dptr(feat), ssp, lsp, _dptr(gamma, at), _dptr(beta, at), _dptr(out, at),
                              _dptr(stats), _dptr(ws), ws.numel(), handle))
    return out, stats


def gn_backward(feat: torch.Tensor, spatial_shape, level_start_index, gamma: torch.Tensor, beta: torch.Tensor,
                stats: torch.Tensor, grad_out: torch.Tensor, num_groups: int, act: str = "none",
                grad_feat: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Backward pass; returns (grad_feat like feat, grad_gamma, grad_beta fp32
    like gamma). grad_out is like feat; grad_feat may be grad_out itself."""
    lib = load_library()
    ss, ls, ssp, lsp = _tables(spatial_shape, level_start_index)
    d = _gn_dims(feat, ss, ls, gamma, beta, num_groups, 1.0, act)
    if grad_out.shape != feat.shape or grad_out.dtype != feat.dtype:
        raise ValueError("grad_out must have feat's shape and type")
    _like(stats, "stats", (d.batch, d.num_cams, d.num_scales, d.num_groups, 2), torch.float32, feat.device)
    with _on_stream(stream, feat.device) as handle:
        grad_feat = _like(grad_feat, "grad_feat", feat.shape, feat.dtype, feat.device)
        grad_gamma, grad_beta = torch.empty_like(gamma), torch.empty_like(beta)
        ws = _scratch(lib, d, ssp, lsp, 1, feat.device)
        at = feat.get_device()
        _check(lib.gn_backward(ctypes.byref(d), _dptr(feat), ssp, lsp, _dptr(gamma, at), _dptr(beta, at),
                               _dptr(stats, at), _dptr(grad_out, at), _dptr(grad_feat, at), _dptr(grad_gamma),
                               _dptr(grad_beta), _dptr(ws), ws.numel(), handle))
    return grad_feat, grad_gamma, grad_beta


class GroupNormActFunction(torch.autograd.Function):
    """Autograd wrapper: apply(feat, spatial_shape, level_start_index, gamma,
    beta, num_groups, eps, act) -> out. It has no second derivative: asking
    for one raises RuntimeError."""

    @staticmethod
    def forward(ctx, feat, spatial_shape, level_start_index, gamma, beta, num_groups, eps=1e-5, act="none"):
        feat, gamma, beta = feat.contiguous(), gamma.contiguous(), beta.contiguous()
        ss, ls = _host_i32(spatial_shape), _host_i32(level_start_index)
        out, stats = gn_forward(feat, ss, ls, gamma, beta, num_groups, eps, act)
        ctx.save_for_backward(feat, gamma, beta, stats)
        ctx.rest = (ss, ls, num_groups, act)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_output):
        feat, gamma, beta, stats = ctx.saved_tensors
        ss, ls, num_groups, act = ctx.rest
        gf, gg, gb = gn_backward(feat, ss, ls, gamma, beta, stats, grad_output.to(feat.dtype).contiguous(),
                                 num_groups, act)
        return gf, None, None, gg, gb, None, None, None
