"""The rotary norm and the attention over a paged cache from their definitions
in 64 bits (include/qkr.h, include/paged.h), with the sums of magnitudes from
which the tests' tolerances are made. Plain torch; shares no code with the
package. Tolerances count roundings as in operator_refs.py: U = 2^-24 is half a
step of fp32, half_step(t) that of the tensors' type.
"""
import ctypes
import math

import torch

from operator_refs import U, half_step


# The structures of include/qkr.h and include/paged.h, for tests of the C ABI.

class QkrProblem(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "num_queries", "num_keys", "num_heads", "num_kv_heads", "width",
                                               "rotated", "dtype", "interleaved", "normed")]
                + [("eps", ctypes.c_float), ("magnitude", ctypes.c_float), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                   ("q_stride", ctypes.c_int64 * 4), ("k_stride", ctypes.c_int64 * 4)]
                + [(n, ctypes.c_void_p) for n in ("q_weight", "k_weight", "turns", "pos_q", "pos_k")])


class PgCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64 * 4), ("v_stride", ctypes.c_int64 * 3),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("table_pages", ctypes.c_int32),
                ("page_table", ctypes.c_void_p), ("lengths", ctypes.c_void_p), ("counts", ctypes.c_void_p)]


class PgProblem(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "num_tokens", "num_heads", "num_kv_heads", "width", "value_width",
                                               "dtype", "num_buckets", "reach", "causal")]
                + [("scale", ctypes.c_float), ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64 * 4), ("cache", PgCache)]
                + [(n, ctypes.c_void_p) for n in ("lam", "bias_table", "bucket_map", "pos_q", "pos_k", "key_mask", "tree")])


def serving_library(lib):
    """libda.so with the argument types of the calls that the tests make themselves."""
    vp = ctypes.c_void_p
    size = ctypes.POINTER(ctypes.c_size_t)
    for name, types in (("qkr_forward", [vp] * 4), ("qkr_workspace_size", [vp, size]), ("qkr_backward", [vp] * 8 + [ctypes.c_size_t, vp]),
                        ("pg_append", [vp, vp, vp, ctypes.c_int32, vp, vp, vp]), ("pg_path", [vp]), ("pg_workspace_size", [vp, size]),
                        ("pg_attention", [vp] * 3 + [ctypes.c_size_t, vp])):
        f = getattr(lib, name)
        f.argtypes, f.restype = types, ctypes.c_int
    return lib


def radians(turns):
    """Angles of one position, from turns in units of 2^-64 (signed)."""
    return [t / 2 ** 64 * 2 * math.pi for t in turns.tolist()]


def turned(pos, turns):
    """cos and sin [..., R / 2] of positions [...]: the product modulo a turn in
    whole numbers, so that far positions cost nothing."""
    flat = [[(p * t) % 2 ** 64 / 2 ** 64 * 2 * math.pi for t in turns.tolist()] for p in pos.reshape(-1).tolist()]
    a = torch.tensor(flat, dtype=torch.float64).reshape(*pos.shape, len(turns))
    return a.cos().to(pos.device), a.sin().to(pos.device)


def _pairs(D, R, interleaved):
    a = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    return a, a + (1 if interleaved else R // 2)


def qkr_reference(x, turns=None, weight=None, pos=None, eps=1e-6, interleaved=False, magnitude=1.0, grad=None):
    """One tensor x [B, L, H, 2, D] with pos [B, L]: out, and with grad grad_x and grad_weight."""
    B, L, H, _, D = x.shape
    dt, o = x.dtype, half_step(x.dtype)
    x = x.double()
    R = 0 if turns is None else 2 * len(turns)
    w = torch.ones(D, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    rn = torch.ones_like(x[..., :1]) if eps is None else (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = x * rn
    y = n * w
    a, b = _pairs(D, R, interleaved)
    if R:
        if pos is None:
            pos = torch.arange(L, device=x.device).expand(B, L)
        c, s = (t[:, :, None, None] * magnitude for t in turned(pos, turns))

    def turn(t, s, size):
        """Turned pairs; with `size`, the magnitudes of what is summed."""
        z = t.clone()
        if R:
            ta, tb, cc, ss = (t[..., a], t[..., b], c, s) if not size else (t[..., a].abs(), t[..., b].abs(), c * 0 + magnitude, s * 0 + magnitude)
            z[..., a], z[..., b] = ta * cc - tb * ss if not size else ta * cc + tb * ss, ta * ss + tb * cc
        return z.abs() if size else z

    S = s if R else None
    # The sum of squares takes 2 roundings for each of a lane's channels and one
    # for each exchange, at most 40, of which rsqrt halves the effect; rsqrt, the
    # norm's two products, the cosine (its angle's rounding and 2 of its own,
    # times the magnitude) and the turn's two products are 12 more.
    val = {"out": turn(y, S, False)}
    tol = {"out": turn(y, S, True) * 32 * U + o * val["out"].abs()}
    if grad is not None:
        g = grad.double()
        gy, ga = turn(g, -S if R else None, False), turn(g, S, True)
        h, ha = gy * w, ga * w.abs()
        val["grad_weight"] = (gy * n).sum((0, 1, 2, 3))
        # A lane adds its own vectors in a row, some dozens here, then lanes, warps and rows.
        tol["grad_weight"] = (ga * n.abs()).sum((0, 1, 2, 3)) * (32 + 128) * U
        if eps is None:
            val["grad_x"], size = gy, ga
        else:
            val["grad_x"] = rn * (h - n * (h * n).mean(-1, keepdim=True))
            size = rn * (ha + n.abs() * (ha * n.abs()).mean(-1, keepdim=True))
        # h has 12 roundings, n 24, the mean of their products 40 more and n in
        # it twice, the factor before all 24.
        tol["grad_x"] = size * 128 * U + o * val["grad_x"].abs()
    if dt != torch.float32:
        tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
        for name in ("out", "grad_x"):
            if name in tol:
                tol[name] = tol[name] + tiny
    return val, tol


def paged_reference(q, k_cache, v_cache, lam, page_table, key_lengths, counts=None, tree=None, bias_table=None, bucket_map=None,
                    pos_q=None, pos_k=None, key_mask=None, causal=True, scale=None, rounded=True):
    """Value and tolerance of out; `rounded`: weights are rounded to the type."""
    B, T, H, _, D = q.shape
    P, S, Hk, Dv = v_cache.shape
    N, dt = page_table.shape[1], q.dtype
    L = N * S
    G = H // Hk
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(B, T, H, Dv, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    r, o = (half_step(dt) if rounded and dt != torch.float32 else 0.0), half_step(dt)
    for b in range(B):
        n = min(max(int(key_lengths[b]), 0), L)
        c = T if counts is None else min(max(int(counts[b]), 0), T)
        j = torch.arange(n, device=q.device)
        page = page_table[b].long()[j // S]
        there = (page >= 0) & (page < P)
        if key_mask is not None:
            there &= key_mask[b, :n]
        j, page = j[there], page[there]
        if len(j) == 0 or c == 0:
            continue
        k = k_cache[page, j % S].double().repeat_interleave(G, 1).permute(1, 2, 0, 3)     # [H, 2, n, D]
        v = v_cache[page, j % S].double().repeat_interleave(G, 1).permute(1, 0, 2)        # [H, n, Dv]
        pk = j if pos_k is None else pos_k[b].long()[j]
        pq = n - c + torch.arange(c, device=q.device) if pos_q is None else pos_q[b, :c].long()
        rel = pk[None] - pq[:, None]
        if tree is not None:
            new = j - (n - c)
            see = (new < 0)[None] | tree[b, :c][:, new.clamp(0, T - 1)]
        else:
            see = rel <= 0 if causal else torch.ones_like(rel, dtype=torch.bool)
        some = see.any(1)[None, :, None]
        qb = q[b, :c].double().permute(1, 2, 0, 3).masked_fill(~some[:, None], 0)
        bias = 0.0
        if bias_table is not None:
            reach = bucket_map.shape[0] // 2
            bias = bias_table.double()[bucket_map.long()[rel.clamp(-reach, reach) + reach]].permute(2, 0, 1)[:, None]
        t = (qb @ k.transpose(-1, -2) * scale + bias).masked_fill(~see, float("-inf"))
        e = (t - t.amax(-1, keepdim=True).masked_fill(~some[:, None], 0)).exp()
        p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
        lm = lam.double()[:, None, None]
        res = (p[:, 0] - lm * p[:, 1]) @ v
        # As for dattn_forward: a score is a sum of D products and the bias.
        big = float((qb.abs() @ k.abs().transpose(-1, -2)).amax() * abs(scale)) + (float(bias_table.abs().max()) if bias_table is not None else 0)
        eps = U * (2 * (D / 4 + 16) * (big + 1) + 64 + L / 64)
        M = (p[:, 0] + lm.abs() * p[:, 1]) @ v.abs()
        out[b, :c] = res.permute(1, 0, 2)
        # Rounded weights p + e are divided by their own sum: off by sum e (v - out), at most r (M + |out|).
        tol[b, :c] = (M * (eps + r) + (o + r) * res.abs()).permute(1, 0, 2)
    if dt != torch.float32:  # weights below fp16's normal numbers round to absolute steps
        tol += torch.finfo(dt).smallest_normal * torch.finfo(dt).eps * (1 + 8 * L ** 0.5)
    return {"out": out}, {"out": tol}
