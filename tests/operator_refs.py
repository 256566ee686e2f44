"""The group norm and the differential attention from their definitions in 64
bits (include/gn.h, include/dattn.h), with the sums of magnitudes from which
the tests' tolerances are made. Plain torch; shares no code with the package.

Tolerances count roundings. u = 2^-24 is half a step of fp32, r half a step
of the type of the tensors (finfo(t).eps / 2; 2^-8 for bf16, 2^-11 for fp16),
u for fp32. A value formed from terms of magnitudes summing to M with n
roundings in a row is off by at most about n * u * M.
"""
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gn_reference(x, maps, gamma, beta, groups, eps, act, grad=None):
    """x [B, rows, C]; maps: (start, pixels, scale) of each; gamma, beta [S, C].
    Returns values and tolerances as dicts: out, and with grad grad_feat,
    grad_gamma, grad_beta ([S, C]). Rows of no map are zeros."""
    B, _, C = x.shape
    dt, r = x.dtype, half_step(x.dtype)
    x, gamma, beta = x.double(), gamma.double(), beta.double()
    val = {"out": torch.zeros_like(x)}
    tol = {"out": torch.zeros_like(x)}
    if grad is not None:
        grad = grad.double()
        for d in (val, tol):
            d.update(grad_feat=torch.zeros_like(x), grad_gamma=torch.zeros_like(gamma), grad_beta=torch.zeros_like(beta))
    for start, n, s in maps:
        part = slice(start, start + n)
        t = x[:, part].reshape(B, n, groups, C // groups)
        mean = t.mean((1, 3), keepdim=True)
        var = (t - mean).square().mean((1, 3), keepdim=True)
        rstd = (var + eps).rsqrt()
        norm = ((t - mean) * rstd).reshape(B, n, C)
        # The mean is off by about 8 roundings of itself and of the spread;
        # the deviations' sum by 16 of its own, and rstd by half of that.
        off = ((8 * U) * (mean.abs() * rstd + 1) + 16 * U * norm.reshape(t.shape).abs()).reshape(B, n, C)
        g, b = gamma[s], beta[s]
        z = norm * g + b
        sig = torch.sigmoid(z)
        off_z = off * g.abs() + 4 * U * (z.abs() + b.abs())
        slope = {"none": torch.ones_like(z), "relu": (z > 0).double(), "silu": sig * (1 + z * (1 - sig))}[act]
        y = {"none": z, "relu": z.clamp(min=0), "silu": z * sig}[act]
        val["out"][:, part] = y
        # |act'| <= 1.1; the exponential and the quotient of silu cost 16 more
        # roundings, plus one per unit of |z| in the exponent.
        tol["out"][:, part] = 1.1 * off_z + (16 + 4 * z.abs()) * U * y.abs() + r * y.abs()
        if grad is None:
            continue
        h = grad[:, part] * slope
        # silu'' <= 0.5
        off_h = grad[:, part].abs() * ((off_z * 0.5 if act == "silu" else 0) + (16 + 4 * z.abs()) * U * slope.abs() + 4 * U)
        val["grad_gamma"][s] += (h * norm).sum((0, 1))
        val["grad_beta"][s] += h.sum((0, 1))
        # Per-tile partial sums and their joins: 64 roundings of the magnitudes.
        tol["grad_gamma"][s] += (h.abs() * off + off_h * norm.abs() + 64 * U * (h * norm).abs()).sum((0, 1))
        tol["grad_beta"][s] += (off_h + 64 * U * h.abs()).sum((0, 1))
        gh = (g * h).reshape(t.shape)
        nt = norm.reshape(t.shape)
        m1, m2 = gh.mean((1, 3), keepdim=True), (gh * nt).mean((1, 3), keepdim=True)
        dx = rstd * (gh - m1 - nt * m2)
        val["grad_feat"][:, part] = dx.reshape(B, n, C)
        o_gh, o_n = (g.abs() * off_h + 4 * U * (g * h).abs()).reshape(t.shape), off.reshape(t.shape)
        o_m1 = (o_gh + 64 * U * gh.abs()).mean((1, 3), keepdim=True)
        o_m2 = (o_gh * nt.abs() + gh.abs() * o_n + 64 * U * (gh * nt).abs()).mean((1, 3), keepdim=True)
        e = rstd * (o_gh + o_m1 + nt.abs() * o_m2 + o_n * m2.abs() + 20 * U * (gh.abs() + m1.abs() + (nt * m2).abs()))
        tol["grad_feat"][:, part] = (e + r * dx.abs()).reshape(B, n, C)
    if dt != torch.float32:  # below the smallest normal number a step is absolute
        tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
        for name in ("out", "grad_feat"):
            if name in tol:
                tol[name] += tiny
    return val, tol


def dattn_reference(q, k, v, lam, table=None, bucket_map=None, pos_q=None, pos_k=None, key_mask=None, key_lengths=None,
                    causal=False, scale=None, grad=None):
    """Values and tolerances as dicts: out, and with grad grad_q, grad_k,
    grad_v, grad_lam, grad_table."""
    B, Lq, H, _, D = q.shape
    Lk, Hk, Dv = v.shape[1:]
    G, dev, dt = H // Hk, q.device, q.dtype
    scale = D ** -0.5 if scale is None else scale
    length = torch.full((B,), Lk, device=dev) if key_lengths is None else key_lengths.long().clamp(0, Lk)
    at = torch.arange(Lk, device=dev).expand(B, Lk)
    there = at < length[:, None]
    if key_mask is not None:
        there = there & key_mask
    pk = at if pos_k is None else pos_k.long()
    pq = torch.arange(Lq, device=dev) + length[:, None] - Lq if pos_q is None else pos_q.long()
    rel = pk[:, None] - pq[:, :, None]                                    # [B, Lq, Lk]
    see = (there[:, None] & ((rel <= 0) if causal else torch.ones_like(rel, dtype=torch.bool)))[:, None]
    some = see.any(-1, keepdim=True)                                      # [B, 1, Lq, 1]
    q = q.double().permute(0, 2, 3, 1, 4).masked_fill(~some[:, :, None], 0)              # [B, H, 2, Lq, D]
    k = k.double().masked_fill(~there[:, :, None, None, None], 0).permute(0, 2, 3, 1, 4).repeat_interleave(G, 1)
    v = v.double().masked_fill(~there[:, :, None, None], 0).permute(0, 2, 1, 3).repeat_interleave(G, 1)
    lam = lam.double()[:, None, None]
    bias, bucket = torch.zeros(1, dtype=torch.float64, device=dev), None
    if table is not None:
        reach = bucket_map.shape[0] // 2
        bucket = bucket_map.long()[rel.clamp(-reach, reach) + reach]
        bias = table.double()[bucket].permute(0, 3, 1, 2)                 # [B, H, Lq, Lk]

    def softmax(m):
        t = (q[:, :, m] @ k[:, :, m].transpose(-1, -2) * scale + bias).masked_fill(~see, float("-inf"))
        e = (t - t.amax(-1, keepdim=True).masked_fill(~some, 0)).exp() if Lk else t
        return e / e.sum(-1, keepdim=True).clamp(min=1e-300)

    p0, p1 = softmax(0), softmax(1)
    out = (p0 - lam * p1) @ v
    # A score is a sum of D products and the bias, kept times log2(e); its
    # error moves a weight by as much relatively, and the weights' sum too.
    # 2^x adds a few roundings, the sums over keys about one per tile of 64
    # and 64 within one.
    big = 0.0
    if Lk and Lq:
        big = float((q.abs() @ k.abs().transpose(-1, -2)).amax() * abs(scale) + bias.abs().max())
    eps = U * (2 * (D / 4 + 16) * (big + 1) + 64 + Lk / 64)
    r = half_step(dt) if dt != torch.float32 else 0.0  # roundings of weights as operands
    o = half_step(dt)                                  # rounding of the result
    absp = p0 + lam.abs() * p1
    M = absp @ v.abs()
    val, tol = {"out": out}, {"out": M * (eps + r) + o * out.abs()}
    if grad is not None:
        g = grad.double().permute(0, 2, 1, 3).masked_fill(~some, 0)
        e, ea = g @ v.transpose(-1, -2), g.abs() @ v.abs().transpose(-1, -2)
        d0, d1 = (p0 * e).sum(-1, keepdim=True), (p1 * e).sum(-1, keepdim=True)
        a0, a1 = (p0 * ea).sum(-1, keepdim=True), (p1 * ea).sum(-1, keepdim=True)
        s = (p0 * (e - d0), -lam * p1 * (e - d1))
        # Magnitudes of the terms of s. In 16 bits grad_q's d_m come from
        # rounded outputs: 2 r of the magnitudes of both maps' sums.
        sa = (p0 * (ea + a0 + 2 * lam.abs() * a1), lam.abs() * p1 * (ea + 2 * a1))
        eps2 = 2 * eps + U * (Dv / 4 + 64)

        def heads(t):
            return t.reshape(B, Hk, G, *t.shape[2:]).sum(2)

        val["grad_v"] = heads((p0 - lam * p1).transpose(-1, -2) @ g)
        tol["grad_v"] = heads(absp.transpose(-1, -2) @ g.abs()) * (eps + r) + o * val["grad_v"].abs()
        val["grad_q"] = scale * torch.stack([s[m] @ k[:, :, m] for m in (0, 1)], 2)
        tol["grad_q"] = abs(scale) * torch.stack([sa[m] @ k[:, :, m].abs() for m in (0, 1)], 2) * (eps2 + 4 * r) + o * val["grad_q"].abs()
        val["grad_k"] = scale * heads(torch.stack([s[m].transpose(-1, -2) @ q[:, :, m] for m in (0, 1)], 2))
        tol["grad_k"] = (abs(scale) * heads(torch.stack([sa[m].transpose(-1, -2) @ q[:, :, m].abs() for m in (0, 1)], 2)) * (eps2 + r)
                         + o * val["grad_k"].abs())
        val["grad_lam"], tol["grad_lam"] = -d1.sum((0, 2, 3)), a1.sum((0, 2, 3)) * (eps2 + U)
        for d in (val, tol):
            d["grad_v"] = d["grad_v"].permute(0, 2, 1, 3)
            d["grad_q"], d["grad_k"] = d["grad_q"].permute(0, 3, 1, 2, 4), d["grad_k"].permute(0, 3, 1, 2, 4)
        if table is not None:
            for d, t in ((val, s[0] + s[1]), (tol, (sa[0] + sa[1]) * (eps2 + 64 * U))):
                d["grad_table"] = torch.stack([(t * (bucket == n)[:, None]).sum((0, 2, 3)) for n in range(table.shape[0])])
            tol["grad_table"] = tol["grad_table"] + U * val["grad_table"].abs()
    for d in (val, tol):
        d["out"] = d["out"].permute(0, 2, 1, 3)
    if dt != torch.float32:
        tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
        for name in ("out", "grad_q", "grad_k", "grad_v"):
            if name in tol:
                # Weights below fp16's normal numbers round to absolute steps.
                tol[name] = tol[name] + tiny * (1 + 8 * Lk ** 0.5 + (Lq * G) ** 0.5)
    return val, tol


def check(got, val, tol, what=""):
    """Every element of got within its tolerance of val."""
    for name, want in val.items():
        x = got[name].double()
        assert x.shape == want.shape, f"{what} {name}: shape {tuple(x.shape)} for {tuple(want.shape)}"
        assert bool(torch.isfinite(x).all()), f"{what} {name}: not finite"
        bad = (x - want).abs() > tol[name]
        if bool(bad.any()):
            ratio = ((x - want).abs() / tol[name].clamp(min=1e-300))
            i = int(ratio.argmax())
            raise AssertionError(f"{what} {name}: {int(bad.sum())} of {bad.numel()} off; worst {float(ratio.max()):.3g} x its "
                                 f"tolerance at {i}: {float(x.reshape(-1)[i])} for {float(want.reshape(-1)[i])}")
