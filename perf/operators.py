"""What the feature-norm and differential-attention operators are measured on.

Two families of cases, as they occur around the deformable aggregation:

* ``norm``: group norm with an activation over the packed channels-last
  feature maps [B, rows, C] that the aggregation samples, every (batch item,
  camera, scale) map normalised on its own; forward alone or with its
  backward pass.
* ``attention``: differential attention with a learned relative position bias
  by buckets, among the instances that the aggregation's output updates and
  over their history; forward alone (one query token up to long ones) or with
  its backward pass.

``run`` with ``own`` false computes each in plain elementary operations in 32
bits; with ``own`` true it calls the package's entry points.
"""
import math

import torch

own = False

# The feature pyramids of this repository's workloads.
SP4D = "64x176,32x88,16x44,8x22"
LARGE = "80x200,40x100,20x50,10x25"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
KEPT = 0.85  # share of the keys that a key mask keeps


def _norm(name, **kw):
    return {"name": name, "op": "norm", "batch": 1, "cams": 1, "maps": SP4D, "channels": 256, "groups": 32,
            "type": "bf16", "act": "silu", "per_scale": False, "train": False, **kw}


def _attention(name, **kw):
    return {"name": name, "op": "attention", "batch": 1, "queries": 900, "keys": 900, "heads": 4, "kv_heads": 4,
            "width": 32, "value_width": 64, "type": "bf16", "buckets": 32, "reach": 128, "causal": False,
            "frames": 0, "key_mask": False, "ragged": False, "train": False, **kw}


def listed():
    return [
        # The toy map of the tests: the launch and the host's work are what counts.
        _norm("norm, one small map", maps="16x16", channels=32, groups=8, type="f32", act="relu"),
        # The 6-camera, 4-scale neck at inference.
        _norm("norm, six cameras", cams=6),
        # The neck's training step at the aggregation's training shape: far larger than the caches.
        _norm("norm, training batch", batch=6, cams=6, type="f32", train=True),
        # Odd map sides down to a single pixel, a width that is no power of two, scales with weights of their own.
        _norm("norm, odd maps training", batch=3, cams=2, maps="57x101,29x51,7x13,1x1", channels=96, groups=12,
              type="f16", per_scale=True, train=True),
        # The larger-image variant in 16 bits.
        _norm("norm, large images training", cams=6, maps=LARGE, train=True),
        # One new token against a short history: latency.
        _attention("attention, one token", queries=1, keys=77, causal=True),
        # Serving: one token each for a batch with long, ragged caches and shared key heads.
        _attention("attention, long caches", batch=8, queries=1, keys=32768, heads=16, kv_heads=4, width=64,
                   value_width=128, causal=True, ragged=True),
        # The head's self-attention among 900 anchors, in the framework's default type.
        _attention("attention, anchors", type="f32"),
        # The head's training step: 900 anchors over the frame's own and four past frames' instances, some of
        # them invalid, one batch item with no valid instance at all.
        _attention("attention, frames training", batch=6, keys=2100, frames=5, key_mask=True, train=True),
        # An odd sequence trained in 32 bits.
        _attention("attention, odd sequence training", batch=2, queries=333, keys=333, heads=6, kv_heads=2, width=24,
                   value_width=48, type="f32", causal=True, train=True),
        # A prompt that is taken in at once, of odd length, in half precision.
        _attention("attention, prompt", queries=2047, keys=4095, heads=8, kv_heads=2, width=64, value_width=128,
                   type="f16", causal=True),
        # Long sequences trained.
        _attention("attention, long sequence training", batch=2, queries=8192, keys=8192, heads=8, kv_heads=4,
                   width=64, value_width=128, causal=True, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("f32", "bf16", "f16"))
    if rng.random() < 0.4:
        groups = rng.choice((1, 4, 6, 8, 16, 32))
        batch, cams = rng.randint(1, 6), rng.randint(1, 6)
        maps = ["%dx%d" % (_log(rng, 1, 80), _log(rng, 1, 200)) for _ in range(rng.randint(1, 4))]
        channels = groups * rng.choice((3, 4, 5, 8, 12, 16))
        return {k: v for k, v in _norm("", batch=batch, cams=cams, maps=",".join(maps), channels=channels,
                                       groups=groups, type=kind, act=rng.choice(("none", "silu")),
                                       per_scale=rng.random() < 0.5, train=rng.random() < 0.5).items() if k != "name"}
    kv, shared = rng.choice((1, 2, 3, 4)), rng.choice((1, 1, 2, 3, 4))
    width = rng.choice((16, 24, 32, 40, 48, 64))
    serve = rng.random() < 0.3
    queries = rng.randint(1, 4) if serve else _log(rng, 2, 4096)
    keys = _log(rng, 1, 32768) if serve else max(1, int(queries * rng.uniform(0.7, 1.5)))
    causal = rng.random() < 0.6
    keys = max(keys, queries) if causal else keys
    batch = rng.randint(1, 6)
    while batch > 1 and batch * kv * shared * queries * keys > 1 << 28:
        batch -= 1
    frames = 0 if causal or serve else rng.choice((0, 0, 1, 3, 5))
    return {k: v for k, v in _attention("", batch=batch, queries=queries, keys=keys, heads=kv * shared, kv_heads=kv,
                                        width=width, value_width=2 * width, type=kind,
                                        buckets=rng.choice((0, 8, 16, 32)), reach=rng.choice((32, 100, 128)),
                                        causal=causal, frames=frames, key_mask=rng.random() < 0.3,
                                        ragged=serve and rng.random() < 0.6,
                                        train=not serve and rng.random() < 0.6).items() if k != "name"}


# ---------------------------------------------------------------- inputs

def _shapes(case):
    return [tuple(int(n) for n in s.split("x")) for s in case["maps"].split(",")]


def _lengths(case):
    """The caches' lengths: the first is full, the last about half full."""
    return [case["keys"] - (b * case["keys"]) // (2 * case["batch"]) for b in range(case["batch"])]


def _buckets(buckets, reach):
    """Bucket of each relative position -reach..reach (key minus query): one half of the buckets for keys at or
    before the query, one for keys after it; within a half, the first half of the buckets hold one distance each and
    the others grow with the logarithm of the distance, up to `reach`. In whole numbers:
    floor(log(n/e) / log(reach/e) * w) >= t  <=>  n^w * e^t >= reach^t * e^w."""
    half = buckets // 2
    e = max(half // 2, 1)
    w = half - e
    of = []
    for r in range(-reach, reach + 1):
        n = abs(r)
        b = n
        if n >= e:
            b = e + max([t for t in range(1, w) if n ** w * e ** t >= reach ** t * e ** w], default=0)
        of.append(min(b, half - 1) + (half if r > 0 else 0))
    return of


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    kind = DTYPES[case["type"]]

    def normal(*shape, std=1.0, mean=0.0, to=kind):
        t = torch.empty(shape, device=dev, dtype=torch.float32).normal_(mean, std, generator=g)
        return t.to(to)

    s = {"case": case}
    if case["op"] == "norm":
        shapes = _shapes(case)
        K, S, C, B = case["cams"], len(shapes), case["channels"], case["batch"]
        pixels = sum(h * w for h, w in shapes)
        start, at = [], 0
        for _ in range(K):
            for h, w in shapes:
                start.append(at)
                at += h * w
        # Activations of a convolution: each channel with a mean and a spread of its own.
        x = torch.empty((B, K * pixels, C), device=dev).normal_(generator=g)
        x.mul_(normal(C, to=torch.float32).abs() + 0.2).add_(normal(C, to=torch.float32))
        s["x"] = x.to(kind)
        s["shape"] = torch.tensor([shapes] * K, dtype=torch.int32)
        s["start"] = torch.tensor(start, dtype=torch.int32).reshape(K, S)
        affine = (S, C) if case["per_scale"] else (C,)
        s["gamma"] = normal(*affine, std=0.2, mean=1.0, to=torch.float32)
        s["beta"] = normal(*affine, std=0.2, to=torch.float32)
        if case["train"]:
            s["grad"] = normal(B, K * pixels, C, std=0.1)
        return s
    B, Lq, Lk, H, Hk, D, Dv = (case[k] for k in ("batch", "queries", "keys", "heads", "kv_heads", "width", "value_width"))
    s["q"] = normal(B, Lq, H, 2, D)
    s["k"] = normal(B, Lk, Hk, 2, D)
    s["v"] = normal(B, Lk, Hk, Dv)
    s["lam"] = torch.rand(H, device=dev, generator=g) * 0.6 + 0.2
    s["table"] = s["map"] = s["pos_q"] = s["pos_k"] = s["mask"] = s["lengths"] = None
    if case["buckets"]:
        s["table"] = normal(case["buckets"], H, std=0.5, to=torch.float32)
        s["map"] = torch.tensor(_buckets(case["buckets"], case["reach"]), dtype=torch.int32, device=dev)
    if case["frames"]:
        # The queries are of the current frame, 0; the keys of it and of the frames before it, in order.
        s["pos_q"] = torch.zeros(B, Lq, dtype=torch.int32, device=dev)
        back = torch.arange(Lk, device=dev) * case["frames"] // Lk
        s["pos_k"] = (-back).to(torch.int32).expand(B, Lk).contiguous()
    if case["key_mask"]:
        s["mask"] = torch.rand(B, Lk, device=dev, generator=g) < KEPT
        if B > 1:
            s["mask"][B - 1] = False  # no valid instance in this item
    if case["ragged"]:
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
        for b, n in enumerate(_lengths(case)):  # what a cache holds past its length is not to be read
            s["k"][b, n:] = float("nan")
            s["v"][b, n:] = float("nan")
    if case["train"]:
        s["grad"] = normal(B, Lq, H, Dv)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if case["op"] == "norm":
        return _run_norm(state, case)
    return _run_attention(state, case)


def _run_norm(s, case):
    if own:
        import deformable_view_feature_gb300 as da
        y, stats = da.gn_forward(s["x"], s["shape"], s["start"], s["gamma"], s["beta"], case["groups"], EPS, case["act"])
        if not case["train"]:
            return y
        gx, gg, gb = da.gn_backward(s["x"], s["shape"], s["start"], s["gamma"], s["beta"], stats, s["grad"],
                                    case["groups"], case["act"])
        return {"y": y, "grad_x": gx, "grad_gamma": gg, "grad_beta": gb}
    x, G, K = s["x"], case["groups"], case["cams"]
    B, rows, C = x.shape
    x = x.float().reshape(B, K, rows // K, C)
    sizes = [h * w for h, w in _shapes(case)]
    gammas = s["gamma"].expand(len(sizes), C)
    betas = s["beta"].expand(len(sizes), C)
    grads = s["grad"].float().reshape(x.shape).split(sizes, 2) if case["train"] else [None] * len(sizes)
    each = [_plain_norm(*a, G, case["act"]) for a in zip(x.split(sizes, 2), gammas, betas, grads)]
    y = torch.cat([e[0] for e in each], 2).reshape(B, rows, C).to(s["x"].dtype)
    if not case["train"]:
        return y
    gx = torch.cat([e[1] for e in each], 2).reshape(B, rows, C).to(s["x"].dtype)
    gg, gb = torch.stack([e[2] for e in each]), torch.stack([e[3] for e in each])
    if not case["per_scale"]:
        gg, gb = gg.sum(0), gb.sum(0)
    return {"y": y, "grad_x": gx, "grad_gamma": gg, "grad_beta": gb}


def _plain_norm(x, gamma, beta, grad, G, act):
    """One scale's maps [B, K, pixels, C]."""
    B, K, N, C = x.shape
    x = x.reshape(B, K, N, G, C // G)
    gamma, beta = gamma.reshape(G, C // G), beta.reshape(G, C // G)
    over = (2, 4)
    mean = x.mean(over, keepdim=True)
    centred = x - mean
    rstd = (centred.square().mean(over, keepdim=True) + EPS).rsqrt()
    n = centred * rstd
    z = n * gamma + beta
    sig = 1 / (1 + (-z).exp()) if act == "silu" else None
    y = z * sig if act == "silu" else z.clamp(min=0) if act == "relu" else z
    if grad is None:
        return (y.reshape(B, K, N, C),)
    g = grad.reshape(z.shape)
    g = g * (sig * (1 + z * (1 - sig))) if act == "silu" else g * (z > 0) if act == "relu" else g
    gg, gb = (g * n).sum((0, 1, 2)).reshape(C), g.sum((0, 1, 2)).reshape(C)
    g = g * gamma
    gx = rstd * (g - g.mean(over, keepdim=True) - n * (g * n).mean(over, keepdim=True))
    return y.reshape(B, K, N, C), gx.reshape(B, K, N, C), gg, gb


def _places(s, case):
    """The positions of queries [B, Lq] and keys [B, Lk], and which keys there are [B, Lk]."""
    B, Lq, Lk = case["batch"], case["queries"], case["keys"]
    dev = s["q"].device
    length = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), Lk, device=dev)
    at = torch.arange(Lk, device=dev).expand(B, Lk)
    there = at < length[:, None]
    if s["mask"] is not None:
        there = there & s["mask"]
    pk = s["pos_k"].long() if s["pos_k"] is not None else at
    pq = s["pos_q"].long() if s["pos_q"] is not None else torch.arange(Lq, device=dev) + length[:, None] - Lq
    return pq, pk, there


def _run_attention(s, case):
    args = [s[n] for n in ("q", "k", "v", "lam", "table", "map", "pos_q", "pos_k", "mask", "lengths")]
    if own:
        import deformable_view_feature_gb300 as da
        names = ("bias_table", "bucket_map", "pos_q", "pos_k", "key_mask", "key_lengths")
        opt = dict(zip(names, args[4:]), causal=case["causal"])
        if not case["train"]:
            return da.dattn_forward(*args[:4], **opt)
        out, saved = da.dattn_forward(*args[:4], **opt, keep_for_backward=True)
        gq, gk, gv, gl, gt = da.dattn_backward(*args[:4], out, saved, s["grad"], **opt)
        r = {"out": out, "grad_q": gq, "grad_k": gk, "grad_v": gv, "grad_lam": gl}
        return {**r, "grad_table": gt} if s["table"] is not None else r
    B, Lq, H, _, D = s["q"].shape
    Lk, Hk, Dv = s["v"].shape[1:]
    G = H // Hk
    pq, pk, there = _places(s, case)
    rel = pk[:, None, :] - pq[:, :, None]
    see = there[:, None, :] & (rel <= 0) if case["causal"] else there[:, None, :].expand(B, Lq, Lk)
    see = see[:, None, None]
    # Keys that are not there may hold anything.
    k = s["k"].float().masked_fill(~there[:, :, None, None, None], 0)
    v = s["v"].float().masked_fill(~there[:, :, None, None], 0).permute(0, 2, 1, 3)[:, :, None]   # [B, Hk, 1, Lk, Dv]
    q = s["q"].float().reshape(B, Lq, Hk, G, 2, D)
    q1, q2 = (q[..., m, :].permute(0, 2, 3, 1, 4) for m in (0, 1))                # [B, Hk, G, Lq, D]
    k1, k2 = (k[:, :, :, m].permute(0, 2, 1, 3)[:, :, None] for m in (0, 1))      # [B, Hk, 1, Lk, D]
    lam = s["lam"].reshape(1, Hk, G, 1, 1)
    bias = None
    if s["table"] is not None:
        reach = case["reach"]
        bucket = s["map"].long()[rel.clamp(-reach, reach) + reach]                # [B, Lq, Lk]
        bias = s["table"].t().reshape(Hk, G, -1)[:, :, bucket].permute(2, 0, 1, 3, 4)
    scale = D ** -0.5
    p1, p2 = (_plain_softmax(a, b, scale, bias, see) for a, b in ((q1, k1), (q2, k2)))
    out = (p1 - lam * p2) @ v
    kind = s["q"].dtype

    def rows(t):  # [B, Hk, G, Lq, X] -> [B, Lq, H, X]
        return t.permute(0, 3, 1, 2, 4).reshape(B, Lq, H, -1)

    if not case["train"]:
        return rows(out).to(kind)
    g = s["grad"].float().reshape(B, Lq, Hk, G, Dv).permute(0, 2, 3, 1, 4)
    gv = ((p1 - lam * p2).transpose(-1, -2) @ g).sum(2).transpose(1, 2)
    gp = g @ v.transpose(-1, -2)
    gl = -(p2 * gp).sum((0, 3, 4)).reshape(H)
    s1 = p1 * (gp - (p1 * gp).sum(-1, keepdim=True))
    s2 = -lam * p2 * (gp - (p2 * gp).sum(-1, keepdim=True))
    gq = torch.stack([rows(s1 @ k1), rows(s2 @ k2)], 3) * scale
    gk = torch.stack([(t.transpose(-1, -2) @ a).sum(2).transpose(1, 2) for t, a in ((s1, q1), (s2, q2))], 3) * scale
    r = {"out": rows(out).to(kind), "grad_q": gq.to(kind), "grad_k": gk.to(kind), "grad_v": gv.to(kind), "grad_lam": gl}
    if bias is not None:
        # Query by query as a product with the buckets' indicators, then over the queries in 64 bits.
        each = (bucket[..., None] == torch.arange(case["buckets"], device=bucket.device)).float()  # [B, Lq, Lk, buckets]
        both = (s1 + s2).reshape(B, H, Lq, Lk).transpose(1, 2) @ each
        r["grad_table"] = both.double().sum((0, 1)).t().float()
    return r


def _plain_softmax(q, k, scale, bias, see):
    """Softmax over the keys that are seen; zeros where none is."""
    t = q @ k.transpose(-1, -2) * scale
    if bias is not None:
        t = t + bias
    t = t.masked_fill(~see, float("-inf"))
    top = t.amax(-1, keepdim=True)
    e = (t - top.masked_fill(top == float("-inf"), 0)).exp()
    return e / e.sum(-1, keepdim=True).clamp(min=1e-30)


# ---------------------------------------------------------------- the least work

def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "norm":
        n = case["batch"] * case["cams"] * sum(h * w for h, w in _shapes(case)) * case["channels"]
        return {"bytes": n * size * (4 if case["train"] else 2), "flops": n * (30 if case["train"] else 10)}
    B, Lq, Lk, H, Hk, D, Dv = (case[k] for k in ("batch", "queries", "keys", "heads", "kv_heads", "width", "value_width"))
    lengths = _lengths(case) if case["ragged"] else [Lk] * B
    if case["key_mask"] and B > 1:
        lengths = lengths[:-1]
    keep = KEPT if case["key_mask"] else 1.0
    unseen = lambda n: Lq * n - min(n, Lq) * (2 * n - min(n, Lq) + 1) // 2 if case["causal"] else 0  # noqa: E731
    pairs = sum(keep * (Lq * n - unseen(n)) for n in lengths) * H
    of_q, of_k = B * Lq * H * (2 * D + Dv), keep * sum(lengths) * Hk * (2 * D + Dv)
    times = 2 if case["train"] else 1  # every input read once, its gradient or the output written once
    return {"bytes": int(size * times * (of_q + of_k)), "flops": int(pairs * (4 * D + 2 * Dv + (times - 1) * (12 * D + 4 * Dv)))}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s, case) if case["op"] == "norm" else _exact_attention(s, case)


def _exact_norm(s, case):
    """Map by map, the gradients by automatic differentiation of the definition."""
    gamma, beta = (s[n].double().requires_grad_(case["train"]) for n in ("gamma", "beta"))
    shapes, G = _shapes(case), case["groups"]
    y, gx = (torch.empty(s["x"].shape, dtype=torch.float64, device=s["x"].device) for _ in range(2))
    gg, gb = torch.zeros_like(gamma), torch.zeros_like(beta)
    for k in range(case["cams"]):
        for i, (h, w) in enumerate(shapes):
            at = int(s["start"][k, i])
            part = slice(at, at + h * w)
            x = s["x"][:, part].double().requires_grad_(case["train"])
            t = x.reshape(x.shape[0], h * w, G, -1)
            var, mean = torch.var_mean(t, (1, 3), correction=0, keepdim=True)
            z = ((t - mean) / (var + EPS).sqrt()).reshape(x.shape)
            z = z * (gamma[i] if case["per_scale"] else gamma) + (beta[i] if case["per_scale"] else beta)
            z = z * torch.sigmoid(z) if case["act"] == "silu" else torch.relu(z) if case["act"] == "relu" else z
            y[:, part] = z.detach()
            if case["train"]:
                a, b, c = torch.autograd.grad(z, (x, gamma, beta), s["grad"][:, part].double())
                gx[:, part] = a
                gg += b
                gb += c
    return {"y": y, "grad_x": gx, "grad_gamma": gg.detach(), "grad_beta": gb.detach()} if case["train"] else y


def _exact_attention(s, case):
    """Head by head and in rows of at most 1024 queries, the gradients by automatic differentiation."""
    B, Lq, H, _, D = s["q"].shape
    Hk, Dv = s["v"].shape[2:]
    if B * H * Lq * case["keys"] > 1 << 31:
        return None
    pq, pk, there = _places(s, case)
    new = {n: torch.zeros(s[n].shape, dtype=torch.float64, device=s["q"].device) for n in ("q", "k", "v", "lam")}
    out = torch.zeros(B, Lq, H, Dv, dtype=torch.float64, device=s["q"].device)
    table = torch.zeros(s["table"].shape, dtype=torch.float64, device=s["q"].device) if s["table"] is not None else None
    for b in range(B):
        keys = there[b].nonzero()[:, 0]
        if keys.numel() == 0:
            continue
        for h in range(H):
            n = h * Hk // H
            for at in range(0, Lq, 1024):
                part = slice(at, min(at + 1024, Lq))
                q = s["q"][b, part, h].double().requires_grad_(case["train"])
                k = s["k"][b, keys, n].double().requires_grad_(case["train"])
                v = s["v"][b, keys, n].double().requires_grad_(case["train"])
                lam = s["lam"][h].double().requires_grad_(case["train"])
                leaves = [q, k, v, lam]
                rel = pk[b, keys][None, :] - pq[b, part][:, None]
                t = torch.einsum("imd,jmd->mij", q, k) / math.sqrt(D)
                if table is not None:
                    w = s["table"][:, h].double().requires_grad_(case["train"])
                    leaves.append(w)
                    t = t + w[s["map"].long()[rel.clamp(-case["reach"], case["reach"]) + case["reach"]]]
                if case["causal"]:
                    t = t.masked_fill(rel > 0, float("-inf"))
                    t = t.masked_fill((rel > 0).all(1)[None, :, None], 0.0)
                    none = (rel > 0).all(1)[:, None]
                else:
                    none = torch.zeros(rel.shape[0], 1, dtype=torch.bool, device=rel.device)
                p = torch.softmax(t, -1)
                o = ((p[0] - lam * p[1]) @ v).masked_fill(none, 0.0)
                out[b, part, h] = o.detach()
                if case["train"]:
                    grads = torch.autograd.grad(o, leaves, s["grad"][b, part, h].double())
                    new["q"][b, part, h] = grads[0]
                    new["k"][b, :, n].index_add_(0, keys, grads[1])
                    new["v"][b, :, n].index_add_(0, keys, grads[2])
                    new["lam"][h] += grads[3]
                    if table is not None:
                        table[:, h] += grads[4]
    if not case["train"]:
        return out
    r = {"out": out, "grad_q": new["q"], "grad_k": new["k"], "grad_v": new["v"], "grad_lam": new["lam"]}
    return {**r, "grad_table": table} if table is not None else r
