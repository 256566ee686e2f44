"""What the rotary norm of queries and keys, the paged cache and the attention over it are measured on.

Three families of cases, as they occur around the differential attention:

* ``rotary``: every head's query and key vectors normalised and rotated by
  their positions, forward alone or with the backward pass.
* ``append``: new tokens' keys, normalised and rotated, and values stored into
  a paged cache, their queries normalised and rotated on the way.
* ``attend``: differential attention of new tokens (one each, a prompt's next
  part, a tree of drafted ones) over such a cache.

``run`` with ``own`` false computes each in plain elementary operations in 32
bits; with ``own`` true it calls the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
KEPT = 0.85  # share of the keys that a key mask keeps


def _rotary(name, **kw):
    return {"name": name, "op": "rotary", "batch": 1, "queries": 900, "keys": 900, "heads": 4, "kv_heads": 4, "width": 32,
            "rotated": 32, "type": "bf16", "interleaved": False, "base": 10000.0, "stretch": 1.0, "magnitude": 1.0,
            "weights": True, "places": "index", "train": False, **kw}


def _append(name, **kw):
    return {"name": name, "op": "append", "batch": 1, "tokens": 1, "capacity": 128, "page": 16, "heads": 4, "kv_heads": 4,
            "width": 32, "value_width": 64, "rotated": 32, "type": "bf16", "interleaved": False, "base": 10000.0,
            "stretch": 1.0, "magnitude": 1.0, "weights": True, "ragged": False, **kw}


def _attend(name, **kw):
    return {"name": name, "op": "attend", "batch": 1, "tokens": 1, "keys": 77, "page": 16, "heads": 4, "kv_heads": 4,
            "width": 32, "value_width": 64, "type": "bf16", "buckets": 0, "reach": 128, "tree": False, "key_mask": False,
            "ragged": False, **kw}


def listed():
    return [
        # One new token of a small head: the launch and the host's work are what counts.
        _rotary("rotary, one token", queries=1, keys=1),
        # Instances of frames, in 32 bits, whose heads rotate 16 of 24 channels, in pairs of neighbours.
        _rotary("rotary, frames training", batch=6, queries=900, keys=2100, heads=6, kv_heads=2, width=24, rotated=16,
                type="f32", interleaved=True, places="frames", train=True),
        # A long prompt whose positions are far out, with stretched angles, in half precision.
        _rotary("rotary, far prompt", queries=4095, keys=4095, heads=16, kv_heads=4, width=64, rotated=64, type="f16",
                stretch=8.0, magnitude=1.2, places="far"),
        # The attention's long sequences trained: far larger than what latency hides.
        _rotary("rotary, long sequence training", batch=2, queries=8192, keys=8192, heads=8, kv_heads=4, width=64,
                rotated=64, train=True),
        # Serving: one token each for a batch.
        _append("append, one token each", batch=64, capacity=2048, heads=16, kv_heads=4, width=64, value_width=128,
                rotated=64),
        # Instances of a frame in 32 bits, a padded batch, pages that are no power of two.
        _append("append, padded frames", batch=5, tokens=301, capacity=1300, page=20, heads=6, kv_heads=2, width=24,
                value_width=48, rotated=16, type="f32", interleaved=True, ragged=True),
        # Prompts that are taken in at once.
        _append("append, prompts", batch=4, tokens=4095, capacity=8192, page=64, heads=8, kv_heads=4, width=64,
                value_width=128, rotated=64, type="f16"),
        # One new token against a short history: latency.
        _attend("attend, one token"),
        # Serving: one token each for a batch with long, ragged caches and shared key heads.
        _attend("attend, long caches", batch=8, keys=32768, page=64, heads=16, kv_heads=4, width=64, value_width=128,
                ragged=True),
        # Drafted trees over ragged caches of small pages, with a bias by distance.
        _attend("attend, drafted trees", batch=4, tokens=31, keys=8191, heads=8, kv_heads=2, width=64, value_width=128,
                type="f16", buckets=32, tree=True, ragged=True),
        # The next part of a padded batch of prompts, of odd lengths.
        _attend("attend, prompts", batch=2, tokens=1021, keys=8001, page=32, heads=8, kv_heads=2, width=64,
                value_width=128, ragged=True),
        # Some instances over their history in 32 bits, some of it invalid; pages that are no power of two.
        _attend("attend, instances", batch=6, tokens=60, keys=2100, page=20, width=32, value_width=64, type="f32",
                key_mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "append", "attend", "attend"))
    kv, shared = rng.choice((1, 2, 3, 4)), rng.choice((1, 1, 2, 3, 4))
    width = rng.choice((16, 24, 32, 40, 48, 64))
    d = dict(batch=rng.randint(1, 8), heads=kv * shared, kv_heads=kv, width=width, type=rng.choice(("f32", "bf16", "f16")))
    if op != "attend":
        d.update(rotated=rng.choice((width, width, width // 2)), interleaved=rng.random() < 0.4,
                 base=rng.choice((10000.0, 500000.0)), weights=rng.random() < 0.8)
        d.update(stretch=rng.choice((1.0, 1.0, 4.0)), magnitude=rng.choice((1.0, 1.0, 1.1)))
    if op == "rotary":
        keys = _log(rng, 1, 8192)
        queries = keys if rng.random() < 0.6 else max(1, int(keys * rng.uniform(0.1, 1.0)))
        d.update(queries=queries, keys=keys, places=rng.choice(("index", "index", "far", "frames")), train=rng.random() < 0.5)
        made = _rotary("", **d)
    elif op == "append":
        tokens = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
        d.update(tokens=tokens, capacity=tokens + _log(rng, 1, 4096), page=rng.choice((8, 16, 20, 32, 64, 128)),
                 value_width=2 * width, ragged=rng.random() < 0.4)
        if tokens == 1:
            d["batch"] = _log(rng, 1, 64)
        made = _append("", **d)
    else:
        tokens = 1 if rng.random() < 0.4 else _log(rng, 2, 64) if rng.random() < 0.6 else _log(rng, 64, 1024)
        tree = 1 < tokens <= 64 and rng.random() < 0.6
        keys = tokens + _log(rng, 1, 32768 if tokens <= 64 else 8192)
        d.update(tokens=tokens, keys=keys, page=rng.choice((8, 16, 20, 32, 64, 128)), value_width=2 * width, tree=tree,
                 buckets=rng.choice((0, 0, 8, 32)), reach=rng.choice((32, 100, 128)), ragged=rng.random() < 0.6,
                 key_mask=rng.random() < 0.2)
        made = _attend("", **d)
    # No more than the largest of the listed ones.
    most = {"rotary": 2.0e8, "append": 1.3e8, "attend": 4.0e8}[op]
    while True:
        w = work(made)
        if w["bytes"] <= most and w["flops"] <= 4.8e10:
            return {k: v for k, v in made.items() if k != "name"}
        long = "keys" if "keys" in made else "tokens"
        if made["batch"] > 1:
            made["batch"] -= 1
        else:
            made[long] = made[long] * 3 // 4
            for short in ("tokens", "queries"):
                if short in made:
                    made[short] = min(made[short], made[long])


# ---------------------------------------------------------------- inputs

def _counts(case):
    """The new tokens of each item: the first has all, the last about half of them."""
    B, T = case["batch"], case["tokens"]
    return [T - (b * T) // (2 * B) if case["ragged"] else T for b in range(B)]


def _lengths(case):
    """The keys of each item, its new ones among them: the first's cache is full, the last's about half full."""
    B, n = case["batch"], case["keys"]
    return [max(n - (b * n) // (2 * B), c) if case["ragged"] else n for b, c in enumerate(_counts(case))]


def _before(case):
    """The tokens that an item's cache holds before new ones are appended, none in the second item's."""
    B, room = case["batch"], case["capacity"] - case["tokens"]
    return [room - (b * room) // (2 * B) if b != 1 else 0 for b in range(B)]


def _frequencies(case):
    """Angle for each position of each rotated pair, in radians."""
    n = case["rotated"] // 2
    return [case["base"] ** (-i / n) / case["stretch"] for i in range(n)]


def _buckets(buckets, reach):
    """Bucket of each relative position -reach..reach (key minus query): one half of the buckets for keys at or
    before the query, one for keys after it; half of each hold one distance each, the others grow with the logarithm
    of the distance, in whole numbers."""
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
        return torch.empty(shape, device=dev, dtype=torch.float32).normal_(mean, std, generator=g).to(to)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi, shape, device=dev, dtype=torch.int32, generator=g)

    s = {"case": case}
    B, H, Hk, D = (case[k] for k in ("batch", "heads", "kv_heads", "width"))
    if case["op"] != "attend":
        # What a model keeps: its angles for each position, as radians and in units of 2^-64 of a turn, and its weights.
        f = _frequencies(case)
        s["radians"] = torch.tensor(f, dtype=torch.float64, device=dev)
        s["turns"] = torch.tensor([round(x / (2 * math.pi) * 2 ** 64) for x in f], dtype=torch.int64, device=dev)
        s["wq"], s["wk"] = (normal(D, std=0.2, mean=1.0, to=torch.float32) if case["weights"] else None for _ in range(2))
    if case["op"] == "rotary":
        Lq, Lk = case["queries"], case["keys"]
        s["q"], s["k"] = normal(B, Lq, H, 2, D, std=2.0), normal(B, Lk, Hk, 2, D, std=0.5)
        s["pos_q"] = s["pos_k"] = None
        if case["places"] == "far":  # the sequences begin anywhere in a long context
            begin = whole(0, 1 << 20, B, 1)
            s["pos_k"] = (begin + torch.arange(Lk, device=dev, dtype=torch.int32)).contiguous()
            s["pos_q"] = s["pos_k"][:, Lk - Lq:].contiguous() if Lq <= Lk else whole(0, 1 << 20, B, Lq)
        elif case["places"] == "frames":  # queries of the current frame, keys of it and of the four before it
            s["pos_q"] = torch.zeros(B, Lq, dtype=torch.int32, device=dev)
            s["pos_k"] = (-(torch.arange(Lk, device=dev) * 5 // Lk)).to(torch.int32).expand(B, Lk).contiguous()
        if case["train"]:
            s["gq"], s["gk"] = normal(B, Lq, H, 2, D, std=0.1), normal(B, Lk, Hk, 2, D, std=0.1)
        return s
    T, page, Dv = case["tokens"], case["page"], case["value_width"]
    room = case["capacity"] if case["op"] == "append" else case["keys"]
    each = -(-room // page)                # pages of an item
    pages = B * each + 3
    s["k_cache"] = normal(pages, page, Hk, 2, D)
    s["v_cache"] = normal(pages, page, Hk, Dv)
    # The items' pages lie anywhere; those past an item's tokens are not there yet.
    table = torch.randperm(pages, device=dev, generator=g)[: B * each].to(torch.int32).reshape(B, each)
    used = [b + c for b, c in zip(_before(case), _counts(case))] if case["op"] == "append" else _lengths(case)
    for b, n in enumerate(used):
        table[b, -(-n // page):] = -1
    s["table"] = table
    s["q"] = normal(B, T, H, 2, D, std=2.0 if case["op"] == "append" else 1.0)
    s["counts"] = torch.tensor(_counts(case), dtype=torch.int32, device=dev) if case["ragged"] else None
    if case["op"] == "append":
        s["k"], s["v"] = normal(B, T, Hk, 2, D, std=0.5), normal(B, T, Hk, Dv)
        s["before"] = torch.tensor(_before(case), dtype=torch.int32, device=dev)
        return s
    L = each * page
    lengths = _lengths(case)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["lam"] = torch.rand(H, device=dev, generator=g) * 0.6 + 0.2
    s["bias"] = s["map"] = s["pos_q"] = s["pos_k"] = s["mask"] = s["tree"] = None
    if case["buckets"]:
        s["bias"] = normal(case["buckets"], H, std=0.5, to=torch.float32)
        s["map"] = torch.tensor(_buckets(case["buckets"], case["reach"]), dtype=torch.int32, device=dev)
    old = [n - c for n, c in zip(lengths, _counts(case))]
    if case["tree"]:
        # Each drafted token continues one of those before it, mostly one of the last; it stands one position after that.
        sees = torch.eye(T, dtype=torch.bool).expand(B, T, T).clone()
        depth = torch.zeros(B, T, dtype=torch.int32)
        pick = torch.rand(B, T, device=dev, generator=g).cpu()
        for i in range(1, T):
            parent = (i - 1 - (pick[:, i] ** 2 * min(i, 6)).long()).clamp(min=0)
            rows = torch.arange(B)
            sees[:, i] |= sees[rows, parent]
            depth[:, i] = depth[rows, parent] + 1
        s["tree"] = sees.to(dev)
        s["pos_q"] = depth.to(dev) + torch.tensor(old, dtype=torch.int32, device=dev)[:, None]
        s["pos_k"] = torch.arange(L, dtype=torch.int32, device=dev).expand(B, L).contiguous()
        for b, n in enumerate(lengths):
            s["pos_k"][b, old[b]: n] = s["pos_q"][b, : n - old[b]]
    if case["key_mask"]:
        s["mask"] = torch.rand(B, L, device=dev, generator=g) < KEPT
        if B > 1:
            s["mask"][B - 1] = False  # no valid instance in this item
    # What the cache holds where no key is is not to be read.
    hold = torch.zeros(pages * page, dtype=torch.bool, device=dev)
    for b, n in enumerate(lengths):
        at = torch.arange(n, device=dev)
        hold[table[b].long()[at // page] * page + at % page] = True
    s["k_cache"].view(pages * page, -1)[~hold] = float("nan")
    s["v_cache"].view(pages * page, -1)[~hold] = float("nan")
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    return {"rotary": _run_rotary, "append": _run_append, "attend": _run_attend}[case["op"]](state, case)


def _run_rotary(s, case):
    if own:
        import deformable_view_feature_gb300 as da
        opt = dict(frequencies=s["turns"], q_weight=s["wq"], k_weight=s["wk"], pos_q=s["pos_q"], pos_k=s["pos_k"], eps=EPS,
                   interleaved=case["interleaved"], magnitude=case["magnitude"])
        q, k = da.qkr_forward(s["q"], s["k"], **opt)
        if not case["train"]:
            return {"q": q, "k": k}
        gq, gk, gwq, gwk = da.qkr_backward(s["q"], s["k"], s["gq"], s["gk"], **opt)
        r = {"q": q, "k": k, "grad_q": gq, "grad_k": gk}
        return {**r, "grad_q_weight": gwq, "grad_k_weight": gwk} if case["weights"] else r
    r = {}
    Lq, Lk = case["queries"], case["keys"]
    for x, L, first in (("q", Lq, Lk - Lq), ("k", Lk, 0)):
        pos = s["pos_" + x]
        if pos is None:
            pos = torch.arange(L, device=s[x].device)[None] + first
        cos, sin = _angles(pos, s, case)
        n, rstd = _plain_norm(s[x])
        w = s["w" + x]
        r[x] = _plain_turn(n if w is None else n * w, cos, sin, case).to(s[x].dtype)
        if case["train"]:
            g = _plain_turn(s["g" + x].float(), cos, -sin, case)
            if w is not None:
                r["grad_" + x + "_weight"] = (g * n).sum((0, 1, 2, 3))
                g = g * w
            r["grad_" + x] = (rstd * (g - n * (g * n).mean(-1, keepdim=True))).to(s[x].dtype)
    return r


def _angles(pos, s, case):
    """cos and sin [B, L, 1, 1, rotated / 2] of the positions [B, L], the angles in 64 bits."""
    a = (pos.double()[..., None] * s["radians"])[:, :, None, None]
    return (a.cos() * case["magnitude"]).float(), (a.sin() * case["magnitude"]).float()


def _plain_norm(x):
    x = x.float()
    rstd = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * rstd, rstd


def _plain_turn(x, cos, sin, case):
    R = case["rotated"]
    rest = x[..., R:]
    if case["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        both = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        both = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([both, rest], -1)


def _run_append(s, case):
    if own:
        import deformable_view_feature_gb300 as da
        q = da.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["before"], counts=s["counts"], q=s["q"],
                            frequencies=s["turns"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                            interleaved=case["interleaved"], magnitude=case["magnitude"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    B, T, page = case["batch"], case["tokens"], case["page"]
    t = torch.arange(T, device=s["q"].device)
    place = s["before"].long()[:, None] + t                                   # [B, T]
    cos, sin = _angles(place, s, case)
    new = {}
    for x in ("q", "k"):
        n, w = _plain_norm(s[x])[0], s["w" + x]
        new[x] = _plain_turn(n if w is None else n * w, cos, sin, case).to(s[x].dtype)
    each = s["table"].shape[1]
    at = s["table"].long().gather(1, (place // page).clamp(max=each - 1)), place % page
    k, v = new["k"], s["v"]
    if s["counts"] is not None:
        there = t < s["counts"][:, None]
        at, k, v = (at[0][there], at[1][there]), k[there], v[there]
    s["k_cache"][at] = k
    s["v_cache"][at] = v
    return {"q": new["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _sees(s, case):
    """Which keys [B, T, L] each new token sees, and their relative positions, L the places of the pages."""
    B, T = case["batch"], case["tokens"]
    L = s["table"].shape[1] * case["page"]
    dev = s["q"].device
    length = s["lengths"].long()[:, None]
    count = s["counts"].long()[:, None] if s["counts"] is not None else torch.full((B, 1), T, device=dev)
    at, t = torch.arange(L, device=dev).expand(B, L), torch.arange(T, device=dev).expand(B, T)
    there = at < length
    if s["mask"] is not None:
        there = there & s["mask"]
    pk = s["pos_k"].long() if s["pos_k"] is not None else at
    pq = s["pos_q"].long() if s["pos_q"] is not None else length - count + t
    rel = pk[:, None, :] - pq[:, :, None]
    see = there[:, None, :] & (t < count)[:, :, None]
    if s["tree"] is None:
        return see & (rel <= 0), rel
    new = at - (length - count)                                               # which of the new tokens a key is of
    tree = s["tree"].gather(2, new.clamp(0, T - 1)[:, None].expand(B, T, L))
    return see & ((new < 0)[:, None] | tree), rel


def _run_attend(s, case):
    if own:
        import deformable_view_feature_gb300 as da
        return da.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["lam"], s["table"], s["lengths"], counts=s["counts"],
                                  tree=s["tree"], bias_table=s["bias"], bucket_map=s["map"], pos_q=s["pos_q"],
                                  pos_k=s["pos_k"], key_mask=s["mask"])
    B, T, H, _, D = s["q"].shape
    Hk, Dv = s["v_cache"].shape[2:]
    G = H // Hk
    see, rel = _sees(s, case)
    table = s["table"].long().clamp(min=0)
    used = see.any(1)                                                         # [B, L]; what is elsewhere may be anything
    k = s["k_cache"][table].flatten(1, 2).float().masked_fill(~used[:, :, None, None, None], 0)
    v = s["v_cache"][table].flatten(1, 2).float().masked_fill(~used[:, :, None, None], 0).permute(0, 2, 1, 3)[:, :, None]
    q = s["q"].float().reshape(B, T, Hk, G, 2, D)
    bias = None
    if s["bias"] is not None:
        reach = case["reach"]
        bucket = s["map"].long()[rel.clamp(-reach, reach) + reach]            # [B, T, L]
        bias = s["bias"].t().reshape(Hk, G, -1)[:, :, bucket].permute(2, 0, 1, 3, 4)
    p = []
    for m in (0, 1):
        t = q[..., m, :].permute(0, 2, 3, 1, 4) @ k[:, :, :, m].permute(0, 2, 3, 1)[:, :, None] * D ** -0.5
        if bias is not None:
            t = t + bias
        t = t.masked_fill(~see[:, None, None], float("-inf"))
        top = t.amax(-1, keepdim=True)
        e = (t - top.masked_fill(top == float("-inf"), 0)).exp()
        p.append(e / e.sum(-1, keepdim=True).clamp(min=1e-30))
    out = (p[0] - s["lam"].reshape(1, Hk, G, 1, 1) * p[1]) @ v                # [B, Hk, G, T, Dv]
    return out.permute(0, 3, 1, 2, 4).reshape(B, T, H, Dv).to(s["q"].dtype)


# ---------------------------------------------------------------- the least work

def work(case):
    size = 4 if case["type"] == "f32" else 2
    B, H, Hk, D = (case[k] for k in ("batch", "heads", "kv_heads", "width"))
    if case["op"] == "rotary":
        n = B * (case["queries"] * H + case["keys"] * Hk) * 2 * D
        return {"bytes": n * size * (4 if case["train"] else 2), "flops": n * (20 if case["train"] else 8)}
    T, Dv = case["tokens"], case["value_width"]
    if case["op"] == "append":
        new = sum(_counts(case)) * Hk * (2 * D + Dv)
        return {"bytes": 2 * size * (B * T * H * 2 * D + new), "flops": 8 * (B * T * H * 2 * D + new)}
    counts, lengths = _counts(case), _lengths(case)
    if case["key_mask"] and B > 1:
        lengths = lengths[:-1]
    keep = KEPT if case["key_mask"] else 1.0
    pairs = keep * H * sum(c * n - c * (c - 1) // 2 for c, n in zip(counts, lengths))
    return {"bytes": int(size * (sum(counts) * H * (2 * D + Dv) + keep * sum(lengths) * Hk * (2 * D + Dv))),
            "flops": int(pairs * (4 * D + 2 * Dv))}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "append": _exact_append, "attend": _exact_attend}[case["op"]](s, case)


def _exact_vectors(x, w, pos, s, case):
    """The definition as complex numbers: x [B, L, heads, 2, D] in 64 bits, pos [B, L]."""
    R = case["rotated"]
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    if w is not None:
        y = y * w
    turn = torch.polar(torch.full((), case["magnitude"], dtype=torch.float64, device=x.device).expand(*pos.shape, R // 2),
                       pos.double()[..., None] * s["radians"])[:, :, None, None]
    part = y[..., :R].unflatten(-1, (R // 2, 2) if case["interleaved"] else (2, R // 2))
    at = -1 if case["interleaved"] else -2
    z = torch.complex(part.select(at, 0), part.select(at, 1)) * turn
    return torch.cat([torch.stack([z.real, z.imag], at).flatten(-2), y[..., R:]], -1)


def _exact_rotary(s, case):
    r = {}
    Lq, Lk = case["queries"], case["keys"]
    for x, L, first in (("q", Lq, Lk - Lq), ("k", Lk, 0)):
        pos = s["pos_" + x] if s["pos_" + x] is not None else (torch.arange(L, device=s[x].device) + first).expand(case["batch"], L)
        leaves = [s[x].double().requires_grad_(case["train"])]
        w = None
        if s["w" + x] is not None:
            w = s["w" + x].double().requires_grad_(case["train"])
            leaves.append(w)
        y = _exact_vectors(leaves[0], w, pos, s, case)
        r[x] = y.detach()
        if case["train"]:
            grads = torch.autograd.grad(y, leaves, s["g" + x].double())
            r["grad_" + x] = grads[0]
            if w is not None:
                r["grad_" + x + "_weight"] = grads[1]
    return r


def _exact_append(s, case):
    """Item by item."""
    B, T, page = case["batch"], case["tokens"], case["page"]
    place = torch.tensor(_before(case), device=s["q"].device)[:, None] + torch.arange(T, device=s["q"].device)
    q, k = (_exact_vectors(s[x].double(), None if s["w" + x] is None else s["w" + x].double(), place, s, case) for x in ("q", "k"))
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for b, n in enumerate(_counts(case)):
        row = s["table"][b].long()[place[b, :n] // page] * page + place[b, :n] % page
        kc.view(-1, *kc.shape[2:])[row] = k[b, :n]
        vc.view(-1, *vc.shape[2:])[row] = s["v"][b, :n].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _exact_attend(s, case):
    """Head by head and in rows of at most 512 tokens."""
    B, T, H, _, D = s["q"].shape
    Hk, Dv = s["v_cache"].shape[2:]
    if B * H * T * case["keys"] > 1 << 29:
        return None
    out = torch.zeros(B, T, H, Dv, dtype=torch.float64, device=s["q"].device)
    dev, page = s["q"].device, case["page"]
    for b, (n, c) in enumerate(zip(_lengths(case), _counts(case))):
        j = torch.arange(n, device=dev)
        if s["mask"] is not None:
            j = j[s["mask"][b, :n]]
        if j.numel() == 0:
            continue
        row = s["table"][b].long()[j // page] * page + j % page
        pk = s["pos_k"][b].long()[j] if s["pos_k"] is not None else j
        pq = s["pos_q"][b].long() if s["pos_q"] is not None else n - c + torch.arange(T, device=dev)
        for at in range(0, c, 512):
            i = torch.arange(at, min(at + 512, c), device=dev)
            rel = pk[None, :] - pq[i][:, None]
            if s["tree"] is not None:
                hidden = (j >= n - c)[None, :] & ~s["tree"][b][i][:, (j - (n - c)).clamp(min=0)]
            else:
                hidden = rel > 0
            none = hidden.all(1)[:, None]
            for h in range(H):
                k = s["k_cache"].flatten(0, 1)[row, h * Hk // H].double()
                v = s["v_cache"].flatten(0, 1)[row, h * Hk // H].double()
                t = torch.einsum("imd,jmd->mij", s["q"][b, i, h].double(), k) / math.sqrt(D)
                if s["bias"] is not None:
                    t = t + s["bias"][:, h].double()[s["map"].long()[rel.clamp(-case["reach"], case["reach"]) + case["reach"]]]
                p = torch.softmax(t.masked_fill(hidden, float("-inf")).masked_fill(none, 0.0), -1)
                out[b, i, h] = ((p[0] - s["lam"][h].double() * p[1]) @ v).masked_fill(none, 0.0)
    return out
