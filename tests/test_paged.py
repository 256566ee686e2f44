"""The paged cache (paged_append) and the attention over it (paged_attention):
refusals on the CPU, results on the GPU against 64 bits."""
import ctypes

import pytest
import torch

import deformable_view_feature_gb300 as da
from operator_refs import check
from serving_refs import PgCache, PgProblem, QkrProblem, paged_reference, qkr_reference, serving_library

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FAKE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    da.build.build()
    return serving_library(da.load_library())


# ---- refusals and host logic: no GPU, nothing is launched ------------------

def _fake_cache(**kw):
    d = dict(k=FAKE, v=FAKE, num_pages=9, page_size=16, table_pages=4, page_table=FAKE, lengths=FAKE)
    d.update(kw)
    c = PgCache(**d)
    c.k_stride[:] = (2048, 128, 64, 32)
    c.v_stride[:] = (2048, 128, 64)
    return c


def _problem(cache=None, q_stride=(1024, 256, 64, 32), **kw):
    d = dict(batch=2, num_tokens=4, num_heads=4, num_kv_heads=2, width=32, value_width=64, dtype=1, num_buckets=8, reach=16, causal=1,
             scale=0.1, q=FAKE, lam=FAKE, bias_table=FAKE, bucket_map=FAKE)
    d.update(kw)
    p = PgProblem(**d)
    p.q_stride[:] = q_stride
    p.cache = _fake_cache(**(cache or {}))
    return p


CACHE_FAULTS = [
    (dict(num_pages=-1), 2), (dict(table_pages=-1), 2), (dict(page_size=0), 2), (dict(table_pages=1 << 25), 4), (dict(k=FAKE + 1), 3),
    (dict(v=FAKE + 1), 3), (dict(page_table=FAKE + 2), 3), (dict(lengths=FAKE + 1), 3), (dict(counts=FAKE + 2), 3), (dict(lengths=None), 1),
    (dict(page_table=None), 1),
]


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(batch=-1), 2), (dict(num_tokens=-1), 2), (dict(num_heads=3), 2), (dict(num_kv_heads=0), 2), (dict(width=0), 2),
    (dict(width=129), 4), (dict(value_width=257), 4), (dict(dtype=5), 2), (dict(scale=float("nan")), 2), (dict(num_buckets=-1), 2),
    (dict(reach=0), 2), (dict(reach=2000), 4), (dict(num_buckets=300), 4), (dict(num_buckets=0, reach=0), 0), (dict(batch=70000), 4),
    (dict(num_tokens=1 << 29), 4), (dict(q_stride=(1024, -256, 64, 32)), 2),
] + [(dict(cache=c), s) for c, s in CACHE_FAULTS])
def test_sizes_are_checked(lib, kw, status):
    assert lib.pg_workspace_size(ctypes.byref(_problem(**kw)), ctypes.byref(ctypes.c_size_t(0))) == status


def test_buffers_are_checked(lib):
    vp = ctypes.c_void_p
    n = ctypes.c_size_t(0)
    p = _problem(cache=dict(table_pages=400))
    assert lib.pg_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0

    def call(p=p, out=FAKE, ws=FAKE, size=n.value):
        return lib.pg_attention(ctypes.byref(p), vp(out), vp(ws), size, None)

    for kw in (dict(q=None), dict(lam=None), dict(bias_table=None), dict(bucket_map=None), dict(cache=dict(k=None)), dict(cache=dict(v=None))):
        assert call(_problem(**kw)) == 1, kw
    assert call(out=None) == 1 and call(out=FAKE + 1) == 3 and call(_problem(q=FAKE + 1)) == 3 and call(_problem(pos_k=FAKE + 1)) == 3
    assert call(size=n.value - 1) == 6 and call(ws=None) == 6 and call(ws=FAKE + 64) == 6
    assert lib.pg_attention(None, None, None, 0, None) == 1
    assert call(_problem(num_tokens=0, q=None)) == 0  # nothing to do


def test_appends_are_checked(lib):
    def call(cache=None, out=FAKE, v=FAKE, width=64, stride=(1024, 128, 64), q_stride=(1024, 256, 64, 32), **kw):
        d = dict(batch=2, num_queries=4, num_keys=4, num_heads=4, num_kv_heads=2, width=32, rotated=32, dtype=1, normed=1, eps=1e-6,
                 magnitude=1.0, q=FAKE, k=FAKE, turns=FAKE)
        d.update(kw)
        p = QkrProblem(**d)
        p.q_stride[:] = q_stride
        p.k_stride[:] = (1024, 128, 64, 32)
        vp = ctypes.c_void_p
        return lib.pg_append(ctypes.byref(p), vp(v), (ctypes.c_int64 * 3)(*stride), width, ctypes.byref(_fake_cache(**(cache or {}))), vp(out), None)

    for c, status in CACHE_FAULTS:
        assert call(cache=c) == status, c
    for kw, status in ((dict(cache=dict(k=None)), 1), (dict(cache=dict(v=None)), 1), (dict(out=None), 1), (dict(v=None), 1), (dict(v=FAKE + 1), 3),
                       (dict(out=FAKE + 1), 3), (dict(width=0), 2), (dict(width=257), 4), (dict(stride=(1, -1, 1)), 2), (dict(num_queries=3), 2),
                       (dict(rotated=33), 2), (dict(turns=None), 1), (dict(k=None), 1), (dict(q=None), 1), (dict(eps=0.0), 2)):
        assert call(**kw) == status, kw
    assert call(num_queries=0, num_keys=0) == 0  # nothing to do
    assert lib.pg_append(None, None, None, 0, None, None, None) == 1


def test_binding_checks_shapes_and_types():
    i32 = torch.int32
    k, v, q = torch.zeros(2, 3, 2, 2, 8), torch.zeros(2, 3, 2, 16), torch.zeros(2, 3, 4, 2, 8)
    kc, vc, table, lengths = torch.zeros(5, 4, 2, 2, 8), torch.zeros(5, 4, 2, 16), torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32)
    for bad in ((k[0], v, kc, vc, table, lengths), (k, v[:, :2], kc, vc, table, lengths), (k, v, kc[..., :4], vc, table, lengths),
                (k, v, kc, vc[:, :, :1], table, lengths), (k, v, kc, vc[..., :8], table, lengths), (k, v, kc[:4], vc, table, lengths),
                (k, v, kc, vc, table[0], lengths), (k, v, kc, vc, table[:1], lengths), (k, v, kc, vc, table.long(), lengths),
                (k, v, kc, vc, table, lengths[:1]), (k, v, kc, vc, table, lengths.long()), (k, v.half(), kc, vc, table, lengths)):
        with pytest.raises((ValueError, TypeError)):
            da.paged_append(*bad)
    with pytest.raises(TypeError):
        da.paged_append(k, v, kc.half(), vc.half(), table, lengths)
    for kw in (dict(q=q[:, :2]), dict(q=q[:1]), dict(counts=lengths.long()), dict(positions=lengths), dict(k_weight=torch.ones(4))):
        with pytest.raises(ValueError):
            da.paged_append(k, v, kc, vc, table, lengths, **kw)
    lam = torch.zeros(4)
    for bad in ((q[0], kc, vc, lam, table, lengths), (q[..., :4], kc, vc, lam, table, lengths), (q, kc[0], vc, lam, table, lengths),
                (q, kc, vc[..., 0], lam, table, lengths), (q, kc[:, :2], vc, lam, table, lengths), (q, kc, vc, lam, table[:1], lengths)):
        with pytest.raises(ValueError):
            da.paged_attention(*bad)
    with pytest.raises(TypeError):
        da.paged_attention(q.double(), kc, vc, lam, table, lengths)
    with pytest.raises(TypeError):
        da.paged_attention(q, kc.half(), vc, lam, table, lengths)
    with pytest.raises(ValueError, match="together"):
        da.paged_attention(q, kc, vc, lam, table, lengths, bias_table=torch.zeros(4, 4))


# ---- inputs ----------------------------------------------------------------

def _pool(g, lengths, N, S, spare=3, holes=False):
    """page_table [B, N] with the pages of sequences of these lengths anywhere in the pool; other entries are of no page."""
    B = len(lengths)
    pages = B * N + spare
    order = torch.randperm(pages, generator=g)[: B * N].to(torch.int32).reshape(B, N)
    for b, n in enumerate(lengths):
        order[b, -(-max(n, 0) // S):] = torch.tensor([-1, pages, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)[torch.randint(0, 4, (1,), generator=g)]
        if holes and N > 1:
            order[b, N // 2] = -1
    return order, pages


def _tree(g, B, T):
    sees = torch.eye(T, dtype=torch.bool).expand(B, T, T).clone()
    for b in range(B):
        for i in range(1, T):
            p = int(torch.randint(max(0, i - 4), i, (1,), generator=g))
            sees[b, i] |= sees[b, p]
    return sees


def _attention_case(B=1, T=1, S=16, N=4, lengths=None, counts=None, H=2, Hk=2, D=32, Dv=None, kind="f32", causal=True, buckets=0, reach=16,
                    pos=None, mask=None, tree=None, scale=None, layout="plain", holes=False, shared=False, peaked=1.0, seed=0):
    Dv = 2 * D if Dv is None else Dv
    g = torch.Generator().manual_seed(seed + T * 131 + S * 17 + N + H + D)
    dt = DT[kind]
    L = N * S
    lengths = [L] * B if lengths is None else lengths
    table, pages = _pool(g, [min(max(n, 0), L) for n in lengths], N, S, holes=holes)
    if shared:  # the first pages of all sequences are the first one's
        table[:, : N // 2] = table[0, : N // 2]
    t = dict(q=(torch.randn(B, T, H, 2, D, generator=g) * peaked).to(dt), k_cache=torch.randn(pages, S, Hk, 2, D, generator=g).to(dt),
             v_cache=torch.randn(pages, S, Hk, Dv, generator=g).to(dt), lam=torch.rand(H, generator=g) + 0.1, page_table=table,
             key_lengths=torch.tensor(lengths, dtype=torch.int32))
    opt = dict(causal=causal, scale=scale)
    if counts is not None:
        t["counts"] = torch.tensor(counts, dtype=torch.int32)
    if tree == "random":
        t["tree"] = _tree(g, B, T)
    elif tree == "none":
        t["tree"] = torch.zeros(B, T, T, dtype=torch.bool)
    if buckets:
        t["bias_table"], t["bucket_map"] = torch.randn(buckets, H, generator=g), da.relative_buckets(buckets, reach)
    if pos == "random":
        t["pos_q"], t["pos_k"] = (torch.randint(-50, 50, (B, x), generator=g, dtype=torch.int32) for x in (T, L))
    elif pos == "depth":
        old = t["key_lengths"] - (T if counts is None else t["counts"])
        t["pos_q"] = (old[:, None] + torch.arange(T) // 2).to(torch.int32).contiguous()
        t["pos_k"] = torch.arange(L, dtype=torch.int32).expand(B, L).contiguous()
    if mask is not None:
        t["key_mask"] = torch.rand(B, L, generator=g) < mask
        t["key_mask"][-1, : L // 2] = False
    t = {n: x.cuda() for n, x in t.items()}
    if layout == "heads first":
        for n in ("q", "k_cache", "v_cache"):
            t[n] = t[n].transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "one tensor":  # keys and values of a place side by side
        both = torch.cat([t["k_cache"].flatten(3), t["v_cache"]], -1)
        t["k_cache"], t["v_cache"] = both[..., : 2 * D].unflatten(-1, (2, D)), both[..., 2 * D:]
    elif layout == "odd offset":
        for n in ("q", "k_cache", "v_cache"):
            t[n] = torch.empty(t[n].numel() + 1, dtype=dt, device="cuda")[1:].view(t[n].shape).copy_(t[n])
    elif layout == "maps outside":
        for n in ("q", "k_cache"):
            t[n] = t[n].permute(3, 0, 1, 2, 4).contiguous().permute(1, 2, 3, 0, 4)
    return t, opt


CASES = {
    "one key": dict(N=1, S=1),
    "one key bf16": dict(N=1, S=8, lengths=[1], kind="bf16"),
    "one token": dict(N=6, lengths=[77]),
    "one token bf16": dict(N=6, lengths=[77], kind="bf16", H=4, Hk=4),
    "one token, shared heads": dict(B=3, N=20, lengths=[320, 1, 129], H=8, Hk=2, D=64, kind="bf16"),
    "one token, twelve heads": dict(B=2, N=9, S=64, H=12, Hk=1, kind="f16", lengths=[576, 300]),
    "sixteen rows": dict(B=2, N=9, S=64, T=2, H=8, Hk=1, kind="bf16", lengths=[576, 300]),
    "seventeen rows": dict(B=2, N=9, S=64, T=17, kind="bf16", lengths=[576, 300]),
    "thirty-three rows": dict(B=2, N=9, S=64, T=11, H=3, Hk=1, kind="f16", lengths=[576, 300]),
    "sixty-five rows": dict(B=2, N=9, S=64, T=65, kind="bf16", lengths=[576, 300]),
    "empty": dict(B=4, N=9, S=16, T=3, kind="bf16", lengths=[0, 1, 2, 144]),
    "empty f32": dict(B=4, N=9, S=16, T=3, lengths=[0, 1, 2, 144]),
    "lengths out of range": dict(B=3, N=5, S=16, T=2, kind="bf16", lengths=[-7, 1000, 80]),
    "counts": dict(B=5, N=9, S=16, T=7, kind="bf16", lengths=[144, 90, 3, 50, 64], counts=[7, 0, 5, 1, 100]),
    "counts f32": dict(B=5, N=9, S=16, T=7, lengths=[144, 90, 3, 50, 64], counts=[7, 0, 5, -3, 100]),
    "counts, many rows": dict(B=3, N=12, S=32, T=150, H=4, Hk=2, D=64, kind="f16", lengths=[384, 200, 130], counts=[150, 20, 129]),
    "holes": dict(B=2, N=9, S=16, T=3, kind="bf16", lengths=[144, 100], holes=True),
    "holes f32": dict(B=2, N=9, S=16, T=3, lengths=[144, 100], holes=True),
    "shared pages": dict(B=4, N=10, S=16, T=2, kind="bf16", lengths=[160, 150, 140, 81], shared=True),
    "pages of 1": dict(B=2, N=70, S=1, T=2, kind="bf16", lengths=[70, 33]),
    "pages of 3": dict(B=2, N=30, S=3, T=2, kind="bf16", lengths=[90, 33]),
    "pages of 8": dict(B=2, N=50, S=8, T=2, kind="bf16", lengths=[400, 133]),
    "pages of 20": dict(B=2, N=15, S=20, T=2, lengths=[300, 133]),
    "pages of 24": dict(B=2, N=15, S=24, T=2, D=64, kind="f16", lengths=[360, 133]),
    "pages of 48": dict(B=2, N=8, S=48, T=2, kind="bf16", lengths=[384, 133]),
    "pages of 100": dict(B=2, N=4, S=100, T=2, kind="bf16", lengths=[400, 133]),
    "pages of 128": dict(B=2, N=4, S=128, T=2, kind="bf16", lengths=[512, 133]),
    "pages of 1000": dict(B=2, N=2, S=1000, T=2, D=64, kind="bf16", lengths=[2000, 133]),
    "tree": dict(B=2, N=20, S=16, T=15, H=4, Hk=2, D=64, kind="bf16", lengths=[320, 100], tree="random"),
    "tree f32": dict(B=2, N=20, S=16, T=15, H=4, Hk=2, lengths=[320, 100], tree="random"),
    "tree, depths": dict(B=2, N=20, S=16, T=31, H=4, Hk=2, D=64, kind="f16", lengths=[320, 100], tree="random", pos="depth", buckets=32, reach=20),
    "tree alone": dict(B=2, N=4, S=16, T=33, H=4, Hk=2, D=64, kind="bf16", lengths=[33, 33], tree="random"),
    "tree, counts": dict(B=3, N=20, S=16, T=40, H=2, Hk=2, kind="bf16", lengths=[320, 139, 5], counts=[40, 11, 5], tree="random"),
    "tree across steps": dict(B=1, N=20, S=16, T=200, H=2, Hk=2, kind="bf16", lengths=[300], tree="random"),
    "tree that sees nothing": dict(B=2, N=4, S=16, T=5, kind="bf16", lengths=[5, 20], tree="none"),
    "tree that sees nothing f32": dict(B=2, N=4, S=16, T=5, lengths=[5, 20], tree="none"),
    "all": dict(B=2, N=9, S=16, T=40, kind="bf16", lengths=[144, 77], causal=False),
    "all f32": dict(B=2, N=9, S=16, T=40, lengths=[144, 77], causal=False),
    "bias": dict(B=2, N=30, S=16, T=3, H=4, Hk=2, kind="bf16", lengths=[480, 77], buckets=32, reach=128),
    "bias, near": dict(B=2, N=30, S=16, T=50, H=4, Hk=2, kind="f16", lengths=[480, 77], buckets=8, reach=30),
    "bias f32": dict(B=2, N=30, S=16, T=3, H=4, Hk=2, lengths=[480, 77], buckets=32, reach=128),
    "bias, all": dict(B=2, N=30, S=16, T=3, H=4, Hk=2, kind="bf16", lengths=[480, 77], buckets=32, reach=128, causal=False),
    "positions": dict(B=2, N=9, S=16, T=40, H=2, kind="bf16", lengths=[144, 77], pos="random", buckets=16, reach=30),
    "positions f32": dict(B=2, N=9, S=16, T=40, H=2, lengths=[144, 77], pos="random", buckets=16, reach=30),
    "mask": dict(B=3, N=9, S=16, T=2, H=4, kind="bf16", lengths=[144, 77, 72], mask=0.7),
    "mask f32": dict(B=3, N=9, S=16, T=2, H=4, lengths=[144, 77, 72], mask=0.7),
    "mask of all": dict(B=2, N=9, S=16, T=2, H=4, kind="f16", lengths=[144, 77], mask=0.0),
    "width 24": dict(B=2, N=9, S=16, T=2, D=24, kind="bf16", lengths=[144, 77]),
    "width 16": dict(B=2, N=9, S=16, T=20, D=16, kind="f16", lengths=[144, 77]),
    "width 40": dict(B=2, N=9, S=16, T=20, D=40, kind="bf16", lengths=[144, 77]),
    "width 17": dict(B=2, N=9, S=16, T=2, D=17, Dv=33, kind="bf16", lengths=[144, 77]),
    "width 128": dict(B=2, N=9, S=16, T=2, D=128, kind="bf16", lengths=[144, 77]),
    "width 128 f32": dict(B=2, N=9, S=16, T=2, D=128, lengths=[144, 77]),
    "value width apart": dict(B=2, N=9, S=16, T=2, D=64, Dv=40, kind="bf16", lengths=[144, 77]),
    "value width 8": dict(B=2, N=9, S=16, T=70, D=32, Dv=8, kind="bf16", lengths=[144, 77]),
    "peaked": dict(B=2, N=30, S=16, T=3, kind="bf16", lengths=[480, 77], peaked=8.0),
    "peaked f16": dict(B=2, N=30, S=16, T=70, D=64, kind="f16", lengths=[480, 77], peaked=8.0),
    "negative scale": dict(B=2, N=9, S=16, T=2, kind="bf16", lengths=[144, 77], scale=-0.3),
    "no scale": dict(B=2, N=9, S=16, T=2, kind="bf16", lengths=[144, 77], scale=0.0),
    "heads first": dict(B=2, N=9, S=16, T=2, H=4, Hk=2, kind="bf16", lengths=[144, 77], layout="heads first"),
    "one tensor": dict(B=2, N=9, S=16, T=2, H=4, Hk=2, kind="bf16", lengths=[144, 77], layout="one tensor"),
    "odd offset": dict(B=2, N=9, S=16, T=2, H=4, Hk=2, kind="bf16", lengths=[144, 77], layout="odd offset"),
    "odd offset f32": dict(B=2, N=9, S=16, T=2, H=4, Hk=2, lengths=[144, 77], layout="odd offset"),
    "maps outside": dict(B=2, N=9, S=16, T=2, H=4, Hk=2, kind="f16", lengths=[144, 77], layout="maps outside"),
    "long": dict(B=2, N=200, S=64, H=8, Hk=2, D=64, kind="bf16", lengths=[12800, 7001]),
    "long f16": dict(B=3, N=200, S=32, T=3, H=8, Hk=4, D=64, kind="f16", lengths=[6400, 1, 3001], buckets=16, reach=64),
    "three rows f32": dict(B=2, N=9, S=16, T=1, H=6, Hk=2, D=64, lengths=[144, 77], buckets=8, reach=20),
    "six rows f32": dict(B=2, N=9, S=16, T=3, H=4, Hk=2, D=64, lengths=[144, 77], tree="random", mask=0.8),
    "eight rows f16": dict(B=2, N=20, S=20, T=4, H=4, Hk=2, D=40, kind="f16", lengths=[400, 301], tree="random", buckets=8, reach=20, pos="depth"),
    "three wide rows": dict(B=2, N=9, S=16, T=1, H=3, Hk=1, D=96, Dv=200, lengths=[144, 77]),
    "five odd rows": dict(B=2, N=30, S=3, T=5, H=1, Hk=1, D=127, Dv=255, kind="bf16", lengths=[90, 33]),
    "nine rows f32": dict(B=2, N=40, S=20, T=3, H=3, Hk=1, D=64, lengths=[800, 333]),
    "thirty rows f32": dict(B=2, N=40, S=20, T=15, H=4, Hk=2, D=64, lengths=[800, 333], tree="random", mask=0.7),
    "thirty wide rows f32": dict(B=2, N=40, S=20, T=15, H=4, Hk=2, D=100, lengths=[800, 333], counts=[15, 4], buckets=8, reach=20),
    "small pages, many rows": dict(B=2, N=300, S=3, T=45, H=4, Hk=2, D=32, kind="bf16", lengths=[900, 333], tree="random"),
    "many parts f32": dict(B=1, N=500, S=16, T=1, H=2, Hk=1, lengths=[8000]),
    "long f32": dict(B=2, N=200, S=20, H=4, Hk=2, lengths=[4000, 3001]),
    "one long among short": dict(B=40, N=40, S=64, H=4, Hk=2, D=32, kind="bf16", lengths=[2560] + [3 + b for b in range(39)]),
    "many short": dict(B=300, N=2, S=16, H=4, Hk=4, kind="bf16", lengths=[(b * 7) % 33 for b in range(300)]),
    "prompt": dict(B=2, N=40, S=32, T=333, H=6, Hk=2, D=64, kind="bf16", lengths=[1280, 800], buckets=32, reach=128),
    "prompt from nothing": dict(B=1, N=40, S=32, T=700, H=4, Hk=4, D=32, kind="f16", lengths=[700]),
    "prompt longer than its keys": dict(B=1, N=4, S=32, T=150, H=2, kind="bf16", lengths=[100]),
    "widest group": dict(B=1, N=9, S=16, T=3, H=64, Hk=1, kind="bf16", lengths=[144]),
    "group of forty": dict(B=2, N=9, S=16, T=1, H=40, Hk=1, D=64, kind="f16", lengths=[144, 100]),
    "sixty-four rows": dict(B=2, N=40, S=16, T=16, H=8, Hk=2, D=64, kind="bf16", lengths=[640, 401], tree="random"),
    "sixty-five rows": dict(B=2, N=40, S=16, T=13, H=10, Hk=2, D=64, kind="bf16", lengths=[640, 401]),
    "wider group": dict(B=1, N=9, S=16, T=3, H=65, Hk=1, kind="bf16", lengths=[144]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_against_64_bits(name):
    t, opt = _attention_case(**CASES[name])
    got = da.paged_attention(**t, **opt)
    val, tol = paged_reference(**t, **opt)
    check({"out": got}, val, tol)
    assert torch.equal(got, da.paged_attention(**t, **opt)), "results vary from run to run"


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T,H", [(1, 4), (4, 4), (8, 4), (11, 4), (2, 32), (64, 1)])
def test_few_rows_are_rounded_once(kind, T, H):
    """Up to 64 rows, of groups of up to 32 heads, carry what rounding took from the weights: in a norm their outputs are off by what one
    rounding of the exact ones costs, and by a thousandth more for 64 bits' own and fp32's steps."""
    t, opt = _attention_case(B=2, T=T, N=40, S=16, H=H, Hk=1, D=64, kind=kind, lengths=[640, 401])
    assert da.paged_path(**t, **opt) == "tensor" and T * H <= 64
    want = paged_reference(**t, **opt)[0]["out"]
    once = float((want.to(DT[kind]).double() - want).norm())
    assert float((da.paged_attention(**t, **opt).double() - want).norm()) <= 1.02 * once


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,D", [(1, 64), (9, 32), (12, 64), (70, 32), (70, 64)])
def test_maxima_that_climb(kind, T, D):
    """Scores that grow along the keys by hundreds in all, or fall, so that references are raised in most steps or never."""
    t, opt = _attention_case(B=2, T=T, N=60, S=16, H=4, Hk=2, D=D, kind=kind, lengths=[960, 777])
    t["q"] = t["q"].abs()
    t["k_cache"] = t["k_cache"].abs()
    for b, n in enumerate([960, 777]):
        at = torch.arange(n, device="cuda")
        slope = 8 * at / n if b == 0 else 8 - 8 * at / n
        places = t["page_table"][b].long()[at // 16], at % 16
        t["k_cache"][places] = (t["k_cache"][places].float() * slope[:, None, None, None]).to(DT[kind])
    val, tol = paged_reference(**t, **opt)
    check({"out": da.paged_attention(**t, **opt)}, val, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T,D", [("f32", 3, 32), ("bf16", 3, 32), ("f16", 30, 64), ("bf16", 90, 64), ("bf16", 3, 17)])
def test_what_masked_places_hold_is_not_used(kind, T, D):
    t, opt = _attention_case(B=4, T=T, N=20, S=16, H=4, Hk=2, D=D, kind=kind, mask=0.6, lengths=[320, 130, 0, 100], holes=True)
    t["key_mask"][0, 100:260] = False
    want = da.paged_attention(**t, **opt)
    used = torch.zeros(t["k_cache"].shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate([320, 130, 0, 100]):
        for j in range(n):
            if int(t["page_table"][b, j // 16]) >= 0 and bool(t["key_mask"][b, j]):
                used[t["page_table"][b, j // 16], j % 16] = True
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(DT[kind]).min):
        u = {**t, "k_cache": t["k_cache"].masked_fill(~used[..., None, None, None], bad), "v_cache": t["v_cache"].masked_fill(~used[..., None, None], bad)}
        assert torch.equal(da.paged_attention(**u, **opt), want), bad


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T", [("f32", 5), ("bf16", 5), ("bf16", 70)])
def test_rows_past_the_count_are_zeros_whatever_they_hold(kind, T):
    t, opt = _attention_case(B=3, T=T, N=20, S=16, H=4, Hk=2, kind=kind, lengths=[320, 130, 77], counts=[T, 2, 0], tree="random")
    want = da.paged_attention(**t, **opt)
    assert not bool(want[1, 2:].any()) and not bool(want[2].any())
    t["q"][1, 2:], t["q"][2] = float("nan"), float("inf")
    t["tree"][1, 2:], t["tree"][2] = True, True
    got = da.paged_attention(**t, **opt, out=torch.full_like(want, float("nan")))
    assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_biases_that_hide(kind):
    """A bias of -infinity, or one that overflows in base 2, hides its bucket's keys; a row of hidden keys gives 0."""
    for low in (-float("inf"), torch.finfo(torch.float32).min):
        t, opt = _attention_case(B=2, T=2, N=9, S=16, H=2, kind=kind, lengths=[144, 20], buckets=4, reach=8)
        t["bias_table"][1] = low                   # the farther half before the query
        u = {n: x for n, x in t.items() if n not in ("bias_table", "bucket_map")}
        got = da.paged_attention(**t, **opt)
        assert bool(torch.isfinite(got).all()) and bool(got.any())
        t["bias_table"][:] = low
        assert not bool(da.paged_attention(**t, **opt).any())
        assert bool(da.paged_attention(**u, **opt).any())


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements: pages near its end."""
    S, Hk, D, Dv = 16, 8, 64, 128
    pages = (1 << 32) // (S * Hk * 2 * D) + 20
    k, v = (torch.empty(pages, S, Hk, *w, dtype=torch.bfloat16, device="cuda") for w in ((2, D), (Dv,)))
    table = torch.tensor([[pages - 1, 3, pages - 7], [5, pages - 2, 0]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    new_k, new_v = (torch.randn(2, 40, Hk, *w, generator=g).to(torch.bfloat16).cuda() for w in ((2, D), (Dv,)))
    lengths = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    k[pages - 1, :3], v[pages - 1, :3] = 0.5, 0.25
    da.paged_append(new_k, new_v, k, v, table, lengths, eps=None)
    for b, at in ((0, 3), (1, 0)):
        rows = [(int(table[b, (at + t) // S]), (at + t) % S) for t in range(40)]
        assert all(torch.equal(k[p, s], new_k[b, t]) and torch.equal(v[p, s], new_v[b, t]) for t, (p, s) in enumerate(rows))
    q, lam = torch.randn(2, 1, 16, 2, D, generator=g).to(torch.bfloat16).cuda(), torch.rand(16, generator=g).cuda()
    got = da.paged_attention(q, k, v, lam, table, lengths + 40)
    small = table.clone()
    pick = table.reshape(-1).long()
    small[:] = torch.arange(6, dtype=torch.int32, device="cuda").reshape(2, 3)
    assert torch.equal(got, da.paged_attention(q, k[pick], v[pick], lam, small, lengths + 40))


# ---- append ----------------------------------------------------------------

def _append_case(B=2, T=5, S=16, N=4, before=None, counts=None, H=4, Hk=2, D=32, Dv=None, R=None, kind="bf16", q=True, weights=True,
                 eps=1e-6, interleaved=False, magnitude=1.0, positions=False, layout="plain", holes=False, seed=0):
    Dv = 2 * D if Dv is None else Dv
    g = torch.Generator().manual_seed(seed + T * 31 + S + D)
    dt = DT[kind]
    before = [(b * 7) % 20 for b in range(B)] if before is None else before
    table, pages = _pool(g, [min(max(n, 0) + T, N * S) for n in before], N, S, holes=holes)
    R = D if R is None else R
    t = dict(k=torch.randn(B, T, Hk, 2, D, generator=g).to(dt), v=torch.randn(B, T, Hk, Dv, generator=g).to(dt),
             k_cache=torch.randn(pages, S, Hk, 2, D, generator=g).to(dt), v_cache=torch.randn(pages, S, Hk, Dv, generator=g).to(dt),
             page_table=table, lengths=torch.tensor(before, dtype=torch.int32))
    if q:
        t["q"] = torch.randn(B, T, H, 2, D, generator=g).to(dt)
    if counts is not None:
        t["counts"] = torch.tensor(counts, dtype=torch.int32)
    if R:
        t["frequencies"] = da.rotary_frequencies(R)
    if weights and eps is not None:
        t["k_weight"] = torch.randn(D, generator=g)
        if q:
            t["q_weight"] = torch.randn(D, generator=g)
    if positions:
        t["positions"] = torch.randint(-5, 100000, (B, T), generator=g, dtype=torch.int32)
    t = {n: x.cuda() for n, x in t.items()}
    if layout == "heads first":
        for n in ("q", "k", "v", "k_cache", "v_cache"):
            t[n] = t[n].transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "one tensor":
        both = torch.cat([t["k_cache"].flatten(3), t["v_cache"]], -1)
        t["k_cache"], t["v_cache"] = both[..., : 2 * D].unflatten(-1, (2, D)), both[..., 2 * D:]
    elif layout == "odd offset":
        for n in ("k", "v", "k_cache"):
            t[n] = torch.empty(t[n].numel() + 1, dtype=dt, device="cuda")[1:].view(t[n].shape).copy_(t[n])
    return t, dict(eps=eps, interleaved=interleaved, magnitude=magnitude)


APPENDS = {
    "one token": dict(B=1, T=1),
    "one token each": dict(B=33, T=1, N=9, D=64, H=16, Hk=4, before=[(b * 5) % 143 for b in range(33)]),
    "f32": dict(kind="f32"),
    "f32, parts": dict(kind="f32", D=24, R=16, interleaved=True, S=20, T=30),
    "no queries": dict(q=False),
    "f16": dict(kind="f16", D=64, T=40),
    "counts": dict(B=5, T=9, counts=[9, 0, 4, -1, 100]),
    "past the table": dict(B=3, T=9, N=2, before=[30, 32, 100]),
    "below zero": dict(B=2, T=9, before=[-4, 2]),
    "holes": dict(B=2, T=40, N=4, before=[0, 10], holes=True),
    "pages of 1": dict(S=1, N=40, T=7),
    "pages of 3": dict(S=3, N=20, T=7, kind="f16"),
    "wide values": dict(D=32, Dv=256, kind="f32"),
    "narrow values": dict(D=64, Dv=8),
    "odd widths": dict(D=17, Dv=33, R=16),
    "odd values": dict(D=64, Dv=127),
    "values of 1": dict(D=32, Dv=1),
    "no norm": dict(eps=None),
    "as it is": dict(eps=None, R=0),
    "positions": dict(positions=True, magnitude=1.2),
    "heads first": dict(layout="heads first"),
    "one tensor": dict(layout="one tensor"),
    "odd offset": dict(layout="odd offset"),
    "prompt": dict(B=3, T=700, N=60, S=16, before=[0, 200, 77], counts=[700, 650, 3]),
    "no places": dict(N=0, T=3),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(APPENDS))
def test_append_against_64_bits(name):
    t, opt = _append_case(**APPENDS[name])
    B, T = t["k"].shape[:2]
    S, N, P = t["k_cache"].shape[1], t["page_table"].shape[1], t["k_cache"].shape[0]
    before_k, before_v = t["k_cache"].clone(), t["v_cache"].clone()
    lengths = t["lengths"].clone()
    out = da.paged_append(**t, **opt)
    assert torch.equal(lengths, t["lengths"])
    place = t["lengths"].long()[:, None] + torch.arange(T, device="cuda")
    pos = t["positions"].long() if "positions" in t else place
    ref = {n: qkr_reference(t[n], t.get("frequencies"), t.get(n + "_weight"), pos, **opt) for n in ("q", "k") if n in t}
    if "q" in t:
        check({"out": out}, *ref["q"], "queries")
    else:
        assert out is None
    want, tol = before_k.double(), torch.zeros_like(before_k, dtype=torch.float64)
    want_v = before_v.clone()
    val, off = ref["k"][0]["out"], ref["k"][1]["out"]
    for b in range(B):
        for i in range(T if "counts" not in t else min(max(int(t["counts"][b]), 0), T)):
            j = int(place[b, i])
            if not 0 <= j < N * S:
                continue
            page = int(t["page_table"][b, j // S])
            if 0 <= page < P:
                want[page, j % S], tol[page, j % S], want_v[page, j % S] = val[b, i], off[b, i], t["v"][b, i]
    check({"k": t["k_cache"]}, {"k": want}, {"k": tol}, "keys")  # what was not written is as it was: no tolerance
    assert torch.equal(t["v_cache"], want_v)
    again = {**t, "k_cache": before_k, "v_cache": before_v}
    out2 = da.paged_append(**again, **opt)
    assert torch.equal(before_k, t["k_cache"]) and (out is None or torch.equal(out, out2))


@pytest.mark.gpu
def test_append_gives_the_rotary_norms_bits():
    t, opt = _append_case(B=3, T=9, before=[0, 3, 11], N=4)
    q = da.paged_append(**t, **opt)
    pos = (t["lengths"][:, None] + torch.arange(9, device="cuda")).to(torch.int32).contiguous()
    wq, wk = da.qkr_forward(t["q"], t["k"], t["frequencies"], t["q_weight"], t["k_weight"], pos, pos, **opt)
    assert torch.equal(q, wq)
    for b in range(3):
        for i in range(9):
            j = int(pos[b, i])
            assert torch.equal(t["k_cache"][t["page_table"][b, j // 16], j % 16], wk[b, i])


# ---- as they are used together ---------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("kind,D,S", [("f32", 32, 20), ("bf16", 64, 16), ("f16", 32, 24)])
def test_a_run_of_prompts_tokens_and_drafts(kind, D, S):
    """Ragged prompts, single tokens, a drafted tree whose accepted branch is appended for good: each step's attention
    equals that of the same keys in a row (dattn_forward), whose keys were rotated by qkr_forward."""
    g = torch.Generator().manual_seed(D)
    B, H, Hk, N = 3, 4, 2, 12
    dt = DT[kind]
    table, pages = _pool(g, [N * S] * B, N, S)
    table = table.cuda()
    kc, vc = (torch.full((pages, S, Hk, *w), float("nan"), dtype=dt, device="cuda") for w in ((2, D), (2 * D,)))
    turns, lam = da.rotary_frequencies(D).cuda(), torch.rand(H, generator=g).cuda()
    wq, wk = (torch.randn(D, generator=g).cuda() for _ in range(2))
    opt = dict(frequencies=turns, q_weight=wq, k_weight=wk)
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    hist = [[torch.empty(0, Hk, 2, D, dtype=dt, device="cuda"), torch.empty(0, Hk, 2 * D, dtype=dt, device="cuda")] for _ in range(B)]

    def new(T):
        return [torch.randn(B, T, *s, generator=g).to(dt).cuda() for s in ((H, 2, D), (Hk, 2, D), (Hk, 2 * D))]

    def compare(out, q, b, n):
        """Rows of sequence b against dattn_forward over its first n keys in a row."""
        k, v = hist[b][0][None, :n].contiguous(), hist[b][1][None, :n].contiguous()
        want = da.dattn_forward(q, k, v, lam, causal=True)
        # Both are within paged_reference's tolerance of the same values; here a norm: twice a rounding of weights and result.
        r = torch.finfo(dt).eps if dt != torch.float32 else 64 * 2.0 ** -23
        assert float((out.double() - want.double()).norm()) <= 2 * r * float(want.double().norm()) + 1e-30

    def append(q, k, v, counts=None, keep=True):
        nq = da.paged_append(k, v, kc, vc, table, lengths, counts=counts, q=q, **opt)
        for b in range(B):
            c = k.shape[1] if counts is None else int(counts[b])
            pos = (torch.arange(c, device="cuda", dtype=torch.int32) + lengths[b]).to(torch.int32)[None].contiguous()
            rk = da.qkr_forward(None, k[b: b + 1, :c].contiguous(), turns, None, wk, None, pos)[1]
            hist[b][0] = torch.cat([hist[b][0][: int(lengths[b])], rk[0]])
            hist[b][1] = torch.cat([hist[b][1][: int(lengths[b])], v[b, :c]])
        return nq

    counts = torch.tensor([2 * S + 3, 70, 1], dtype=torch.int32, device="cuda")
    q = append(*new(int(counts.max())), counts=counts)
    out = da.paged_attention(q, kc, vc, lam, table, counts, counts=counts)
    for b in range(B):
        c = int(counts[b])
        compare(out[b: b + 1, :c], q[b: b + 1, :c].contiguous(), b, c)
        assert not bool(out[b, c:].any())
    lengths += counts
    for _ in range(3):
        q = append(*new(1))
        lengths += 1
        out = da.paged_attention(q, kc, vc, lam, table, lengths)
        for b in range(B):
            compare(out[b: b + 1], q[b: b + 1], b, int(lengths[b]))
    # A tree of two branches, 0-1-2 and 0-3-4: the second one is what a plain chain 0, 3, 4 gives.
    T = 5
    qn, kn, vn = new(T)
    depth = torch.tensor([0, 1, 2, 1, 2], dtype=torch.int32, device="cuda")
    tree = torch.zeros(T, T, dtype=torch.bool)
    for i, up in enumerate(([0], [0, 1], [0, 1, 2], [0, 3], [0, 3, 4])):
        tree[i, up] = True
    at = (lengths[:, None] + depth).to(torch.int32).contiguous()
    q = da.paged_append(kn, vn, kc, vc, table, lengths, q=qn, positions=at, **opt)
    out = da.paged_attention(q, kc, vc, lam, table, lengths + T, tree=tree.cuda().expand(B, T, T).contiguous())
    pick = torch.tensor([0, 3, 4], device="cuda")
    chain = append(qn[:, pick], kn[:, pick], vn[:, pick])   # accepted: over the drafted tokens' places
    lengths += 3
    assert torch.equal(chain, q[:, pick])
    plain = da.paged_attention(chain, kc, vc, lam, table, lengths)
    r = torch.finfo(dt).eps if dt != torch.float32 else 64 * 2.0 ** -23
    assert float((plain.double() - out[:, pick].double()).norm()) <= 2 * r * float(plain.double().norm())
    for b in range(B):
        compare(plain[b: b + 1], chain[b: b + 1].contiguous(), b, int(lengths[b]))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_a_captured_step(kind):
    """One decoding step in a graph, replayed while the cache grows, on a side stream; and the same eagerly."""
    dt = DT[kind]
    g = torch.Generator().manual_seed(9)
    B, H, Hk, D, S, N = 3, 4, 2, 32, 16, 8
    table, pages = _pool(g, [N * S] * B, N, S)
    table = table.cuda()
    caches = [[torch.full((pages, S, Hk, *w), float("nan"), dtype=dt, device="cuda") for w in ((2, D), (2 * D,))] for _ in range(2)]
    turns, lam = da.rotary_frequencies(D).cuda(), torch.rand(H, generator=g).cuda()
    lengths = [torch.tensor([0, 15, 40], dtype=torch.int32, device="cuda") for _ in range(2)]
    for kc, vc in caches:
        kc[:], vc[:] = 0.5, 0.25
    x = [torch.zeros(B, 1, *s, dtype=dt, device="cuda") for s in ((H, 2, D), (Hk, 2, D), (Hk, 2 * D))]

    def step(c, n, q, k, v):
        q = da.paged_append(k, v, *c, table, n, q=q, frequencies=turns)
        n += 1
        return da.paged_attention(q, *c, lam, table, n)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches[0], lengths[0], *x)
    side = torch.cuda.Stream()
    for _ in range(60):
        now = [torch.randn(*t.shape, generator=g).to(dt).cuda() for t in x]
        want = step(caches[1], lengths[1], *now)
        for a, b in zip(x, now):
            a.copy_(b)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want)
    assert torch.equal(lengths[0], lengths[1]) and all(torch.equal(a, b) for a, b in zip(*caches))


@pytest.mark.gpu
def test_on_a_given_stream():
    t, opt = _attention_case(B=2, N=60, S=16, H=8, Hk=2, D=64, kind="bf16", lengths=[960, 100])
    want = da.paged_attention(**t, **opt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [da.paged_attention(**t, **opt, stream=s) for s in (side, None, side)]
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_training_through_the_rotary_norm_and_the_attention(kind):
    """q and k through QkRotaryFunction into DifferentialAttentionFunction, gradients against 64 bits in a norm."""
    g = torch.Generator().manual_seed(4)
    dt = DT[kind]
    B, L, H, Hk, D = 2, 60, 4, 2, 32
    turns = da.rotary_frequencies(16)
    q, k, v, gr = (torch.randn(B, L, *s, generator=g).to(dt).cuda() for s in ((H, 2, D), (Hk, 2, D), (Hk, 2 * D), (H, 2 * D)))
    wq, wk = (torch.randn(D, generator=g).cuda() for _ in range(2))
    lam = torch.rand(H, generator=g).cuda()
    leaves = [t.detach().requires_grad_(True) for t in (q, k, v, wq, wk, lam)]
    rq, rk = da.QkRotaryFunction.apply(leaves[0], leaves[1], turns.cuda(), leaves[3], leaves[4])
    out = da.DifferentialAttentionFunction.apply(rq, rk, leaves[2], leaves[5], None, None, None, None, None, None, True, None)
    got = (out, *torch.autograd.grad(out, leaves, gr))
    ex = [t.detach().double().requires_grad_(True) for t in (q, k, v, wq, wk, lam)]
    a = torch.arange(L, dtype=torch.float64, device="cuda")[:, None] * torch.tensor([10000.0 ** (-i / 8) for i in range(8)], device="cuda", dtype=torch.float64)
    c, s = a.cos()[:, None, None], a.sin()[:, None, None]

    def turn(x, w):
        y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        return torch.cat([y[..., :8] * c - y[..., 8:16] * s, y[..., :8] * s + y[..., 8:16] * c, y[..., 16:]], -1)

    tq, tk = turn(ex[0], ex[3]), turn(ex[1], ex[4]).repeat_interleave(2, 2)
    p = torch.softmax((torch.einsum("bihmd,bjhmd->bhmij", tq, tk) / D ** 0.5).masked_fill(torch.ones(L, L, device="cuda").triu(1).bool(), float("-inf")), -1)
    o = torch.einsum("bhij,bjhe->bihe", p[:, :, 0] - ex[5][:, None, None] * p[:, :, 1], ex[2].repeat_interleave(2, 2))
    want = (o, *torch.autograd.grad(o, ex, gr.double()))
    # In 16 bits: q, k, weights, s_m and results are each rounded once on the way, and scores move by D/4 such steps at most.
    r = 2e-5 if kind == "f32" else 8 * 2.0 ** -8
    for name, x, y in zip(("out", "q", "k", "v", "wq", "wk", "lam"), got, want):
        assert float((x.detach().double() - y.detach()).norm()) <= r * float(y.detach().norm()), name


@pytest.mark.parametrize("kw,path", [
    (dict(), 1), (dict(dtype=2), 1), (dict(dtype=0), 0), (dict(width=64, value_width=128), 1), (dict(width=20), 0), (dict(width=72), 0),
    (dict(value_width=136), 0), (dict(num_heads=130, num_buckets=0, reach=0), 0), (dict(cache=dict(page_size=20)), 0), (dict(cache=dict(page_size=24)), 1),
    (dict(cache=dict(num_pages=0)), 0), (dict(cache=dict(table_pages=0)), 0), (dict(q=FAKE + 8), 0), (dict(cache=dict(k=FAKE + 8)), 0),
    (dict(num_buckets=128, num_heads=4, reach=1024), 0), (dict(num_tokens=0), 0), (dict(q_stride=(1024, 252, 64, 32)), 0),
    (dict(q_stride=(0, 256, 64, 32)), 0), (dict(width=-1), -1),
])
def test_which_kernels_a_problem_takes(lib, kw, path):
    assert lib.pg_path(ctypes.byref(_problem(**kw))) == path
