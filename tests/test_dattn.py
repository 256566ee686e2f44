"""Differential attention with a relative position bias (dattn_forward,
dattn_backward, DifferentialAttentionFunction): refusals on the CPU, results on
the GPU against 64 bits."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import deformable_view_feature_gb300 as da
from deformable_view_feature_gb300 import attention
from operator_refs import check, dattn_reference

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FAKE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    da.build.build()
    return da.load_library()


# ---- refusals and host logic: no GPU, nothing is launched ------------------

def _problem(**kw):
    d = dict(batch=1, num_queries=4, num_keys=8, num_heads=4, num_kv_heads=2, width=32, value_width=64, dtype=1,
             num_buckets=8, reach=16, causal=0, scale=0.1, q=FAKE, k=FAKE, v=FAKE, lam=FAKE, bias_table=FAKE,
             bucket_map=FAKE)
    stride = kw.pop("q_stride", (1024, 256, 64, 32))
    d.update(kw)
    p = attention.DattnProblem(**d)
    p.q_stride[:] = stride
    p.k_stride[:] = (1024, 128, 64, 32)
    p.v_stride[:] = (1024, 128, 64)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(batch=-1), 2), (dict(num_queries=-1), 2), (dict(num_heads=3), 2), (dict(num_kv_heads=0), 2),
    (dict(width=0), 2), (dict(width=129), 4), (dict(value_width=257), 4), (dict(dtype=5), 2),
    (dict(scale=float("inf")), 2), (dict(num_buckets=-1), 2), (dict(reach=0), 2), (dict(reach=2000), 4),
    (dict(num_buckets=300), 4), (dict(num_buckets=0, reach=0), 0), (dict(batch=70000), 4),
    (dict(num_queries=1 << 30), 4), (dict(q_stride=(1024, -256, 64, 32)), 2),
])
def test_sizes_are_checked(lib, kw, status):
    n = ctypes.c_size_t(0)
    for backward in (0, 1):
        assert lib.dattn_workspace_size(ctypes.byref(_problem(**kw)), backward, ctypes.byref(n)) == status


def test_buffers_are_checked(lib):
    vp = ctypes.c_void_p

    def forward(out=FAKE, out1=None, lse=None, ws=None, size=0, **kw):
        return lib.dattn_forward(ctypes.byref(_problem(**kw)), vp(out), vp(out1), vp(lse), vp(ws), size, None)

    for name in ("q", "k", "v", "lam", "bias_table", "bucket_map"):
        assert forward(**{name: None}) == 1, name
    assert forward(out=None) == 1 and forward(out1=FAKE) == 1 and forward(lse=FAKE) == 1
    assert forward(q=FAKE + 1) == 3 and forward(lam=FAKE + 2) == 3
    assert lib.dattn_forward(None, None, None, None, None, 0, None) == 1

    n = ctypes.c_size_t(0)
    p = _problem()
    assert lib.dattn_workspace_size(ctypes.byref(p), 1, ctypes.byref(n)) == 0 and n.value > 0

    def backward(size=n.value, ws=FAKE, **kw):
        args = {k: FAKE for k in ("out", "out1", "lse", "grad_out", "grad_q", "grad_k", "grad_v", "grad_lam", "grad_table")}
        args.update(kw)
        return lib.dattn_backward(ctypes.byref(p), *[vp(x) for x in args.values()], vp(ws), size, None)

    for name in ("out", "out1", "lse", "grad_out", "grad_q", "grad_k", "grad_v", "grad_lam", "grad_table"):
        assert backward(**{name: None}) == 1, name
    assert backward(size=n.value - 1) == 6 and backward(ws=None) == 6 and backward(ws=FAKE + 64) == 6
    assert backward(grad_q=FAKE + 1) == 3 and backward(grad_table=FAKE + 1) == 3


def test_nothing_to_do(lib):
    p = _problem(num_queries=0, q=None)
    assert lib.dattn_forward(ctypes.byref(p), None, None, None, None, 0, None) == 0


def test_binding_checks_shapes_and_types():
    q, k, v, lam = torch.zeros(1, 3, 4, 2, 8), torch.zeros(1, 5, 2, 2, 8), torch.zeros(1, 5, 2, 16), torch.zeros(4)
    for bad in ((q[0], k, v), (q, k[..., :1, :], v), (q, k, v[..., 0]), (q, k[:, :4], v), (q, k[..., :4], v),
                (torch.zeros(2, 3, 4, 2, 8), k, v)):
        with pytest.raises(ValueError):
            da.dattn_forward(*bad, lam)
    with pytest.raises(TypeError):
        da.dattn_forward(q.double(), k, v, lam)
    with pytest.raises(TypeError):
        da.dattn_forward(q, k.half(), v, lam)
    with pytest.raises(ValueError, match="together"):
        da.dattn_forward(q, k, v, lam, bias_table=torch.zeros(4, 4))


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("H,D,status", [(3, 8, 2), (4, 129, 4)])  # no multiple of the key heads; too wide
def test_path_of_an_invalid_problem(lib, H, D, status):
    with FakeTensorMode():  # tensors of a device without storage; nothing is launched
        t = [torch.empty(*s, device="cuda:0") for s in ((1, 3, H, 2, D), (1, 5, 2, 2, D), (1, 5, 2, 16), (H,))]
        with pytest.raises(da.DaError) as e:
            da.dattn_path(*t)
    assert e.value.status == status


def test_relative_buckets():
    b = da.relative_buckets(32, 128).tolist()
    assert len(b) == 257 and b[128] == 0 and b[127] == 1 and b[129] == 17
    assert b[:128] == [x - 16 for x in b[:128:-1]]          # the same buckets on both sides
    assert b[0] == 15 and b[256] == 31
    assert all(x >= y for x, y in zip(b[:128], b[1:129]))   # farther: a later bucket
    # exact powers lie in the bucket that begins there: 8 single ones, 8 more up to 128
    assert [b[128 - n] for n in (8, 16, 32, 64, 128)] == [8, 10, 12, 14, 15]
    one = da.relative_buckets(4, 10, bidirectional=False).tolist()
    assert one[10:] == [0] * 11 and max(one) == 3 and len(one) == 21
    with pytest.raises(ValueError):
        da.relative_buckets(1, 8)


# ---- results ---------------------------------------------------------------

def _case(B=1, Lq=64, Lk=64, H=2, Hk=2, D=32, Dv=None, kind="f32", causal=False, buckets=0, reach=16, pos=None,
          mask=None, lengths=None, scale=None, layout="plain", peaked=1.0, seed=0):
    Dv = 2 * D if Dv is None else Dv
    g = torch.Generator().manual_seed(seed + Lq * 131 + Lk * 17 + H + D)
    dt = DT[kind]

    def new(*shape):
        return torch.randn(*shape, generator=g)

    q, k, v = new(B, Lq, H, 2, D) * peaked, new(B, Lk, Hk, 2, D), new(B, Lk, Hk, Dv)
    t = dict(q=q.to(dt), k=k.to(dt), v=v.to(dt), lam=torch.rand(H, generator=g) + 0.1)
    opt = dict(causal=causal, scale=scale)
    if buckets:
        t["bias_table"] = new(buckets, H)
        t["bucket_map"] = da.relative_buckets(buckets, reach)
    if pos == "frames":  # four keys' frames behind the queries' one, in order
        t["pos_q"] = torch.zeros(B, Lq, dtype=torch.int32)
        t["pos_k"] = -(torch.arange(Lk) * 4 // max(Lk, 1)).to(torch.int32).expand(B, Lk).contiguous()
    elif pos == "random":
        t["pos_q"] = torch.randint(-50, 50, (B, Lq), generator=g, dtype=torch.int32)
        t["pos_k"] = torch.randint(-50, 50, (B, Lk), generator=g, dtype=torch.int32)
    elif pos == "far":
        t["pos_q"] = torch.randint(-(1 << 30) + 1, 1 << 30, (B, Lq), generator=g, dtype=torch.int32)
        t["pos_k"] = torch.randint(-(1 << 30) + 1, 1 << 30, (B, Lk), generator=g, dtype=torch.int32)
    if mask is not None:
        t["key_mask"] = torch.rand(B, Lk, generator=g) < mask
        t["key_mask"][-1, : Lk // 2] = False
    if lengths is not None:
        t["key_lengths"] = torch.tensor(lengths, dtype=torch.int32)
    grad = new(B, Lq, H, Dv).to(dt)
    t = {n: x.cuda() for n, x in t.items()}
    if layout == "heads first":  # [B, H, L, ..] storage
        for n in ("q", "k", "v"):
            t[n] = t[n].transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "packed":  # one projection's output holds q, k and v; an odd offset breaks 16-byte alignment
        n = [t[x].reshape(B, -1, t[x].shape[2] * t[x][0, 0, 0].numel()) for x in ("q", "k", "v")]
        both = torch.cat(n, 2).contiguous()
        a, b = n[0].shape[2], n[0].shape[2] + n[1].shape[2]
        t["q"] = both[..., :a].view(B, Lq, H, 2, D)
        t["k"] = both[..., a:b].view(B, Lk, Hk, 2, D)
        t["v"] = both[..., b:].view(B, Lk, Hk, Dv)
    elif layout == "odd offset":
        for n in ("q", "k", "v"):
            x = torch.empty(t[n].numel() + 1, dtype=dt, device="cuda")[1:].view(t[n].shape)
            t[n] = x.copy_(t[n])
    elif layout == "maps outside":  # [2, B, L, H, D] storage
        for n in ("q", "k"):
            t[n] = t[n].permute(3, 0, 1, 2, 4).contiguous().permute(1, 2, 3, 0, 4)
    return t, opt, grad.cuda()


CASES = {
    "one by one": dict(Lq=1, Lk=1),
    "one key": dict(B=2, Lq=70, Lk=1, buckets=4, kind="bf16"),
    "one query": dict(Lq=1, Lk=65, H=4, causal=True, buckets=8),
    "one query, shared, long": dict(B=2, Lq=1, Lk=3001, H=8, Hk=2, causal=True, buckets=16, reach=64, lengths=[3001, 1700]),
    "one query, long, bf16": dict(B=2, Lq=1, Lk=3001, H=8, Hk=2, D=64, kind="bf16", causal=True, buckets=16, reach=64,
                                  lengths=[3001, 1700]),
    "three queries, long, f16": dict(B=1, Lq=3, Lk=2500, H=6, Hk=2, D=64, kind="f16", causal=True, buckets=32, reach=128),
    "tile": dict(B=2, Lq=128, Lk=128, kind="bf16", buckets=8),
    "tile edges": dict(Lq=129, Lk=257, kind="bf16", causal=True, buckets=32, reach=128),
    "tile edges f16": dict(Lq=127, Lk=255, H=4, Hk=1, D=64, kind="f16", causal=True, buckets=32, reach=100),
    "plain f32": dict(B=2, Lq=100, Lk=90, H=4, Hk=2),
    "plain bf16": dict(B=2, Lq=100, Lk=90, H=4, Hk=2, kind="bf16"),
    "frames bf16": dict(B=2, Lq=150, Lk=300, H=4, Hk=4, kind="bf16", buckets=32, reach=128, pos="frames", mask=0.8),
    "frames f32": dict(B=2, Lq=70, Lk=130, H=4, Hk=4, buckets=32, reach=128, pos="frames", mask=0.8),
    "random positions": dict(B=2, Lq=90, Lk=110, kind="bf16", buckets=32, reach=40, pos="random", causal=True),
    "random positions f32": dict(B=2, Lq=90, Lk=110, buckets=32, reach=40, pos="random", causal=True),
    "far positions": dict(Lq=40, Lk=70, kind="bf16", buckets=8, pos="far", causal=True),
    "more queries than keys": dict(B=2, Lq=200, Lk=60, kind="bf16", causal=True, buckets=8),
    "more queries than keys f32": dict(B=2, Lq=200, Lk=60, causal=True, buckets=8),
    "lengths": dict(B=4, Lq=33, Lk=200, kind="bf16", buckets=8, lengths=[0, 1, 64, 200]),
    "lengths out of range": dict(B=2, Lq=33, Lk=100, kind="bf16", lengths=[-5, 1000]),
    "lengths causal f32": dict(B=4, Lq=33, Lk=200, causal=True, buckets=8, lengths=[0, 1, 64, 200]),
    "shared by three": dict(B=1, Lq=100, Lk=140, H=6, Hk=2, D=64, kind="bf16", causal=True, buckets=16, reach=50),
    "shared by twelve": dict(B=1, Lq=50, Lk=140, H=12, Hk=1, kind="f16", buckets=16, reach=50),
    "width 24": dict(Lq=140, Lk=150, H=3, Hk=3, D=24, kind="bf16", buckets=8),
    "width 16": dict(Lq=140, Lk=150, D=16, kind="f16", causal=True),
    "width 40": dict(Lq=100, Lk=150, D=40, kind="bf16", causal=True, buckets=32, reach=32),
    "width 17": dict(Lq=60, Lk=70, D=17, Dv=33, kind="bf16", buckets=8),
    "value width apart": dict(Lq=60, Lk=200, D=64, Dv=40, kind="bf16", buckets=8),
    "width 128": dict(Lq=60, Lk=70, D=128, kind="bf16", causal=True, buckets=8),
    "width 128 f32": dict(Lq=40, Lk=70, D=128, buckets=8),
    "width 1": dict(Lq=20, Lk=30, D=1, Dv=1),
    "peaked": dict(B=1, Lq=130, Lk=400, kind="bf16", buckets=8, peaked=6.0),
    "peaked f16": dict(B=1, Lq=130, Lk=400, D=64, kind="f16", causal=True, peaked=6.0),
    "heads first": dict(B=2, Lq=90, Lk=130, H=4, Hk=2, kind="bf16", layout="heads first"),
    "packed": dict(B=2, Lq=90, Lk=90, H=4, Hk=4, kind="bf16", layout="packed", causal=True, buckets=8),
    "odd offset": dict(B=2, Lq=90, Lk=90, H=4, Hk=4, kind="f16", layout="odd offset", buckets=8),
    "maps outside": dict(B=2, Lq=90, Lk=100, H=4, Hk=2, kind="bf16", layout="maps outside"),
    "negative scale": dict(Lq=50, Lk=60, kind="bf16", scale=-0.3),
    "no scale": dict(Lq=50, Lk=60, kind="bf16", scale=0.0, buckets=8),
    "longer": dict(B=1, Lq=700, Lk=1100, H=4, Hk=2, D=64, kind="bf16", causal=True, buckets=32, reach=128),
    "longer f16": dict(B=1, Lq=513, Lk=900, H=2, Hk=2, D=64, kind="f16", buckets=32, reach=128),
    "widest table": dict(Lq=130, Lk=300, H=16, Hk=1, kind="bf16", buckets=32, reach=1024),
}


def _all(t, opt, grad):
    out, saved = da.dattn_forward(**t, **opt, keep_for_backward=True)
    args = {n: x for n, x in t.items() if n not in ("q", "k", "v", "lam")}
    g = da.dattn_backward(t["q"], t["k"], t["v"], t["lam"], out, saved, grad, **args, **opt)
    r = dict(zip(("grad_q", "grad_k", "grad_v", "grad_lam", "grad_table"), g), out=out)
    if r["grad_table"] is None:
        del r["grad_table"]
    return r


def _reference(t, opt, grad):
    names = {"bias_table": "table"}
    return dattn_reference(**{names.get(n, n): x for n, x in t.items()}, **opt, grad=grad)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_against_64_bits(name):
    t, opt, grad = _case(**CASES[name])
    val, tol = _reference(t, opt, grad)
    only = da.dattn_forward(**t, **opt)
    check({"out": only}, {"out": val["out"]}, tol, "forward alone")
    got = _all(t, opt, grad)
    assert torch.equal(got["out"], only)
    check(got, val, tol)
    again = _all(t, opt, grad)
    assert all(torch.equal(got[n], again[n]) for n in got), "results vary from run to run"


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D", [("f32", 32), ("bf16", 32), ("f16", 64), ("bf16", 17)])
def test_what_masked_places_hold_is_not_used(kind, D):
    t, opt, grad = _case(B=3, Lq=75, Lk=300, H=4, Hk=2, D=D, kind=kind, mask=0.6, lengths=[300, 130, 0], buckets=8, causal=True)
    t["key_mask"][0, 64:200] = False
    want = _all(t, opt, grad)
    there = (torch.arange(300, device="cuda")[None] < t["key_lengths"][:, None]) & t["key_mask"]
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(DT[kind]).min):
        u = {**t, "k": t["k"].masked_fill(~there[:, :, None, None, None], bad), "v": t["v"].masked_fill(~there[:, :, None, None], bad)}
        u["q"] = t["q"].clone()
        u["q"][2] = bad  # this item's queries see no key
        g = grad.clone()
        g[2] = bad
        got = _all(u, opt, g)
        assert all(torch.equal(got[n], want[n]) for n in got), bad
    assert not want["out"][2].any() and not want["grad_q"][2].any() and not want["grad_k"][2].any()
    assert not want["grad_k"][~there].any() and not want["grad_v"][~there].any()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_masks_that_leave_rows_empty(kind):
    t, opt, grad = _case(B=2, Lq=140, Lk=150, kind=kind, buckets=8, causal=True)
    t["pos_q"] = torch.arange(140, dtype=torch.int32, device="cuda").expand(2, 140).contiguous() - 70  # half see nothing
    t["pos_k"] = torch.arange(150, dtype=torch.int32, device="cuda").expand(2, 150).contiguous()
    val, tol = _reference(t, opt, grad)
    got = _all(t, opt, grad)
    check(got, val, tol)
    assert not got["out"][:, :70].any() and not got["grad_q"][:, :70].any()
    t["key_mask"] = torch.zeros(2, 150, dtype=torch.bool, device="cuda")
    got = _all(t, opt, grad)
    assert not any(x.any() for x in got.values())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_rows_of_one_key_give_exactly_no_score_gradient(kind):
    # A softmax over one key is 1 whatever its score.
    for Lk, lengths in ((1, None), (40, [1, 1]), (200, [1, 1])):
        t, opt, grad = _case(B=2, Lq=70, Lk=Lk, H=4, Hk=2, kind=kind, buckets=8, lengths=lengths)
        got = _all(t, opt, grad)
        assert not got["grad_q"].any() and not got["grad_k"].any() and not got["grad_table"].any()
        assert bool(got["grad_v"].any()) and bool(got["grad_lam"].all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_two_keys_keep_their_digits(kind):
    # grad_q of two keys is their scores' difference: no more than 1.7 times
    # the two roundings (of s_m and of the result) may be off, in 2-norm.
    t, opt, grad = _case(B=4, Lq=64, Lk=2, H=4, Hk=4, kind=kind)
    val, _ = _reference(t, opt, grad)
    got = _all(t, opt, grad)
    for n in ("grad_q", "grad_k"):
        assert float((got[n].double() - val[n]).norm() / val[n].norm()) < 1.7 * torch.finfo(DT[kind]).eps / 2


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_infinite_bias(kind):
    # A bucket of -infinity hides its keys; a row with no other keys gives 0.
    t, opt, grad = _case(Lq=80, Lk=80, kind=kind, buckets=8, reach=16)
    t["bias_table"][:4] = -float("inf")
    t["bias_table"][4] = -float("inf")  # only later keys, from the second on, are left
    got = da.dattn_forward(**t, **opt)
    u = {n: x for n, x in t.items()}
    u["bias_table"] = t["bias_table"].clamp(min=-50)  # e^-50 is far below every rounding here
    rel = torch.arange(80, device="cuda")[None] - torch.arange(80, device="cuda")[:, None]
    seen = t["bias_table"][t["bucket_map"].long()[rel.clamp(-16, 16) + 16]][..., 0] > -1e30
    val, tol = dattn_reference(u["q"], u["k"], u["v"], u["lam"], u["bias_table"], u["bucket_map"])
    some = seen.any(1)
    assert bool(some.any()) and not bool(some.all())
    check({"out": got[:, some]}, {"out": val["out"][:, some]}, {"out": tol["out"][:, some]})
    assert not got[:, ~some].any()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_lowest_finite_bias_hides_as_infinity_does(kind):
    t, opt, grad = _case(Lq=150, Lk=150, kind=kind, buckets=8, reach=16, causal=True)
    got = []
    for hidden in (-float("inf"), torch.finfo(torch.float32).min):
        u = {**t, "bias_table": t["bias_table"].clone()}
        u["bias_table"][:2] = hidden  # the key at the query's own place and the one before it
        got.append(_all(u, opt, grad))
    assert all(torch.equal(got[0][n], got[1][n]) for n in got[0])
    assert not got[0]["out"][:, :2].any() and bool(got[0]["out"][:, 2:].any(-1).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_empty_sizes(kind):
    for Lq, Lk in ((0, 5), (5, 0), (0, 0)):
        t, opt, grad = _case(B=2, Lq=Lq, Lk=Lk, kind=kind, buckets=4)
        got = _all(t, opt, grad)
        assert got["out"].shape == (2, Lq, 2, 64) and not any(x.any() for x in got.values())
    t, opt, grad = _case(B=2, Lq=3, Lk=3, kind=kind, buckets=4)
    t = {n: x[:0] if n in "qkv" else x for n, x in t.items()}
    got = _all(t, opt, grad[:0])
    assert not got["grad_lam"].any() and not got["grad_table"].any()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_broadcast_keys_and_autograd(kind):
    t, opt, grad = _case(B=3, Lq=50, Lk=70, H=4, Hk=2, kind=kind, buckets=8)
    base = {n: t[n][:1].clone().requires_grad_(True) for n in ("k", "v")}
    leaves = [t["q"].clone().requires_grad_(True), base["k"], base["v"], t["lam"].clone().requires_grad_(True),
              t["bias_table"].clone().requires_grad_(True)]
    out = da.DifferentialAttentionFunction.apply(leaves[0], base["k"].expand(3, -1, -1, -1, -1), base["v"].expand(3, -1, -1, -1),
                                                 leaves[3], leaves[4], t["bucket_map"], None, None, None, None, False, None)
    grads = torch.autograd.grad(out, leaves, grad)
    t["k"], t["v"] = t["k"][:1].expand(3, -1, -1, -1, -1), t["v"][:1].expand(3, -1, -1, -1)
    val, tol = _reference(t, opt, grad)
    got = dict(zip(("grad_q", "grad_k", "grad_v", "grad_lam", "grad_table"), grads), out=out.detach())
    for n in ("grad_k", "grad_v"):  # autograd sums the three items' gradients in the inputs' type
        step = torch.finfo(DT[kind]).eps
        tol[n] = tol[n].sum(0, keepdim=True) + 2 * step * val[n].abs().sum(0, keepdim=True)
        val[n] = val[n].sum(0, keepdim=True)
    check(got, val, tol)


@pytest.mark.gpu
def test_streams_and_graph_capture():
    t, opt, grad = _case(B=2, Lq=130, Lk=200, H=4, Hk=2, kind="bf16", buckets=8, causal=True)
    want = _all(t, opt, grad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = {n: x for n, x in t.items() if n not in ("q", "k", "v", "lam")}
    out, saved = da.dattn_forward(**t, **opt, keep_for_backward=True, stream=side)
    g = da.dattn_backward(t["q"], t["k"], t["v"], t["lam"], out, saved, grad, **args, **opt, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want["out"]) and torch.equal(g[1], want["grad_k"]) and torch.equal(g[4], want["grad_table"])
    static = {n: torch.zeros_like(x) if n in ("q", "k", "v") else x for n, x in t.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = _all(static, opt, grad)
    for sign in (1, -1):
        for n in ("q", "k", "v"):
            static[n].copy_(t[n] * sign)
        graph.replay()
        want = _all({n: x * sign if n in ("q", "k", "v") else x for n, x in t.items()}, opt, grad)
        assert all(torch.equal(r[n], want[n]) for n in r)


def _off_by_one(x):
    """The same values one element further in memory."""
    y = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)[1:].view(x.shape)
    return y.copy_(x)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D", [("f32", 32), ("bf16", 32), ("f16", 64), ("bf16", 20)])
@pytest.mark.parametrize("odd", ["out", "saved", "grad"])
def test_outputs_and_gradients_of_odd_alignment(kind, D, odd):
    # The backward pass then takes the general kernels, after any forward.
    t, opt, grad = _case(B=2, Lq=90, Lk=130, H=4, Hk=2, D=D, kind=kind, buckets=8, causal=True)
    out, saved = da.dattn_forward(**t, **opt, keep_for_backward=True)
    if odd == "out":
        aligned, out = out, _off_by_one(torch.zeros_like(out))
        again, saved = da.dattn_forward(**t, **opt, out=out, keep_for_backward=True)
        assert again.data_ptr() == out.data_ptr() and torch.equal(out, aligned)
    elif odd == "saved":
        saved = tuple(_off_by_one(x) for x in saved)
    else:
        grad = _off_by_one(grad)
    args = {n: x for n, x in t.items() if n not in ("q", "k", "v", "lam")}
    g = da.dattn_backward(t["q"], t["k"], t["v"], t["lam"], out, saved, grad, **args, **opt)
    val, tol = _reference(t, opt, grad)
    check(dict(zip(("grad_q", "grad_k", "grad_v", "grad_lam", "grad_table"), g), out=out), val, tol)


@pytest.mark.gpu
def test_saved_of_another_type_is_refused():
    t, opt, grad = _case(Lq=4, Lk=4, kind="bf16")
    out, (out1, lse) = da.dattn_forward(**t, **opt, keep_for_backward=True)
    for bad in ((out1.half(), lse), (out1[:, :, :, :1], lse), (out1, lse.double()), (out1, lse[:, :1])):
        with pytest.raises(ValueError, match="saved"):
            da.dattn_backward(t["q"], t["k"], t["v"], t["lam"], out, bad, grad)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_offsets_past_32_bits(kind):
    # The second item's keys lie more than 2^31 elements past the first's.
    t, opt, grad = _case(B=2, Lq=5, Lk=140, kind=kind, buckets=8)
    want = _all(t, opt, grad)
    gap = (1 << 31) + 64
    for n in ("k", "v"):
        one = t[n][0].numel()
        store = torch.empty(gap + one, dtype=t[n].dtype, device="cuda")
        far = torch.as_strided(store, t[n].shape, (gap, *t[n].stride()[1:]))
        t[n] = far.copy_(t[n])
    got = _all(t, opt, grad)
    assert all(torch.equal(got[n], want[n]) for n in got)


@pytest.mark.gpu
def test_fp16_scales_in_a_graph_on_another_stream_and_far_apart():
    # fp16 takes a maximum over v and one over grad_out before its products.
    t, opt, grad = _case(B=2, Lq=130, Lk=200, H=4, Hk=2, D=64, kind="f16", buckets=8, causal=True, mask=0.8, lengths=[200, 150])
    static = {n: torch.zeros_like(x) if n in ("q", "k", "v") else x for n, x in t.items()}
    sgrad = torch.zeros_like(grad)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        r = _all(static, opt, sgrad)
    for size in (1.0, 2.0 ** -12, 2.0 ** 8):  # a maximum is not kept from one replay to the next
        for n in ("q", "k", "v"):
            static[n].copy_(t[n])
        sgrad.copy_(grad * size)
        graph.replay()
        want = _all(t, opt, grad * size)
        assert all(torch.equal(r[n], want[n]) for n in r)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _all(t, opt, grad * size)
    torch.cuda.current_stream().wait_stream(side)
    gap = (1 << 31) + 64
    for n in ("k", "v"):
        store = torch.empty(gap + t[n][0].numel(), dtype=t[n].dtype, device="cuda")
        t[n] = torch.as_strided(store, t[n].shape, (gap, *t[n].stride()[1:])).copy_(t[n])
    far = _all(t, opt, grad * size)
    assert all(torch.equal(other[n], want[n]) and torch.equal(far[n], want[n]) for n in want)


@pytest.mark.gpu
def test_tensors_off_the_gpu_are_refused():
    t, opt, _ = _case(Lq=4, Lk=4)
    with pytest.raises(ValueError, match="CUDA"):
        da.dattn_forward(**{**t, "k": t["k"].cpu()}, **opt)
    with pytest.raises(ValueError, match="contiguous"):
        da.dattn_forward(**{**t, "v": t["v"].transpose(1, 3).contiguous().transpose(1, 3)}, **opt)
    with pytest.raises(ValueError, match="lam"):
        da.dattn_forward(**{**t, "lam": t["lam"][:1]}, **opt)
