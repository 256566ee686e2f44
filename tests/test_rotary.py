"""Rotary norm of queries and keys (qkr_forward, qkr_backward,
QkRotaryFunction, rotary_frequencies): refusals and host logic on the CPU,
results on the GPU against 64 bits."""
import ctypes
import math

import pytest
import torch

import deformable_view_feature_gb300 as da
from operator_refs import check
from serving_refs import QkrProblem, qkr_reference, radians, serving_library

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FAKE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    da.build.build()
    return serving_library(da.load_library())


# ---- refusals and host logic: no GPU, nothing is launched ------------------

def _problem(**kw):
    d = dict(batch=1, num_queries=4, num_keys=8, num_heads=4, num_kv_heads=2, width=32, rotated=32, dtype=1, normed=1, eps=1e-6,
             magnitude=1.0, q=FAKE, k=FAKE, q_weight=FAKE, k_weight=FAKE, turns=FAKE)
    stride = kw.pop("q_stride", (1024, 256, 64, 32))
    d.update(kw)
    p = QkrProblem(**d)
    p.q_stride[:] = stride
    p.k_stride[:] = (1024, 128, 64, 32)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(batch=-1), 2), (dict(num_queries=-1), 2), (dict(num_keys=-1), 2), (dict(num_heads=0), 2), (dict(width=0), 2),
    (dict(width=129), 4), (dict(rotated=34), 2), (dict(rotated=31), 2), (dict(rotated=-2), 2), (dict(rotated=0, turns=None), 0),
    (dict(turns=None), 1), (dict(dtype=4), 2), (dict(eps=0.0), 2), (dict(eps=float("inf")), 2), (dict(eps=float("nan")), 2),
    (dict(normed=0), 2), (dict(normed=0, q_weight=None, k_weight=None, eps=0.0), 0), (dict(magnitude=float("nan")), 2),
    (dict(q_stride=(1024, -1, 64, 32)), 2), (dict(batch=1 << 20, num_keys=1 << 12), 4), (dict(q=FAKE + 1), 3), (dict(q_weight=FAKE + 2), 3),
    (dict(turns=FAKE + 4), 3), (dict(q=None), 1), (dict(q=None, num_queries=0), 0), (dict(k=None, num_keys=0), 0),
])
def test_problems_are_checked(lib, kw, status):
    assert lib.qkr_workspace_size(ctypes.byref(_problem(**kw)), ctypes.byref(ctypes.c_size_t(0))) == status


def test_buffers_are_checked(lib):
    vp = ctypes.c_void_p
    p = _problem()
    assert lib.qkr_forward(ctypes.byref(p), None, vp(FAKE), None) == 1 and lib.qkr_forward(ctypes.byref(p), vp(FAKE), None, None) == 1
    assert lib.qkr_forward(ctypes.byref(p), vp(FAKE + 1), vp(FAKE), None) == 3 and lib.qkr_forward(None, None, None, None) == 1
    n = ctypes.c_size_t(0)
    assert lib.qkr_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0

    def backward(size=n.value, ws=FAKE, p=p, **kw):
        args = {k: FAKE for k in ("grad_out_q", "grad_out_k", "grad_q", "grad_k", "grad_q_weight", "grad_k_weight")}
        args.update(kw)
        return lib.qkr_backward(ctypes.byref(p), *[vp(x) for x in args.values()], vp(ws), size, None)

    for name in ("grad_out_q", "grad_out_k", "grad_q", "grad_k", "grad_q_weight", "grad_k_weight"):
        assert backward(**{name: None}) == 1, name
    assert backward(p=_problem(q_weight=None)) == 1  # a gradient without its weight
    assert backward(size=n.value - 1) == 6 and backward(ws=None) == 6 and backward(ws=FAKE + 64) == 6
    assert backward(grad_out_q=FAKE + 1) == 3 and backward(grad_k_weight=FAKE + 1) == 3


def test_nothing_to_do(lib):
    p = _problem(num_queries=0, num_keys=0, q=None, k=None)
    assert lib.qkr_forward(ctypes.byref(p), None, None, None) == 0


def test_binding_checks_shapes_and_types():
    q, k, w, f = torch.zeros(1, 3, 4, 2, 8), torch.zeros(1, 5, 2, 2, 8), torch.ones(8), torch.zeros(4, dtype=torch.int64)
    for bad in ((q[0], k), (q[..., :1, :], k), (q, k[..., :4]), (torch.zeros(2, 3, 4, 2, 8), k), (None, None)):
        with pytest.raises(ValueError):
            da.qkr_forward(*bad)
    for bad in ((q.double(), None), (q, k.half())):
        with pytest.raises(TypeError):
            da.qkr_forward(*bad)
    for kw in (dict(frequencies=f.float()), dict(frequencies=f[None]), dict(q_weight=w[:4]), dict(q_weight=w.half()),
               dict(pos_q=torch.zeros(1, 4, dtype=torch.int32)), dict(pos_q=torch.zeros(1, 3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            da.qkr_forward(q, k, **kw)
    with pytest.raises(ValueError, match="norm"):
        da.qkr_forward(q, k, q_weight=w, eps=None)
    with pytest.raises(ValueError, match="go with k"):
        da.qkr_forward(q, k_weight=w)
    with pytest.raises(ValueError, match="no input"):
        da.qkr_forward(q, out_k=k)
    with pytest.raises(ValueError, match="out_k must be"):
        da.qkr_forward(q, k, out_k=k[:, :1])
    with pytest.raises(ValueError, match="CUDA device"):
        da.qkr_forward(q, k)
    with pytest.raises(TypeError):
        da.qkr_forward(q, [k])
    with pytest.raises(TypeError):
        da.qkr_forward(q, k, eps="x")
    for grads in ((q, None), (q[:, :2], k), (q.half(), k)):
        with pytest.raises(ValueError):
            da.qkr_backward(q, k, *grads)


def test_frequencies():
    f = radians(da.rotary_frequencies(64))
    for i, x in enumerate(f):
        assert abs(x - 10000.0 ** (-i / 32)) <= 2 ** -52 * x + 2 ** -61
    assert radians(da.rotary_frequencies(8, 500.0, 4.0)) == pytest.approx([500.0 ** (-i / 4) / 4 for i in range(4)], rel=1e-14)
    based = radians(da.rotary_frequencies(8, 500.0, 4.0, "base"))
    assert based[0] == pytest.approx(1.0, rel=1e-14) and based[3] == pytest.approx(500.0 ** (-3 / 4) / 4, rel=1e-13)
    parts = radians(da.rotary_frequencies(64, 10000.0, 8.0, "parts", original_length=4096))
    plain = [10000.0 ** (-i / 32) for i in range(32)]
    assert parts[0] == pytest.approx(plain[0], rel=1e-14)          # 650 turns within the length
    assert parts[31] == pytest.approx(plain[31] / 8, rel=1e-14)    # less than one
    mid = next(i for i in range(32) if 1 < 4096 * plain[i] / (2 * math.pi) < 32)
    keep = (4096 * plain[mid] / (2 * math.pi) - 1) / 31
    assert parts[mid] == pytest.approx(plain[mid] * (keep + (1 - keep) / 8), rel=1e-13)
    fast = da.rotary_frequencies(2, 1.0, 0.2)                      # 5 radians: more than half a turn is a negative number
    assert int(fast[0]) < 0 and math.cos(radians(fast)[0]) == pytest.approx(math.cos(5.0), rel=1e-12)
    for bad in (dict(rotated=3), dict(rotated=0), dict(rotated=8, base=0.0), dict(rotated=8, stretch=float("inf")),
                dict(rotated=8, method="x"), dict(rotated=8, method="parts"), dict(rotated=2, method="base")):
        with pytest.raises(ValueError):
            da.rotary_frequencies(**bad)


@pytest.mark.parametrize("interleaved", [False, True])
def test_references_gradients_against_differences(interleaved):
    g = torch.Generator().manual_seed(3)
    x, gr = (torch.randn(1, 2, 2, 2, 6, generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(6, generator=g, dtype=torch.float64)
    opt = dict(turns=da.rotary_frequencies(4), pos=torch.tensor([[3, -70000]]), eps=0.1, interleaved=interleaved, magnitude=1.3)

    def f(x, w):
        # float64 tensors: the reference reads the step of their own type
        return float((qkr_reference(x, weight=w, **opt)[0]["out"] * gr).sum())

    val, _ = qkr_reference(x, weight=w, grad=gr, **opt)
    for t, got in ((x, val["grad_x"]), (w, val["grad_weight"])):
        for i in range(t.numel()):
            d = torch.zeros_like(t).reshape(-1)
            d[i] = 1e-5
            d = d.reshape(t.shape)
            slope = (f(x + d, w) - f(x - d, w)) / 2e-5 if t is x else (f(x, w + d) - f(x, w - d)) / 2e-5
            assert abs(slope - float(got.reshape(-1)[i])) < 1e-8


# ---- results ---------------------------------------------------------------

def _case(B=1, Lq=5, Lk=5, H=2, Hk=2, D=32, R=None, kind="f32", interleaved=False, weights=True, eps=1e-6, magnitude=1.0, pos=None,
          layout="plain", only=None, size=1.0, seed=0):
    g = torch.Generator().manual_seed(seed + Lq * 131 + Lk * 17 + H + D)
    dt = DT[kind]
    R = D // 2 * 2 if R is None else R
    t = {"q": (torch.randn(B, Lq, H, 2, D, generator=g) * size).to(dt), "k": (torch.randn(B, Lk, Hk, 2, D, generator=g) * size).to(dt)}
    grad = {n: torch.randn(x.shape, generator=g).to(dt) for n, x in t.items()}
    opt = dict(eps=eps, interleaved=interleaved, magnitude=magnitude)
    if R:
        opt["frequencies"] = da.rotary_frequencies(R)
    if weights and eps is not None:
        opt["q_weight"], opt["k_weight"] = torch.randn(D, generator=g), torch.randn(D, generator=g) + 1
    if pos == "far":
        opt["pos_q"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, Lq), generator=g).to(torch.int32)
        opt["pos_k"] = torch.randint(0, 1 << 20, (B, Lk), generator=g, dtype=torch.int32)
    elif pos == "frames":
        opt["pos_q"], opt["pos_k"] = torch.zeros(B, Lq, dtype=torch.int32), -torch.arange(Lk, dtype=torch.int32).expand(B, Lk).contiguous()
    for n in ("q", "k"):
        if only not in (None, n):
            t[n] = grad[n] = None
            for x in (f"{n}_weight", f"pos_{n}"):
                opt.pop(x, None)
    t, grad, opt = ({n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in d.items()} for d in (t, grad, opt))
    for n, x in t.items():
        if x is None:
            continue
        if layout == "heads first":
            t[n] = x.transpose(1, 2).contiguous().transpose(1, 2)
        elif layout == "maps outside":
            t[n] = x.permute(3, 0, 1, 2, 4).contiguous().permute(1, 2, 3, 0, 4)
        elif layout == "odd offset":
            t[n] = torch.empty(x.numel() + 1, dtype=dt, device="cuda")[1:].view(x.shape).copy_(x)
        elif layout == "odd stride":
            wide = torch.zeros(*x.shape[:3], 2, D + 3, dtype=dt, device="cuda")
            wide[..., :D] = x
            t[n] = wide[..., :D]
        elif layout == "broadcast":
            t[n] = x[:, :1].expand(x.shape)
    return t, opt, grad


CASES = {
    "one token": dict(Lq=1, Lk=1),
    "one token bf16": dict(Lq=1, Lk=1, H=16, Hk=4, D=64, kind="bf16"),
    "plain": dict(B=2, Lq=37, Lk=50, H=4),
    "plain bf16": dict(B=2, Lq=37, Lk=50, H=4, D=64, kind="bf16"),
    "plain f16 interleaved": dict(B=3, Lq=20, Lk=33, H=6, Hk=3, D=64, kind="f16", interleaved=True),
    "more queries than keys": dict(B=2, Lq=9, Lk=4, kind="bf16"),
    "interleaved f32": dict(B=2, Lq=9, Lk=14, D=24, R=16, interleaved=True),
    "interleaved, odd pairs": dict(B=2, Lq=9, Lk=14, D=24, R=12, interleaved=True, kind="bf16"),
    "part": dict(B=2, Lq=9, Lk=14, D=48, R=24, kind="bf16"),
    "part, odd pieces": dict(B=2, Lq=9, Lk=14, D=40, R=16, kind="f16"),
    "odd half": dict(B=2, Lq=9, Lk=14, D=40, R=20, kind="f16"),
    "odd pairs": dict(B=2, Lq=9, Lk=14, D=24, R=6, kind="bf16"),
    "odd width": dict(B=2, Lq=9, Lk=14, D=33, R=14, kind="bf16"),
    "odd width f32": dict(B=2, Lq=9, Lk=14, D=17),
    "width 1": dict(Lq=3, Lk=4, D=1),
    "width 2": dict(Lq=3, Lk=4, D=2, kind="f16"),
    "width 128": dict(B=2, Lq=9, Lk=14, D=128, kind="bf16"),
    "width 128 f32": dict(B=2, Lq=9, Lk=14, D=128, interleaved=True),
    "width 127": dict(B=1, Lq=9, Lk=14, D=127, R=126, kind="bf16"),
    "no rotation": dict(B=2, Lq=9, Lk=14, R=0, kind="bf16"),
    "no norm": dict(B=2, Lq=9, Lk=14, eps=None, kind="bf16"),
    "no norm f32": dict(B=2, Lq=9, Lk=14, eps=None, magnitude=0.7),
    "neither": dict(B=2, Lq=9, Lk=14, eps=None, R=0),
    "no weights": dict(B=2, Lq=9, Lk=14, weights=False, kind="f16"),
    "magnitude": dict(B=2, Lq=9, Lk=14, R=16, magnitude=1.25, kind="f16"),
    "far": dict(B=3, Lq=9, Lk=14, pos="far"),
    "far bf16": dict(B=3, Lq=9, Lk=14, D=64, pos="far", kind="bf16", interleaved=True),
    "frames": dict(B=3, Lq=9, Lk=14, pos="frames", kind="bf16"),
    "queries alone": dict(B=2, Lq=9, only="q", kind="bf16", Lk=4),
    "keys alone": dict(B=2, Lk=9, only="k", Lq=4),
    "small values": dict(B=2, Lq=9, Lk=14, size=1e-4),
    "large values": dict(B=2, Lq=9, Lk=14, size=1e4, kind="bf16"),
    "heads first": dict(B=2, Lq=9, Lk=14, H=4, kind="bf16", layout="heads first"),
    "maps outside": dict(B=2, Lq=9, Lk=14, H=4, kind="f16", layout="maps outside"),
    "odd offset": dict(B=2, Lq=9, Lk=14, H=4, kind="bf16", layout="odd offset"),
    "odd offset f32": dict(B=2, Lq=9, Lk=14, H=4, layout="odd offset"),
    "odd stride": dict(B=2, Lq=9, Lk=14, H=4, kind="bf16", layout="odd stride"),
    "broadcast": dict(B=2, Lq=9, Lk=14, H=4, kind="bf16", layout="broadcast"),
    "many heads": dict(B=2, Lq=3, Lk=14, H=65, Hk=1, kind="bf16"),
    "many tokens": dict(B=3, Lq=1501, Lk=2100, H=3, Hk=1, D=64, kind="bf16"),
    "many tokens f32": dict(B=6, Lq=1000, Lk=2100, H=6, Hk=2, D=24, R=16, interleaved=True),
    "many small tokens": dict(B=8, Lq=4097, Lk=5001, H=1, Hk=1, D=16, R=8, kind="f16"),
}


def _all(t, opt, grad):
    o = {n: x for n, x in opt.items()}
    q, k = da.qkr_forward(t["q"], t["k"], **o)
    gq, gk, gwq, gwk = da.qkr_backward(t["q"], t["k"], grad["q"], grad["k"], **o)
    return {"q": dict(out=q, grad_x=gq, grad_weight=gwq), "k": dict(out=k, grad_x=gk, grad_weight=gwk)}


def _reference(t, opt, grad, n):
    x = t[n]
    B, L = x.shape[:2]
    pos = opt.get("pos_" + n)
    if pos is None:
        first = t["k"].shape[1] - L if n == "q" and t["k"] is not None else 0
        pos = (torch.arange(L, device="cuda") + first).expand(B, L)
    return qkr_reference(x, opt.get("frequencies"), opt.get(n + "_weight"), pos, opt["eps"], opt["interleaved"], opt["magnitude"], grad[n])


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_against_64_bits(name):
    t, opt, grad = _case(**CASES[name])
    got, again = _all(t, opt, grad), _all(t, opt, grad)
    for n in ("q", "k"):
        if t[n] is None:
            assert all(x is None for x in got[n].values())
            continue
        val, tol = _reference(t, opt, grad, n)
        if opt.get(n + "_weight") is None:
            assert got[n].pop("grad_weight") is None
            del val["grad_weight"]
        check(got[n], val, tol, n)
        assert all(torch.equal(x, again[n][m]) for m, x in got[n].items()), "results vary from run to run"


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D,R", [("bf16", 64, 64), ("f32", 24, 10)])
def test_in_place(kind, D, R):
    t, opt, _ = _case(B=2, Lq=50, Lk=70, H=5, kind=kind, D=D, R=R)
    want = da.qkr_forward(t["q"], t["k"], **opt)
    q, k = t["q"].clone(), t["k"].clone()
    got = da.qkr_forward(q, k, **opt, out_q=q, out_k=k)
    assert got[0] is q and got[1] is k and torch.equal(q, want[0]) and torch.equal(k, want[1])


@pytest.mark.gpu
def test_rotation_depends_on_differences_alone():
    """q at p and k at p + d: their product is that of 0 and d, however far p is."""
    f = da.rotary_frequencies(64).cuda()
    g = torch.Generator().manual_seed(0)
    q, k = (torch.randn(1, 1, 1, 2, 64, generator=g).cuda() for _ in range(2))

    def product(p, d):
        a, b = (torch.tensor([[x]], dtype=torch.int32, device="cuda") for x in (p, p + d))
        u, v = da.qkr_forward(q, k, f, pos_q=a, pos_k=b, eps=None)
        return (u.double() * v.double()).sum(-1).reshape(-1)

    for d in (0, 5, 1000):
        near = product(0, d)
        for p in (12345, 1 << 24, (1 << 31) - 2000, -(1 << 31)):
            # 2 * 64 terms, each with the tolerance of two rotated values
            assert float((product(p, d) - near).abs().max()) <= 2 * 64 * 2 * 8 * 2.0 ** -24 * float(q.abs().max() * k.abs().max()) * 2


@pytest.mark.gpu
def test_nan_stays_in_its_vector():
    t, opt, grad = _case(B=2, Lq=9, Lk=14, H=4, kind="bf16", weights=False)
    want = _all(t, opt, grad)
    t["q"][0, 3, 1, 1, 5] = float("nan")
    got = _all(t, opt, grad)
    for m in ("out", "grad_x"):
        bad = torch.isnan(got["q"][m]).any(-1)
        assert bool(bad[0, 3, 1, 1]) and int(bad.sum()) == 1
        assert torch.equal(got["q"][m][~bad], want["q"][m][~bad]) and torch.equal(got["k"][m], want["k"][m])


@pytest.mark.gpu
def test_zero_vectors():
    """A vector of zeros gives zeros and the gradient weight * g / sqrt(eps)."""
    x, w = torch.zeros(1, 2, 1, 2, 16, device="cuda"), torch.rand(16, device="cuda") + 0.5
    g = torch.randn(1, 2, 1, 2, 16, device="cuda")
    y, _ = da.qkr_forward(x, q_weight=w)
    gx, _, gw, _ = da.qkr_backward(x, None, g, None, q_weight=w)
    assert not bool(y.any()) and not bool(gw.any())
    assert bool(((gx - g * w * 1e3).abs() <= 4e-7 * (g * w * 1e3).abs()).all())  # 1e-6 in fp32, rsqrt, two products: 5 half-steps


@pytest.mark.gpu
def test_no_tokens():
    w = torch.ones(8, device="cuda")
    q, k = torch.zeros(2, 0, 3, 2, 8, device="cuda"), torch.randn(2, 3, 1, 2, 8, device="cuda")
    oq, ok = da.qkr_forward(q, k, q_weight=w, k_weight=w)
    assert oq.shape == q.shape and bool(torch.isfinite(ok).all())
    gq, gk, gwq, gwk = da.qkr_backward(q, k, q, k, q_weight=w, k_weight=w)
    assert gq.shape == q.shape and not bool(gwq.any()) and bool(gwk.any())
    gwq = da.qkr_backward(q, k[:, :0], q, k[:, :0], q_weight=w, k_weight=w)[2:]
    assert not bool(gwq[0].any()) and not bool(gwq[1].any())


@pytest.mark.gpu
def test_streams_and_graphs():
    t, opt, grad = _case(B=2, Lq=300, Lk=500, H=4, D=64, kind="bf16")
    want = _all(t, opt, grad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, k = da.qkr_forward(t["q"], t["k"], **opt, stream=side)
    back = da.qkr_backward(t["q"], t["k"], grad["q"], grad["k"], **opt, stream=side)
    side.synchronize()
    assert torch.equal(q, want["q"]["out"]) and torch.equal(k, want["k"]["out"]) and torch.equal(back[2], want["q"]["grad_weight"])
    graph = torch.cuda.CUDAGraph()
    src = {n: torch.zeros_like(x) for n, x in t.items()}
    with torch.cuda.graph(graph):
        got = _all(src, opt, grad)
    for n in ("q", "k"):
        src[n].copy_(t[n])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for n in ("q", "k"):
        assert all(torch.equal(x, want[n][m]) for m, x in got[n].items())


@pytest.mark.gpu
def test_autograd():
    t, opt, grad = _case(B=2, Lq=20, Lk=30, H=4, kind="bf16", layout="heads first")
    want = _all(t, opt, grad)
    leaves = [x.detach().requires_grad_(True) for x in (t["q"], t["k"], opt["q_weight"], opt["k_weight"])]
    q, k = da.QkRotaryFunction.apply(leaves[0], leaves[1], opt["frequencies"], leaves[2], leaves[3])
    got = torch.autograd.grad((q, k), leaves, (grad["q"], grad["k"]))
    for x, (n, m) in zip(got, (("q", "grad_x"), ("k", "grad_x"), ("q", "grad_weight"), ("k", "grad_weight"))):
        assert torch.equal(x, want[n][m])
    q, k = da.QkRotaryFunction.apply(leaves[0], leaves[1], opt["frequencies"], leaves[2], leaves[3])
    gq, gwk = torch.autograd.grad(q.float().sum(), [leaves[0], leaves[3]])  # nothing used the keys; a broadcast gradient
    assert bool(gq.any()) and not bool(gwk.any())
    q, none = da.QkRotaryFunction.apply(leaves[0], None, opt["frequencies"], leaves[2])
    assert none is None
    gq, = torch.autograd.grad(q.float().square().sum(), leaves[0], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (gq.float().square().sum() + leaves[0].float().sum()).backward()
