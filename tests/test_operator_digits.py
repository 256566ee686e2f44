"""Digits of the group norm and the differential attention on inputs that a
kernel may lose them on, against 64 bits."""
import pytest
import torch

import deformable_view_feature_gb300 as da
from operator_refs import check, dattn_reference, gn_reference

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    da.build.build()
    return da.load_library()


# ---- group norm ------------------------------------------------------------

@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shape,C,groups,first,rest", [
    ((16, 1000), 1, 1, 100.0, 0.0),     # one tile of one channel
    ((50, 100), 3, 1, 1000.0, 0.0),
    ((32, 64), 8, 2, 0.0, 100.0),       # a padded corner
    ((64, 64), 4, 1, 0.0, 100.0),
    ((32, 64), 8, 2, 1000.0, 0.0),      # one strong response
    ((150, 200), 64, 8, 1000.0, 0.0),   # in the first of many tiles
    ((150, 200), 20, 4, 0.0, 100.0),
])
def test_first_row_unlike_the_rest(shape, C, groups, first, rest, kind):
    g = torch.Generator().manual_seed(C)
    n = shape[0] * shape[1]
    x = torch.randn(1, n, C, generator=g) + rest
    x[:, 0] = first
    x = x.to(DT[kind]).cuda()
    gamma, beta = torch.randn(C, generator=g).cuda() * 0.3 + 1, torch.randn(C, generator=g).cuda() * 0.3
    grad = torch.randn(1, n, C, generator=g).to(DT[kind]).cuda()
    ss, ls = torch.tensor([[shape]], dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    out, stats = da.gn_forward(x, ss, ls, gamma, beta, groups)
    grads = da.gn_backward(x, ss, ls, gamma, beta, stats, grad, groups)
    val, tol = gn_reference(x, [(0, n, 0)], gamma[None], beta[None], groups, 1e-5, "none", grad)
    for d in (val, tol):
        d["grad_gamma"], d["grad_beta"] = d["grad_gamma"][0], d["grad_beta"][0]
    check({"out": out, "grad_feat": grads[0], "grad_gamma": grads[1], "grad_beta": grads[2]}, val, tol)
    # The variance itself: no more than the 32 roundings that the tolerance above counts.
    t = x.double().reshape(n, groups, -1)
    var = t.var((0, 2), correction=0) + 1e-5
    got = stats[0, 0, 0, :, 1].double() ** -2
    assert float(((got - var).abs() / var).max()) < 32 * 2.0 ** -24


# ---- differential attention ------------------------------------------------

NAMES = ("grad_q", "grad_k", "grad_v", "grad_lam", "grad_table")


def _both(t, opt, grad):
    """What the kernels give, and the reference's values and tolerances."""
    out, saved = da.dattn_forward(**t, **opt, keep_for_backward=True)
    rest = {n: x for n, x in t.items() if n not in ("q", "k", "v", "lam")}
    g = da.dattn_backward(t["q"], t["k"], t["v"], t["lam"], out, saved, grad, **rest, **opt)
    got = {"out": out, **{n: x for n, x in zip(NAMES, g) if x is not None}}
    val, tol = dattn_reference(**{"table" if n == "bias_table" else n: x for n, x in t.items()}, **opt, grad=grad)
    return got, val, tol


def _off(got, val, n):
    return float((got[n].double() - val[n]).norm() / val[n].norm())


def _normal(g, kind, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(DT[kind]).cuda()


@pytest.mark.parametrize("kind,D,layout", [("bf16", 32, "tensor"), ("f16", 64, "tensor"), ("bf16", 36, "general"), ("f16", 20, "general")])
@pytest.mark.parametrize("common", [1.0, 2.0])
def test_tokens_with_a_common_part(kind, D, layout, common):
    # q, k and v are projections of tokens that share a part `common` times
    # their own. s_m sums to 0 over the keys, so the common part of the keys
    # takes no part in grad_q, but the roundings of s_m meet it: in 2-norm
    # half a step times sqrt(1 + common^2) for these, and one for the result.
    g = torch.Generator().manual_seed(D)
    B, L, H, C = 1, 400, 4, 256
    x = torch.randn(B, L, C, generator=g) + common * torch.randn(C, generator=g)
    x = x / (1 + common ** 2) ** 0.5

    def project(*shape):
        n = 1
        for s in shape:
            n *= s
        return (x @ torch.randn(C, n, generator=g) / C ** 0.5).reshape(B, L, *shape).to(DT[kind]).cuda()

    t = dict(q=project(H, 2, D), k=project(H, 2, D), v=project(H, 2 * D), lam=torch.full((H,), 0.5).cuda())
    assert da.dattn_path(t["q"], t["k"], t["v"], t["lam"], backward=True) == layout
    got, val, tol = _both(t, dict(causal=False), _normal(g, kind, B, L, H, 2 * D))
    check(got, val, tol)
    step = torch.finfo(DT[kind]).eps / 2
    assert _off(got, val, "grad_q") < step * (1 + (1 + common ** 2) ** 0.5)


@pytest.mark.parametrize("kind,H,Hk,D", [("bf16", 2, 2, 32), ("f16", 2, 2, 64), ("bf16", 6, 2, 64), ("f32", 2, 2, 32),
                                         ("f32", 6, 2, 24), ("bf16", 2, 2, 20), ("f32", 2, 2, 72)])
def test_first_causal_rows(kind, H, Hk, D):
    # The first query sees one key: a softmax over one key is 1 whatever its
    # score. The next few keep their digits, as rows of few keys do elsewhere:
    # 1.7 times the two roundings (of s_m and of the result).
    g = torch.Generator().manual_seed(H + D)
    B, L = 2, 130
    t = dict(q=_normal(g, kind, B, L, H, 2, D), k=_normal(g, kind, B, L, Hk, 2, D), v=_normal(g, kind, B, L, Hk, 2 * D),
             lam=(torch.rand(H, generator=g) + 0.1).cuda(), bias_table=torch.randn(8, H, generator=g).cuda(),
             bucket_map=da.relative_buckets(8, 16).cuda())
    got, val, tol = _both(t, dict(causal=True), _normal(g, kind, B, L, H, 2 * D))
    check(got, val, tol)
    assert not got["grad_q"][:, 0].any()
    few = {n: x["grad_q"][:, 1:4] for n, x in (("got", got), ("val", val))}
    if kind != "f32":
        assert float((few["got"].double() - few["val"]).norm() / few["val"].norm()) < 1.7 * torch.finfo(DT[kind]).eps / 2


@pytest.mark.parametrize("kind,D", [("bf16", 32), ("f16", 64), ("f32", 32), ("bf16", 20)])
@pytest.mark.parametrize("kept", [3, 100, 199])
def test_one_key_kept_of_many(kind, D, kept):
    g = torch.Generator().manual_seed(D)
    B, L, H = 2, 200, 2
    t = dict(q=_normal(g, kind, B, 70, H, 2, D), k=_normal(g, kind, B, L, H, 2, D), v=_normal(g, kind, B, L, H, 2 * D),
             lam=(torch.rand(H, generator=g) + 0.1).cuda(), key_mask=torch.zeros(B, L, dtype=torch.bool).cuda())
    t["key_mask"][0, kept] = True  # the other item sees nothing
    got, val, tol = _both(t, dict(causal=False), _normal(g, kind, B, 70, H, 2 * D))
    check(got, val, tol)
    assert not got["grad_q"].any()


def test_fp16_many_small_weights():
    # One key of weight 1 and 16,384 of 2^-25 each, together 2^-11: half of
    # fp16's smallest number each, as much as eight steps of the result together.
    B, Lq, Lk, H, D = 1, 3, 16385, 2, 64
    q, k, v = torch.zeros(B, Lq, H, 2, D), torch.zeros(B, Lk, H, 2, D), torch.full((B, Lk, H, 2 * D), 8.0)
    q[..., 0] = 1.0
    k[:, 0, :, :, 0] = 25.0
    v[:, 0] = 0.0
    t = dict(q=q.half().cuda(), k=k.half().cuda(), v=v.half().cuda(), lam=torch.tensor([0.5, 0.25]).cuda())
    opt = dict(scale=0.6931471805599453)  # scores in powers of two
    out = da.dattn_forward(**t, **opt)
    val, tol = dattn_reference(**t, **opt)
    assert float(val["out"].abs().min()) > 1e-3
    assert float((out.double() - val["out"]).abs().max() / val["out"].abs().max()) < 2.0 ** -10


@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-4])
def test_fp16_small_gradients(size):
    # s_m and the weights are about size / keys: their roundings as operands
    # may be no more than half a step each, in 2-norm, beside the result's.
    # q, k and the scale are chosen so that the results themselves are not small.
    g = torch.Generator().manual_seed(7)
    B, L, H, D = 1, 2048, 2, 64
    t = dict(q=_normal(g, "f16", B, L, H, 2, D, std=2.0 ** -5), k=_normal(g, "f16", B, L, H, 2, D, std=2.0 ** -5),
             v=_normal(g, "f16", B, L, H, 2 * D), lam=torch.tensor([0.5, 0.8]).cuda())
    got, val, _ = _both(t, dict(scale=2.0 ** 10 / 8), _normal(g, "f16", B, L, H, 2 * D, std=size))
    for n in ("grad_q", "grad_k", "grad_v"):
        step = 2.0 ** -11
        once = float((val[n].half().double() - val[n]).norm() / val[n].norm())
        assert _off(got, val, n) < 1.7 * step + 1.5 * once, n


@pytest.mark.parametrize("Lk,std_v", [(5, 8.0), (130, 64.0)])
@pytest.mark.parametrize("D", [32, 64])
def test_fp16_large_gradients(D, Lk, std_v):
    # e = g v reaches 10^6 and s_m 10^5, past fp16; grad_q, grad_k and grad_v do not.
    g = torch.Generator().manual_seed(D)
    B, Lq, H = 1, 9, 2
    t = dict(q=_normal(g, "f16", B, Lq, H, 2, D, std=3.0), k=_normal(g, "f16", B, Lk, H, 2, D, std=3.0),
             v=_normal(g, "f16", B, Lk, H, 2 * D, std=std_v), lam=torch.tensor([0.5, 0.8]).cuda())
    got, val, tol = _both(t, dict(scale=2.0 ** -7), _normal(g, "f16", B, Lq, H, 2 * D, std=4096.0))
    assert all(float(val[n].abs().max()) < 65504 for n in ("grad_q", "grad_k", "grad_v"))
    check(got, val, tol)
    for n in ("grad_q", "grad_k", "grad_v"):
        assert _off(got, val, n) < 1.7 * 2.0 ** -11, n


def test_fp16_gradients_of_all_sizes():
    # Rows whose gradients differ by 2^20, one head's lam far above 1, a key
    # that is not to be used with infinite values.
    g = torch.Generator().manual_seed(3)
    B, L, H, D = 2, 300, 4, 32
    grad = torch.randn(B, L, H, 2 * D, generator=g) * 2.0 ** torch.randint(-16, 5, (B, L, 1, 1), generator=g)
    t = dict(q=_normal(g, "f16", B, L, H, 2, D), k=_normal(g, "f16", B, L, 2, 2, D), v=_normal(g, "f16", B, L, 2, 2 * D),
             lam=torch.tensor([0.5, 30.0, -0.8, 0.0]).cuda(), key_mask=(torch.rand(B, L, generator=g) < 0.8).cuda(),
             bias_table=torch.randn(8, H, generator=g).cuda(), bucket_map=da.relative_buckets(8, 16).cuda())
    t["v"][~t["key_mask"]] = float("inf")
    got, val, tol = _both(t, dict(causal=True), grad.half().cuda())
    check(got, val, tol)
    each = (got["grad_q"].double() - val["grad_q"]).flatten(2).norm(dim=2)
    once = (val["grad_q"].half().double() - val["grad_q"]).flatten(2).norm(dim=2)
    assert bool((each <= 4 * 2.0 ** -11 * val["grad_q"].flatten(2).norm(dim=2) + 2 * once).all())
