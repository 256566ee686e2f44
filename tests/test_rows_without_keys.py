"""A query that sees no key gives exactly 0, whatever the keys and values hold
that other queries of its tile see, and whatever lam is: padding of a batch and
rows that a mask leaves empty. Every way out of the attention over a paged cache
and of the contiguous one: rows walked by one CTA or split over the keys, on the
fp32 units (few rows, tiles) and on the tensor cores."""
import pytest
import torch

import deformable_view_feature_gb300 as da
from test_paged import _attention_case

INF, NAN = float("inf"), float("nan")
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    da.build.build()


def _paged(**kw):
    """Sequence 1 has one new token and padding, the last token of sequence 2, whose cache holds its new tokens alone, sees nothing."""
    T, L = kw["T"], kw["N"] * kw.get("S", 16)
    t, opt = _attention_case(B=3, lengths=[L, L, T], counts=[T, 1, T], tree="random", **kw)
    t["tree"][2, T - 1] = False
    empty = torch.zeros(3, T, dtype=torch.bool, device="cuda")
    empty[1, 1:] = empty[2, T - 1] = True
    return t, opt, empty


# Which way out: the kernels by type, width and rows, a split by the table's length.
PAGED = {
    "few rows": dict(kind="f32", T=2, N=8),
    "few rows, split": dict(kind="f32", T=2, N=80),
    "few rows, many parts": dict(kind="f32", T=2, N=500),
    "few rows, shared heads": dict(kind="f32", T=2, N=80, H=8, Hk=2, D=64),
    "few odd rows, split": dict(kind="bf16", T=2, N=80, D=17),
    "tiles": dict(kind="f32", T=30, N=7),
    "tiles, split": dict(kind="f32", T=30, N=40),
    "tiles, many parts": dict(kind="f32", T=30, N=200, H=1, Hk=1),
    "wide tiles, split": dict(kind="f32", T=30, N=40, D=100),
    "odd tiles, split": dict(kind="f16", T=30, N=40, D=17),
    "tensor cores": dict(kind="bf16", T=3, N=8),
    "tensor cores, split": dict(kind="bf16", T=3, N=200, D=64),
    "tensor cores, many rows": dict(kind="f16", T=70, N=8, H=4, Hk=2),
    "tensor cores, many rows, split": dict(kind="bf16", T=70, N=100, H=4, Hk=2, D=64),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(PAGED))
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_paged_attention(name, bad):
    t, opt, empty = _paged(**PAGED[name])
    want = da.paged_attention(**t, **opt)
    assert not bool(want[empty].any())
    first = t["page_table"][:, 0].long()        # place 0: every query that sees a key sees it
    for where, value in (("v_cache", bad), ("k_cache", bad), ("lam", bad)):
        u = {**t, where: t[where].clone()}
        if where == "lam":
            u["lam"][:] = value
        else:
            u[where][first, 0] = value
        got = da.paged_attention(**u, **opt)
        assert not bool((got[empty] != 0).any()), where
        assert where == "k_cache" or not bool(torch.isfinite(got[~empty]).any()), "nothing reached the others"


def _contiguous(kind, D, Lq=30, Lk=100, H=4, Hk=2):
    """Item 1 has 5 keys, so that its first queries are before all of them."""
    g = torch.Generator().manual_seed(D + Lk)
    t = [torch.randn(2, *s, generator=g).to(DT[kind]).cuda() for s in ((Lq, H, 2, D), (Lk, Hk, 2, D), (Lk, Hk, 2 * D))]
    opt = dict(key_lengths=torch.tensor([Lk, 5], dtype=torch.int32, device="cuda"), causal=True)
    empty = opt["key_lengths"][:, None] - Lq + torch.arange(Lq, device="cuda") < 0  # positions before key 0
    return *t, torch.rand(H, generator=g).cuda() + 0.1, opt, empty


CONTIGUOUS = {
    "tiles": dict(kind="f32", D=32), "tiles, split": dict(kind="f32", D=32, Lk=1000), "few rows, split": dict(kind="f32", D=64, Lq=7, Lk=1000),
    "odd tiles, split": dict(kind="bf16", D=17, Lk=1000), "tensor cores": dict(kind="bf16", D=32), "tensor cores, wide": dict(kind="f16", D=64, Lq=300),
    "tensor cores, split": dict(kind="bf16", D=64, Lk=1000), "tensor cores, fp16, split": dict(kind="f16", D=32, Lk=1000),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CONTIGUOUS))
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_contiguous_attention(name, bad):
    q, k, v, lam, opt, empty = _contiguous(**CONTIGUOUS[name])
    for where in ("v", "lam"):
        u = {"v": v.clone(), "lam": lam.clone()}
        if where == "v":
            u["v"][:, 0] = bad
        else:
            u["lam"][:] = bad
        out, (out1, lse) = da.dattn_forward(q, k, **u, **opt, keep_for_backward=True)
        assert torch.equal(torch.nan_to_num(out, 0, 1, -1) != 0, torch.nan_to_num(da.dattn_forward(q, k, **u, **opt), 0, 1, -1) != 0)
        assert not bool((out[empty] != 0).any()) and not bool((out1[empty] != 0).any()), where
        assert bool((lse[1, :, :, : int(empty[1].sum())] == INF).all())
        assert not bool(torch.isfinite(out[~empty]).any()), "nothing reached the others"


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CONTIGUOUS))
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_contiguous_gradients(name, bad):
    """Such a query's grad_q is 0."""
    q, k, v, lam, opt, empty = _contiguous(**CONTIGUOUS[name])
    grad = torch.randn(v.shape[0], q.shape[1], q.shape[2], v.shape[3], generator=torch.Generator().manual_seed(1)).to(q.dtype).cuda()
    for where in ("k", "v", "lam"):
        u = {"k": k.clone(), "v": v.clone(), "lam": lam.clone()}
        if where == "lam":
            u["lam"][:] = bad
        else:
            u[where][:, 0] = bad
        out, saved = da.dattn_forward(q, **u, **opt, keep_for_backward=True)
        got = da.dattn_backward(q, u["k"], u["v"], u["lam"], out, saved, grad, **opt)
        assert not bool((got[0][empty] != 0).any()), where


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CONTIGUOUS))
def test_gradients_of_keys_past_the_length(name):
    """They are 0 too where the other keys' are NaN."""
    q, k, v, lam, opt, _ = _contiguous(**CONTIGUOUS[name])
    grad = torch.randn(v.shape[0], q.shape[1], q.shape[2], v.shape[3], generator=torch.Generator().manual_seed(1)).to(q.dtype).cuda()
    k[:, 0] = NAN
    out, saved = da.dattn_forward(q, k, v, lam, **opt, keep_for_backward=True)
    _, gk, gv, _, _ = da.dattn_backward(q, k, v, lam, out, saved, grad, **opt)
    assert not bool((gk[1, 5:] != 0).any()) and not bool((gv[1, 5:] != 0).any())
    assert bool(torch.isnan(gk[1, :5]).all()) and bool(torch.isnan(gv[1, :5]).all())
