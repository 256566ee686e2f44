"""The 64-bit references of the group norm and the differential attention:
their gradients against automatic differentiation and against differences."""
import pytest
import torch

from operator_refs import dattn_reference, gn_reference


def _difference(f, x, direction, h=1e-6):
    return float(f(x + h * direction) - f(x - h * direction)) / (2 * h)


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
def test_gn_reference_gradients(act):
    g = torch.Generator().manual_seed(3)
    maps = [(0, 6, 0), (7, 3, 1)]  # row 6 belongs to no map
    x, gamma, beta, grad = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((2, 10, 6), (2, 6), (2, 6), (2, 10, 6)))
    grad[:, 6] = 0

    def value(x=x, gamma=gamma, beta=beta):
        return (gn_reference(x, maps, gamma, beta, 2, 1e-5, act)[0]["out"] * grad).sum()

    val, _ = gn_reference(x, maps, gamma, beta, 2, 1e-5, act, grad)
    for name, arg in (("grad_feat", "x"), ("grad_gamma", "gamma"), ("grad_beta", "beta")):
        base = {"x": x, "gamma": gamma, "beta": beta}[arg]
        d = torch.randn(base.shape, generator=g, dtype=torch.float64)
        got = float((val[name] * d).sum())
        assert abs(got - _difference(lambda t: value(**{arg: t}), base, d)) < 1e-6 * max(1, abs(got))


@pytest.mark.parametrize("causal", [False, True])
def test_dattn_reference_gradients(causal):
    g = torch.Generator().manual_seed(4)
    B, Lq, Lk, H, Hk, D, Dv = 2, 4, 7, 4, 2, 3, 5
    t = {n: torch.randn(*s, generator=g, dtype=torch.float64) for n, s in
         (("q", (B, Lq, H, 2, D)), ("k", (B, Lk, Hk, 2, D)), ("v", (B, Lk, Hk, Dv)), ("lam", (H,)), ("table", (4, H)))}
    grad = torch.randn(B, Lq, H, Dv, generator=g, dtype=torch.float64)
    opt = dict(bucket_map=torch.tensor([3, 0, 1, 2, 2], dtype=torch.int32), causal=causal,
               key_mask=torch.rand(B, Lk, generator=g) < 0.7, key_lengths=torch.tensor([7, 3], dtype=torch.int32))

    def value(**kw):
        return (dattn_reference(**{**t, **kw}, **opt)[0]["out"] * grad).sum()

    val, _ = dattn_reference(**t, **opt, grad=grad)
    for name, base in t.items():
        d = torch.randn(base.shape, generator=g, dtype=torch.float64)
        got = float((val["grad_" + name] * d).sum())
        assert abs(got - _difference(lambda x: value(**{name: x}), base, d)) < 1e-6 * max(1, abs(got)), name


def test_dattn_reference_against_torch_autograd():
    g = torch.Generator().manual_seed(5)
    B, Lq, Lk, H, D, Dv = 1, 5, 6, 2, 4, 8
    q, k, v = (torch.randn(*s, generator=g, dtype=torch.float64, requires_grad=True)
               for s in ((B, Lq, H, 2, D), (B, Lk, H, 2, D), (B, Lk, H, Dv)))
    lam = torch.tensor([0.3, 0.8], dtype=torch.float64, requires_grad=True)
    grad = torch.randn(B, Lq, H, Dv, generator=g, dtype=torch.float64)
    p = torch.softmax(torch.einsum("bihmd,bjhmd->bhmij", q, k) / D ** 0.5, -1)
    out = torch.einsum("bhij,bjhe->bihe", p[:, :, 0] - lam[:, None, None] * p[:, :, 1], v)
    grads = torch.autograd.grad(out, (q, k, v, lam), grad)
    val, _ = dattn_reference(q.detach(), k.detach(), v.detach(), lam.detach(), grad=grad)
    assert torch.allclose(val["out"], out, rtol=1e-12)
    for name, want in zip(("grad_q", "grad_k", "grad_v", "grad_lam"), grads):
        assert torch.allclose(val[name], want, rtol=1e-9, atol=1e-12), name
