"""smoke()'s checks of the group norm and the differential attention on the
CPU: plain operators pass them; zeros, inputs handed back, or a gradient
without its sums do not."""
import types

import pytest
import torch

import __graft_entry__
from operator_refs import dattn_reference, gn_reference


def _operators():
    def gn(x, gamma, beta, grad=None):
        val, _ = gn_reference(x, [(0, x.shape[1], 0)], gamma[None], beta[None], 32, 1e-5, "silu", grad)
        return {n: t[0] if n in ("grad_gamma", "grad_beta") else t for n, t in val.items()}

    def gn_backward(x, ss, ls, gamma, beta, stats, grad, groups, act):
        val = gn(x, gamma, beta, grad)
        return val["grad_feat"], val["grad_gamma"], val["grad_beta"]

    def dattn_backward(q, k, v, lam, out, saved, grad):
        val, _ = dattn_reference(q, k, v, lam, grad=grad)
        return [val["grad_" + n].to(t.dtype) for n, t in (("q", q), ("k", k), ("v", v), ("lam", lam))] + [None]

    return types.SimpleNamespace(
        gn_forward=lambda x, ss, ls, gamma, beta, groups, act: (gn(x, gamma, beta)["out"], None), gn_backward=gn_backward,
        dattn_forward=lambda q, k, v, lam, keep_for_backward: (dattn_reference(q, k, v, lam)[0]["out"].to(q.dtype), None),
        dattn_backward=dattn_backward)


def _run(**change):
    da = _operators()
    for name, f in change.items():
        setattr(da, name, f(getattr(da, name)))
    __graft_entry__._norm_and_attention(da, torch.randn(1, 64, 256, generator=torch.Generator().manual_seed(1)),
                                        torch.tensor([[[8, 8]]], dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32))


def test_plain_operators_pass():
    _run()


def _zero(at):
    def change(f):
        def g(*args, **kw):
            r = list(f(*args, **kw))
            r[at] = torch.zeros_like(r[at])
            return r
        return g
    return change


@pytest.mark.parametrize("name,results", [("gn_forward", 1), ("gn_backward", 3), ("dattn_forward", 1), ("dattn_backward", 4)])
def test_zeros_do_not_pass(name, results):
    for at in range(results):
        with pytest.raises(AssertionError, match="off by"):
            _run(**{name: _zero(at)})


def test_what_is_not_normalised_does_not_pass():
    with pytest.raises(AssertionError, match="norm is off"):
        _run(gn_forward=lambda f: lambda x, ss, ls, gamma, beta, groups, act: (x - x.mean(), None))
