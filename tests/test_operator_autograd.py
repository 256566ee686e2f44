"""The autograd functions of the group norm and the differential attention on
the CPU, with plain torch in the place of the kernels' calls: a second
derivative, which neither has, is refused and not left out."""
import pytest
import torch

import deformable_view_feature_gb300 as da
from deformable_view_feature_gb300 import attention, norm


@pytest.fixture
def calls(monkeypatch):
    """Calls that give y = x * gamma, and out = the sum of q, k and v, with their gradients."""
    def gn_forward(feat, ss, ls, gamma, beta, groups, eps, act):
        return feat * gamma, torch.zeros(1)

    def gn_backward(feat, ss, ls, gamma, beta, stats, grad, groups, act):
        return grad * gamma, (grad * feat).sum((0, 1)), grad.sum((0, 1))

    def dattn_forward(q, k, v, lam, keep_for_backward=False, **opt):
        return q[..., 0, :] + k[..., 0, :] + v, (torch.zeros(1), torch.zeros(1))

    def dattn_backward(q, k, v, lam, out, saved, grad, **opt):
        both = torch.stack([grad, torch.zeros_like(grad)], 3)
        return both, both, grad, torch.zeros_like(lam), None

    monkeypatch.setattr(norm, "gn_forward", gn_forward)
    monkeypatch.setattr(norm, "gn_backward", gn_backward)
    monkeypatch.setattr(attention, "dattn_forward", dattn_forward)
    monkeypatch.setattr(attention, "dattn_backward", dattn_backward)


@pytest.mark.parametrize("enabled,requires,keeps", [(True, True, True), (True, False, False), (False, True, False)])
def test_attention_keeps_nothing_without_a_backward_pass(calls, monkeypatch, enabled, requires, keeps):
    asked, forward = [], attention.dattn_forward

    def recorded(*args, keep_for_backward=False, **opt):
        asked.append(keep_for_backward)
        out, saved = forward(*args, **opt)
        return (out, saved) if keep_for_backward else out

    monkeypatch.setattr(attention, "dattn_forward", recorded)
    x = torch.randn(1, 4, 2, 2, 3, requires_grad=requires)
    with torch.set_grad_enabled(enabled):
        y = _attention(x)
    assert asked == [keeps] and y.requires_grad == keeps
    assert torch.equal(y.detach(), (2 * x[..., 0, :] + x[..., 0, :]).detach())


def _norm(x):
    ss, ls = torch.tensor([[[2, 2]]], dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    return da.GroupNormActFunction.apply(x, ss, ls, torch.full((3,), 2.0), torch.zeros(3), 1, 1e-5, "none")


def _attention(x):
    return da.DifferentialAttentionFunction.apply(x, x, x[..., 0, :], torch.ones(2))


@pytest.mark.parametrize("function,shape", [(_norm, (1, 4, 3)), (_attention, (1, 4, 2, 2, 3))])
def test_a_second_derivative_is_refused(calls, function, shape):
    x = torch.randn(shape, requires_grad=True)
    first, = torch.autograd.grad(function(x).square().sum(), x)
    assert first.shape == x.shape and not first.requires_grad
    first, = torch.autograd.grad(function(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (first.square().sum() + x.sum()).backward()
