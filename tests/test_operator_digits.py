"""Digits of the group norm and the differential attention on inputs that a
kernel may lose them on, against 64 bits."""
import pytest
import torch

import deformable_view_feature_gb300 as da
from operator_refs import check, gn_reference

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
