"""Group norm with an activation (gn_forward, gn_backward, GroupNormActFunction):
refusals on the CPU, results on the GPU against 64 bits."""
import ctypes

import pytest
import torch

import deformable_view_feature_gb300 as da
from deformable_view_feature_gb300 import norm
from operator_refs import check, gn_reference

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FAKE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    da.build.build()
    return da.load_library()


def _tables(shapes, cams, gap=0):
    """Host tables of `cams` cameras; `gap` rows of no map after each map."""
    start, at, maps = [], 0, []
    for _ in range(cams):
        for s, (h, w) in enumerate(shapes):
            start.append(at)
            maps.append((at, h * w, s))
            at += h * w + gap
    return (torch.tensor([shapes] * cams, dtype=torch.int32), torch.tensor(start, dtype=torch.int32).reshape(cams, len(shapes)),
            maps, at)


# ---- refusals: no GPU, nothing is launched ---------------------------------

def _status(lib, ss=((4, 4),), ls=(0,), backward=0, **kw):
    d = dict(batch=1, num_cams=1, num_scales=len(ls), num_embeds=16, num_groups=4, feat_dtype=0, act=0, affine_scales=0,
             num_feat_rows=16, eps=1e-5)
    d.update(kw)
    shape = (ctypes.c_int32 * (2 * len(ls)))(*[n for s in ss for n in s])
    start = (ctypes.c_int32 * len(ls))(*ls)
    n = ctypes.c_size_t(0)
    dims = norm.GnDims(*[d[f[0]] for f in norm.GnDims._fields_])
    return lib.gn_workspace_size(ctypes.byref(dims), shape, start, backward, ctypes.byref(n)), dims, shape, start, n.value


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(batch=-1), 2), (dict(num_groups=3), 2), (dict(num_embeds=0), 2), (dict(feat_dtype=7), 2),
    (dict(act=3), 2), (dict(eps=0.0), 2), (dict(eps=float("nan")), 2), (dict(num_feat_rows=15), 2),
    (dict(num_embeds=8192), 4), (dict(num_cams=65), 4), (dict(ss=((0, 4),)), 2), (dict(ls=(-1,)), 2),
    (dict(ss=((2, 2), (2, 2)), ls=(0, 3)), 2),   # overlapping maps
    (dict(ss=((2, 2), (2, 2)), ls=(4, 0)), 0),   # any order
    (dict(ss=((2, 2), (2, 2)), ls=(0, 13)), 2),  # past the rows
])
def test_sizes_are_checked(lib, kw, status):
    assert _status(lib, **kw)[0] == status


def test_buffers_are_checked(lib):
    _, d, shape, start, need = _status(lib)
    vp = ctypes.c_void_p

    def call(feat=FAKE, gamma=FAKE, out=FAKE, stats=FAKE, ws=FAKE, size=need):
        return lib.gn_forward(ctypes.byref(d), vp(feat), shape, start, vp(gamma), vp(FAKE), vp(out), vp(stats), vp(ws), size, None)

    assert need > 0
    assert call(feat=None) == 1 and call(gamma=None) == 1 and call(out=None) == 1 and call(stats=None) == 1
    assert call(feat=FAKE + 2) == 3 and call(stats=FAKE + 2) == 3
    assert call(ws=None) == 6 and call(size=need - 1) == 6 and call(ws=FAKE + 16) == 6
    assert lib.gn_forward(None, *[None] * 8, 0, None) == 1
    _, d, shape, start, need = _status(lib, backward=1)
    args = [vp(FAKE)] * 2 + [vp(FAKE)] * 3
    assert lib.gn_backward(ctypes.byref(d), vp(FAKE), shape, start, *args[:3], vp(FAKE), vp(FAKE), None, vp(FAKE), vp(FAKE), need, None) == 1
    assert lib.gn_backward(ctypes.byref(d), vp(FAKE), shape, start, *args[:3], vp(FAKE), vp(FAKE), vp(FAKE + 2), vp(FAKE), vp(FAKE), need, None) == 3


def test_stats_are_aligned_to_their_pairs(lib):
    # The kernels access a group's mean and 1/sqrt(var + eps) together.
    vp = ctypes.c_void_p
    _, d, shape, start, need = _status(lib)
    for off in (2, 4, 12):
        assert lib.gn_forward(ctypes.byref(d), vp(FAKE), shape, start, vp(FAKE), vp(FAKE), vp(FAKE), vp(FAKE + off), vp(FAKE),
                              need, None) == 3
    _, d, shape, start, need = _status(lib, backward=1)
    for off in (2, 4, 12):
        assert lib.gn_backward(ctypes.byref(d), vp(FAKE), shape, start, vp(FAKE), vp(FAKE), vp(FAKE + off), vp(FAKE), vp(FAKE),
                               vp(FAKE), vp(FAKE), vp(FAKE), need, None) == 3


def test_binding_checks_shapes_and_types():
    x, g = torch.zeros(1, 16, 8), torch.ones(8)
    ss, ls, _, _ = _tables([(4, 4)], 1)
    ok = (x, ss, ls, g, g, 2, 1e-5, "relu")
    assert norm._gn_dims(*ok).act == 1
    for at, bad, error in ((0, x[0], ValueError), (0, x.double(), TypeError), (1, ss[0], ValueError), (2, ls[0], ValueError),
                           (3, g[:4], ValueError), (3, g.half(), TypeError), (7, "gelu", ValueError)):
        with pytest.raises(error):
            norm._gn_dims(*ok[:at], bad, *ok[at + 1:])
    with pytest.raises(ValueError):
        da.gn_backward(x, ss, ls, g, g, torch.zeros(1, 1, 1, 2, 2), x.half(), 2)
    with pytest.raises(ValueError, match="stats"):
        da.gn_backward(x, ss, ls, g, g, torch.zeros(1, 1, 1, 3, 2), x, 2)


# ---- results ---------------------------------------------------------------

CASES = {
    # shapes, cams, batch, C, groups, type, act, per scale, gap
    "one pixel": ([(1, 1)], 1, 1, 8, 2, "f32", "none", False, 0),
    "one group": ([(3, 5)], 1, 2, 12, 1, "f32", "silu", False, 0),
    "group per channel": ([(9, 7)], 2, 1, 16, 16, "bf16", "silu", False, 0),
    "tile edge": ([(8, 8), (5, 13), (1, 63)], 1, 1, 32, 8, "f32", "relu", True, 0),
    "gaps": ([(7, 9), (2, 3)], 2, 3, 24, 3, "f32", "silu", False, 5),
    "scalar columns": ([(11, 6)], 1, 2, 15, 5, "f16", "silu", False, 0),
    "odd width": ([(57, 31), (1, 1)], 1, 1, 96, 12, "f16", "none", True, 1),
    "many channels": ([(6, 5)], 1, 1, 2080, 32, "f32", "silu", False, 0),
    "most channels": ([(3, 3)], 1, 1, 4096, 32, "bf16", "none", False, 0),
    "most scalar channels": ([(3, 3)], 1, 1, 4095, 9, "bf16", "silu", False, 0),
    "pyramid": ([(64, 176), (32, 88), (16, 44), (8, 22)], 2, 2, 256, 32, "bf16", "silu", True, 0),
    "pyramid f32": ([(64, 176), (32, 88), (16, 44), (8, 22)], 1, 2, 256, 32, "f32", "none", False, 0),
}


def _inputs(name, mean=1.0, dev="cuda"):
    shapes, cams, B, C, groups, kind, act, per_scale, gap = CASES[name]
    ss, ls, maps, rows = _tables(shapes, cams, gap)
    g = torch.Generator().manual_seed(len(name) * 7 + C)
    x = (torch.randn(B, rows, C, generator=g) * (torch.rand(C, generator=g) + 0.2) + mean * torch.randn(C, generator=g)).to(DT[kind])
    affine = (len(shapes), C) if per_scale else (C,)
    gamma, beta = torch.randn(*affine, generator=g) * 0.3 + 1, torch.randn(*affine, generator=g) * 0.3
    grad = torch.randn(B, rows, C, generator=g).to(DT[kind])
    return (x.to(dev), ss, ls, gamma.to(dev), beta.to(dev), groups, act), maps, grad.to(dev), len(shapes)


def _check_all(args, maps, grad, S, out, grads):
    x, ss, ls, gamma, beta, groups, act = args
    C = x.shape[2]
    val, tol = gn_reference(x, maps, gamma.expand(S, C), beta.expand(S, C), groups, 1e-5, act, grad)
    if gamma.dim() == 1:
        for d in (val, tol):
            d["grad_gamma"], d["grad_beta"] = d["grad_gamma"].sum(0), d["grad_beta"].sum(0)
    if act == "relu":
        # Next to z = 0 a rounding decides the slope: with an element there,
        # only the forward pass can be held to its tolerance.
        z, off = gn_reference(x, maps, gamma.expand(S, C), beta.expand(S, C), groups, 1e-5, "none")
        if bool((z["out"].abs() <= off["out"]).any()):
            check({"out": out}, {"out": val["out"]}, tol)
            return
    check({"out": out, "grad_feat": grads[0], "grad_gamma": grads[1], "grad_beta": grads[2]}, val, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_against_64_bits(name):
    args, maps, grad, S = _inputs(name)
    out, stats = da.gn_forward(*args[:6], act=args[6])
    grads = da.gn_backward(*args[:5], stats, grad, args[5], act=args[6])
    _check_all(args, maps, grad, S, out, grads)


@pytest.mark.gpu
def test_relu_gradient_away_from_its_border():
    # Values on a grid whose norm keeps clear of zero.
    x = (torch.arange(48, device="cuda").reshape(1, 12, 4) % 7 - 2.9).float()
    ss, ls, maps, _ = _tables([(3, 4)], 1)
    one, zero = torch.ones(4, device="cuda"), torch.zeros(4, device="cuda")
    grad = torch.linspace(-1, 1, 48, device="cuda").reshape(1, 12, 4)
    out, stats = da.gn_forward(x, ss, ls, one, zero, 2, act="relu")
    grads = da.gn_backward(x, ss, ls, one, zero, stats, grad, 2, act="relu")
    _check_all((x, ss, ls, one, zero, 2, "relu"), maps, grad, 1, out, grads)


LARGE = {
    # shapes, C, groups, type, act: maps above 64 KB, which several tiles share
    "relu f32": ([(150, 200)], 64, 8, "f32", "relu"),
    "relu bf16": ([(90, 120), (45, 60)], 96, 12, "bf16", "relu"),
    "relu f16": ([(75, 99)], 40, 8, "f16", "relu"),
    "three groups": ([(150, 200)], 24, 3, "f32", "silu"),
    "one group": ([(64, 99)], 32, 1, "bf16", "none"),
    "scalar columns": ([(150, 101), (1, 1)], 15, 5, "f16", "silu"),
    "two scalar groups": ([(201, 200)], 6, 2, "bf16", "silu"),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(LARGE))
def test_large_maps(name):
    shapes, C, groups, kind, act = LARGE[name]
    ss, ls, maps, rows = _tables(shapes, 2)
    g = torch.Generator().manual_seed(C)
    x = (torch.randn(2, rows, C, generator=g) + torch.randn(C, generator=g)).to(DT[kind]).cuda()
    gamma, beta = torch.randn(C, generator=g).cuda() * 0.3 + 1, torch.randn(C, generator=g).cuda() * 0.3
    grad = torch.randn(2, rows, C, generator=g).to(DT[kind]).cuda()
    S = len(shapes)
    if act == "relu":  # next to z = 0 a rounding decides the slope: no gradient comes in there
        z, off = gn_reference(x, maps, gamma.expand(S, C), beta.expand(S, C), groups, 1e-5, "none")
        near = z["out"].abs() <= off["out"]
        assert bool(near.any())
        grad = grad.masked_fill(near, 0)
    out, stats = da.gn_forward(x, ss, ls, gamma, beta, groups, act=act)
    grads = da.gn_backward(x, ss, ls, gamma, beta, stats, grad, groups, act=act)
    val, tol = gn_reference(x, maps, gamma.expand(S, C), beta.expand(S, C), groups, 1e-5, act, grad)
    for d in (val, tol):
        d["grad_gamma"], d["grad_beta"] = d["grad_gamma"].sum(0), d["grad_beta"].sum(0)
    check({"out": out, "grad_feat": grads[0], "grad_gamma": grads[1], "grad_beta": grads[2]}, val, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["one group", "gaps", "scalar columns", "odd width", "most scalar channels"])
def test_in_place_on_small_maps(name):
    args, maps, grad, S = _inputs(name)
    out, stats = da.gn_forward(*args[:6], act=args[6])
    grads = da.gn_backward(*args[:5], stats, grad, args[5], act=args[6])
    x, g = args[0].clone(), grad.clone()
    da.gn_forward(x, *args[1:6], act=args[6], out=x)
    da.gn_backward(*args[:5], stats, g, args[5], act=args[6], grad_feat=g)
    assert torch.equal(x, out) and torch.equal(g, grads[0])


@pytest.mark.gpu
def test_mean_far_above_the_spread():
    args, maps, grad, S = _inputs("pyramid f32", mean=0.0)
    x = args[0] + 1000.0
    out, _ = da.gn_forward(x, *args[1:6], act="none")
    val, tol = gn_reference(x, maps, args[3].expand(S, -1), args[4].expand(S, -1), args[5], 1e-5, "none")
    check({"out": out}, val, tol)


@pytest.mark.gpu
def test_constant_map_and_infinite_values():
    ss, ls, maps, _ = _tables([(5, 5), (4, 4)], 1)
    x = torch.full((1, 41, 8), 3.0, device="cuda")
    gamma, beta = torch.full((8,), 2.0, device="cuda"), torch.full((8,), 0.5, device="cuda")
    out, stats = da.gn_forward(x, ss, ls, gamma, beta, 2)
    assert torch.equal(out, torch.full_like(out, 0.5))  # no spread: norm 0
    # An infinity stays within its map and group.
    x = torch.randn(1, 41, 8, device="cuda")
    x[0, 30, 1] = float("inf")
    y, _ = da.gn_forward(x, ss, ls, gamma, beta, 2)
    assert bool(torch.isnan(y[0, 25:, :4]).any()) and bool(torch.isfinite(y[0, :25]).all())
    assert bool(torch.isfinite(y[0, 25:, 4:]).all())


@pytest.mark.gpu
def test_in_place_same_bits_and_streams():
    args, maps, grad, S = _inputs("pyramid")
    out, stats = da.gn_forward(*args[:6], act=args[6])
    again, stats2 = da.gn_forward(*args[:6], act=args[6])
    assert torch.equal(out, again) and torch.equal(stats, stats2)
    x = args[0].clone()
    y, _ = da.gn_forward(x, *args[1:6], act=args[6], out=x)
    assert y.data_ptr() == x.data_ptr() and torch.equal(x, out)
    grads = da.gn_backward(*args[:5], stats, grad, args[5], act=args[6])
    g = grad.clone()
    da.gn_backward(*args[:5], stats, g, args[5], act=args[6], grad_feat=g)
    assert torch.equal(g, grads[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other, st3 = da.gn_forward(*args[:6], act=args[6], stream=side)
    g3 = da.gn_backward(*args[:5], st3, grad, args[5], act=args[6], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, out) and all(torch.equal(a, b) for a, b in zip(g3, grads))


@pytest.mark.gpu
def test_autograd_and_graph_capture():
    (x, ss, ls, gamma, beta, groups, act), maps, grad, S = _inputs("gaps")
    leaves = [t.clone().requires_grad_(True) for t in (x, gamma, beta)]
    out = da.GroupNormActFunction.apply(leaves[0], ss, ls, leaves[1], leaves[2], groups, 1e-5, act)
    # a gradient that is broadcast, and one that is a transposed view
    grads = torch.autograd.grad(out, leaves, grad.transpose(0, 1).contiguous().transpose(0, 1))
    _check_all((x, ss, ls, gamma, beta, groups, act), maps, grad, S, out.detach(), grads)
    flat = torch.autograd.grad(da.GroupNormActFunction.apply(leaves[0], ss, ls, *leaves[1:], groups, 1e-5, act).sum(), leaves)
    _check_all((x, ss, ls, gamma, beta, groups, act), maps, torch.ones_like(x), S, out.detach(), flat)
    # Calls of the functions capture into a graph and replay on new inputs.
    static, sgrad = torch.zeros_like(x), torch.zeros_like(grad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        da.gn_forward(static, ss, ls, gamma, beta, groups, act=act)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, st = da.gn_forward(static, ss, ls, gamma, beta, groups, act=act)
        g = da.gn_backward(static, ss, ls, gamma, beta, st, sgrad, groups, act=act)
    for shift in (0.0, 1.0):
        static.copy_(x + shift)
        sgrad.copy_(grad)
        graph.replay()
        eager, est = da.gn_forward(x + shift, ss, ls, gamma, beta, groups, act=act)
        eg = da.gn_backward(x + shift, ss, ls, gamma, beta, est, grad, groups, act=act)
        assert torch.equal(y, eager) and all(torch.equal(a, b) for a, b in zip(g, eg))


def test_wait_tries_are_returned(lib):
    usual = lib.da_gn_wait_tries(-1)
    assert usual > 1000 and lib.da_gn_wait_tries(7) == usual and lib.da_gn_wait_tries(usual) == 7


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["pyramid", "pyramid f32"])
def test_waits_that_give_up_leave_nan(lib, name):
    # Waits of no tries: every tile's outputs, the statistics and the
    # parameters' gradients are NaN, not what the memory held.
    args, maps, grad, S = _inputs(name)
    assert not da.waits_gave_up()
    out, stats = da.gn_forward(*args[:6], act=args[6])
    grads = da.gn_backward(*args[:5], stats, grad, args[5], act=args[6])
    usual = lib.da_gn_wait_tries(0)
    try:
        bad, bad_stats = da.gn_forward(*args[:6], act=args[6])
        bad_grads = da.gn_backward(*args[:5], stats, grad, args[5], act=args[6])
        assert da.waits_gave_up() and not da.waits_gave_up()
    finally:
        lib.da_gn_wait_tries(usual)
    assert all(bool(torch.isnan(t).all()) for t in (bad, bad_stats, *bad_grads))
    again, stats2 = da.gn_forward(*args[:6], act=args[6])
    assert torch.equal(again, out) and torch.equal(stats2, stats)
    assert all(torch.equal(a, b) for a, b in zip(da.gn_backward(*args[:5], stats, grad, args[5], act=args[6]), grads))
    assert not da.waits_gave_up()


@pytest.mark.gpu
def test_empty_sizes():
    ss, ls, _, _ = _tables([(2, 2)], 1)
    gamma = torch.ones(4, device="cuda")
    x = torch.zeros(0, 4, 4, device="cuda")
    out, stats = da.gn_forward(x, ss, ls, gamma, gamma, 2)
    gx, gg, gb = da.gn_backward(x, ss, ls, gamma, gamma, stats, x, 2)
    assert out.shape == x.shape and not gg.any() and not gb.any()
    x = torch.ones(2, 5, 4, device="cuda")  # no map at all: every row is of none
    none = torch.zeros(0, 1, 2, dtype=torch.int32), torch.zeros(0, 1, dtype=torch.int32)
    out, stats = da.gn_forward(x, *none, gamma, gamma, 2)
    gx, gg, gb = da.gn_backward(x, *none, gamma, gamma, stats, x, 2)
    assert not out.any() and not gx.any() and not gg.any()


@pytest.mark.gpu
def test_tensors_off_the_gpu_are_refused():
    ss, ls, _, _ = _tables([(2, 2)], 1)
    x, g = torch.zeros(1, 4, 4, device="cuda"), torch.ones(4, device="cuda")
    with pytest.raises(ValueError, match="CUDA"):
        da.gn_forward(x.cpu(), ss, ls, g, g, 2)
    with pytest.raises(ValueError, match="contiguous"):
        da.gn_forward(x.transpose(1, 2), ss, ls, g, g, 2)
