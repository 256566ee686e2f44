"""Two host threads that call one kernel at once, each on a stream of its own,
with calls that need different amounts of shared memory (a bias table or none,
two widths of values, few or many points): both succeed and give what each gives alone. The calls
let other threads run Python meanwhile."""
import threading

import pytest
import torch

import deformable_view_feature_gb300 as da
from test_dattn import _case
from test_paged import _attention_case


@pytest.fixture(scope="module", autouse=True)
def built():
    da.build.build()


def _paged(**kw):
    t, opt = _attention_case(**kw)
    return lambda: da.paged_attention(**t, **opt)


def _forward(**kw):
    t, opt, _ = _case(**kw)
    return lambda: da.dattn_forward(**t, **opt)


def _backward(**kw):
    t, opt, grad = _case(**kw)
    out, saved = da.dattn_forward(**t, **opt, keep_for_backward=True)
    args = {n: x for n, x in t.items() if n not in ("q", "k", "v", "lam")}
    return lambda: torch.cat([g.flatten().float() for g in da.dattn_backward(t["q"], t["k"], t["v"], t["lam"], out, saved, grad, **args, **opt)
                              if g is not None])


def _maps(g):
    feat, ss, ls = torch.randn(1, 64, 32, generator=g).cuda(), torch.tensor([[[8, 8]]], dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    return feat, ss, ls


def _scatter(P):
    g = torch.Generator().manual_seed(P)
    maps = _maps(g)
    loc, w, grad = torch.rand(1, 4, P, 1, 2, generator=g).cuda(), torch.rand(1, 4, P, 1, 1, 1, generator=g).cuda(), torch.randn(1, 4, 32, generator=g).cuda()
    # grad_feat is summed by atomics, in any order
    return lambda: torch.cat([x.flatten() for x in da.da_backward(*maps, loc, w, grad, path="scatter")[1:]])


def _projected(P):
    g = torch.Generator().manual_seed(P)
    maps = _maps(g)
    points, logits = torch.rand(1, 4, P, 3, generator=g).cuda(), torch.randn(1, 4, P, 1, 1, 1, generator=g).cuda()
    camera = torch.eye(4)[None, None].clone().cuda()
    return lambda: da.da_forward_projected(*maps, points, camera, 8.0, 8.0, logits)[0]


# A call, what its two forms share, and what the larger one has besides.
PAIRS = {
    "paged, tensor cores": (_paged, dict(B=2, N=9, T=3, H=4, Hk=2, kind="bf16", lengths=[144, 77]), dict(buckets=32, reach=400)),
    "paged, few rows": (_paged, dict(B=2, N=9, T=2, D=24, Dv=8, lengths=[144, 77]), dict(Dv=128)),
    "paged, few odd rows": (_paged, dict(B=2, N=9, T=2, D=17, Dv=9, kind="bf16", lengths=[144, 77]), dict(Dv=255)),
    "paged, tiles": (_paged, dict(B=2, N=9, T=30, lengths=[144, 77]), dict(buckets=32, reach=1000)),
    "forward, tensor cores": (_forward, dict(B=2, Lq=40, Lk=50, kind="bf16"), dict(buckets=32, reach=1000)),
    "forward, tiles": (_forward, dict(B=2, Lq=40, Lk=50), dict(buckets=32, reach=1000)),
    "backward, tensor cores": (_backward, dict(B=2, Lq=40, Lk=50, kind="f16"), dict(buckets=32, reach=1000)),
    "backward, tiles": (_backward, dict(B=2, Lq=40, Lk=50), dict(buckets=32, reach=1000)),
    "aggregation, scatter": (_scatter, dict(P=900), dict(P=3000)),
    "aggregation, projected": (_projected, dict(P=600), dict(P=1600)),
}


def _at_once(calls, times):
    """Errors of the threads that make these calls again and again, at once."""
    wants = [c() for c in calls]
    torch.cuda.synchronize()
    begin, wrong = threading.Barrier(len(calls)), []

    def work(call, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                begin.wait()
                for _ in range(times):
                    got = call()
                torch.cuda.current_stream().synchronize()
                assert torch.equal(got, want)
        except Exception as e:  # noqa: BLE001 - any of them is the test's finding
            wrong.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(calls, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return wrong


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(PAIRS))
def test_calls_of_different_sizes(name):
    make, common, more = PAIRS[name]
    assert _at_once([make(**common), make(**{**common, **more})], 2000) == []


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["paged_attention", "dattn_forward", "dattn_backward"])
def test_a_threads_first_call(call):
    """Of a thread that has made no CUDA call before: each of these uses the tensor cores, whose operands the driver describes."""
    make = {"paged_attention": _paged, "dattn_forward": _forward, "dattn_backward": _backward}[call]
    run = make(**(dict(B=2, N=9, T=3, H=4, Hk=2, kind="bf16", lengths=[144, 77]) if call == "paged_attention" else dict(B=2, Lq=40, Lk=50, kind="bf16")))
    want, wrong, got = run(), [], []
    torch.cuda.synchronize()

    def work():
        try:
            got.append(run())
        except Exception as e:  # noqa: BLE001 - any of them is the test's finding
            wrong.append(e)

    for _ in range(20):
        t = threading.Thread(target=work)
        t.start()
        t.join()
    assert wrong == [] and all(torch.equal(x, want) for x in got)


@pytest.mark.gpu
def test_a_serving_loop_beside_another():
    """Appends and attention of two caches, each on a thread and a stream of its own."""
    def loop(kind, seed):
        t, opt = _attention_case(B=2, N=9, T=1, H=4, Hk=2, kind=kind, seed=seed)
        t["key_lengths"] = torch.tensor([0, 30], dtype=torch.int32, device="cuda")
        g = torch.Generator().manual_seed(seed)
        new = [torch.randn(20, 2, 1, *s, generator=g).to(t["q"].dtype).cuda() for s in ((2, 2, 32), (2, 64))]
        turns = da.rotary_frequencies(32).cuda()

        def run():
            k, v, n = t["k_cache"].clone(), t["v_cache"].clone(), t["key_lengths"].clone()
            outs = []
            for x, y in zip(*new):
                q = da.paged_append(x, y, k, v, t["page_table"], n, q=t["q"], frequencies=turns)
                n += 1
                outs.append(da.paged_attention(q, k, v, t["lam"], t["page_table"], n, **opt))
            return torch.stack(outs)
        return run

    assert _at_once([loop("bf16", 1), loop("bf16", 2), loop("f32", 3), loop("f32", 4)], 20) == []
