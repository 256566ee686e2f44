"""The rotary norm and the paged cache on the CPU: their headers are plain C,
the library exports what they declare, the binding's structures have the
headers' layout, and tensors of two devices are refused."""
import ctypes
import os
import re
import subprocess
import types
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import __graft_entry__
import deformable_view_feature_gb300 as da
from serving_refs import PgCache, PgProblem, QkrProblem, paged_reference, qkr_reference, serving_library

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


@pytest.fixture(scope="module", autouse=True)
def lib():
    da.build.build()
    return serving_library(da.load_library())


def test_library_exports_what_the_headers_declare(lib):
    for h, prefix, least in (("qkr.h", "qkr", {"qkr_forward", "qkr_backward", "qkr_workspace_size"}),
                             ("paged.h", "pg", {"pg_append", "pg_attention", "pg_workspace_size"})):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, h)).read(), flags=re.S)
        names = set(re.findall(r"\b(" + prefix + r"_[a-z0-9_]+)\s*\(", text))
        assert least <= names
        for n in names:
            getattr(lib, n)


def test_headers_are_plain_c_and_structures_agree(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "paged.h"\n'
                   'int main(void){ printf("%zu %zu %zu %zu %zu %zu %zu %zu\\n", sizeof(qkr_problem), offsetof(qkr_problem, q_stride),'
                   ' offsetof(qkr_problem, turns), sizeof(pg_cache), offsetof(pg_cache, page_table), sizeof(pg_problem),'
                   ' offsetof(pg_problem, cache), offsetof(pg_problem, tree)); return 0; }\n')
    exe = tmp_path / "use"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    Q, C, P = QkrProblem, PgCache, PgProblem
    assert got == [ctypes.sizeof(Q), Q.q_stride.offset, Q.turns.offset, ctypes.sizeof(C), C.page_table.offset, ctypes.sizeof(P),
                   P.cache.offset, P.tree.offset]


F = torch.float32
I32 = torch.int32
ROTARY = dict(q=((1, 3, 2, 2, 8), F), k=((1, 5, 2, 2, 8), F), frequencies=((4,), torch.int64), q_weight=((8,), F), k_weight=((8,), F),
              pos_q=((1, 3), I32), pos_k=((1, 5), I32))
CACHE = dict(k_cache=((4, 2, 2, 2, 8), F), v_cache=((4, 2, 2, 16), F), page_table=((1, 4), I32), counts=((1,), I32))
CALLS = {
    "qkr_forward": {**ROTARY, "out_q": ROTARY["q"], "out_k": ROTARY["k"]},
    "qkr_backward": {**ROTARY, "grad_out_q": ROTARY["q"], "grad_out_k": ROTARY["k"]},
    "paged_append": {"k": ((1, 3, 2, 2, 8), F), "v": ((1, 3, 2, 16), F), **CACHE, "lengths": ((1,), I32), "q": ROTARY["q"],
                     "frequencies": ROTARY["frequencies"], "q_weight": ((8,), F), "k_weight": ((8,), F), "positions": ((1, 3), I32),
                     "out_q": ROTARY["q"]},
    "paged_attention": {"q": ROTARY["q"], **CACHE, "lam": ((2,), F), "key_lengths": ((1,), I32), "tree": ((1, 3, 3), torch.bool),
                        "bias_table": ((4, 2), F), "bucket_map": ((5,), I32), "pos_q": ((1, 3), I32), "pos_k": ((1, 8), I32),
                        "key_mask": ((1, 8), torch.bool), "out": ((1, 3, 2, 16), F)},
}


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU there, tensors without storage need its devices")
@pytest.mark.parametrize("call,other", [(c, n) for c, a in CALLS.items() for n in a])
def test_tensors_of_two_devices_are_refused(monkeypatch, call, other):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 101

    class Current:
        def __init__(self, index):
            pass

        __enter__ = __exit__ = lambda *a: None

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: Stream)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")
        a = {n: torch.empty(s, dtype=t, device="cuda:0" if n == other else "cuda:1") for n, (s, t) in CALLS[call].items()}
        with pytest.raises(ValueError, match="one CUDA device"):
            getattr(da, call)(**a)


# ---- smoke()'s check of these operators: plain ones pass, zeros do not ------

def _plain():
    def forward(q, k, turns, wq, wk):
        return tuple(qkr_reference(x, turns, w)[0]["out"].to(x.dtype) for x, w in ((q, wq), (k, wk)))

    def backward(q, k, gq, gk, turns, wq, wk):
        v = [qkr_reference(x, turns, w, grad=g)[0] for x, w, g in ((q, wq, gq), (k, wk, gk))]
        return v[0]["grad_x"].to(q.dtype), v[1]["grad_x"].to(k.dtype), v[0]["grad_weight"], v[1]["grad_weight"]

    def append(k, v, k_cache, v_cache, table, lengths, q, frequencies, q_weight, k_weight):
        place = lengths[:, None] + torch.arange(k.shape[1])
        at = table.long().gather(1, place // k_cache.shape[1]), place % k_cache.shape[1]
        k_cache[at] = qkr_reference(k, frequencies, k_weight, place)[0]["out"].to(k.dtype)
        v_cache[at] = v
        return qkr_reference(q, frequencies, q_weight, place)[0]["out"].to(q.dtype)

    def attention(q, k_cache, v_cache, lam, table, lengths):
        return paged_reference(q, k_cache, v_cache, lam, table, lengths)[0]["out"].to(q.dtype)

    return types.SimpleNamespace(rotary_frequencies=da.rotary_frequencies, qkr_forward=forward, qkr_backward=backward, paged_append=append,
                                 paged_attention=attention)


def test_plain_operators_pass_smoke():
    __graft_entry__._serving(_plain(), torch.device("cpu"))


@pytest.mark.parametrize("name,at", [("qkr_forward", 0), ("qkr_forward", 1), ("qkr_backward", 0), ("qkr_backward", 1), ("qkr_backward", 2),
                                     ("qkr_backward", 3), ("paged_append", None), ("paged_attention", None)])
def test_zeros_do_not_pass_smoke(name, at):
    ops = _plain()
    right = getattr(ops, name)

    def wrong(*args, **kw):
        r = right(*args, **kw)
        if at is None:
            return torch.zeros_like(r)
        return tuple(torch.zeros_like(x) if i == at else x for i, x in enumerate(r))

    setattr(ops, name, wrong)
    with pytest.raises(AssertionError, match="off by"):
        __graft_entry__._serving(ops, torch.device("cpu"))
