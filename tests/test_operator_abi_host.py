"""The C ABI of the group norm and the differential attention on the CPU: the
headers are plain C, the library exports what they declare, and the binding's
structures have the headers' layout."""
import ctypes
import os
import re
import subprocess

import pytest

import deformable_view_feature_gb300 as da
from deformable_view_feature_gb300 import attention, norm

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


@pytest.fixture(scope="module")
def lib():
    da.build.build()
    return da.load_library()


def test_library_exports_what_the_headers_declare(lib):
    names = set()
    for h in ("gn.h", "dattn.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, h)).read(), flags=re.S)
        names |= set(re.findall(r"\b((?:gn|dattn)_[a-z0-9_]+)\s*\(", text))
    assert {"gn_forward", "gn_backward", "gn_workspace_size", "gn_device_status", "dattn_forward", "dattn_backward",
            "dattn_workspace_size", "dattn_path", "dattn_device_status"} == names
    for n in names:
        getattr(lib, n)


def test_headers_are_plain_c_and_structures_agree(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gn.h"\n#include "dattn.h"\n'
                   'int main(void){ printf("%zu %zu %zu %zu %zu\\n", sizeof(gn_dims), offsetof(gn_dims, eps),'
                   ' sizeof(dattn_problem), offsetof(dattn_problem, q_stride), offsetof(dattn_problem, key_lengths));'
                   ' return 0; }\n')
    exe = tmp_path / "use"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    G, P = norm.GnDims, attention.DattnProblem
    assert got == [ctypes.sizeof(G), G.eps.offset, ctypes.sizeof(P), P.q_stride.offset, P.key_lengths.offset]


@pytest.mark.parametrize("kw,forward,backward", [
    (dict(), 1, 1),
    (dict(dtype=2), 1, 1),
    (dict(dtype=0), 0, 0),                      # fp32
    (dict(width=64, value_width=128), 1, 1),
    (dict(width=24, value_width=48), 1, 1),
    (dict(width=20), 0, 0),                     # rows of no whole 16 bytes
    (dict(width=72), 0, 0),                     # wider than the tiles
    (dict(value_width=136), 0, 0),
    (dict(num_buckets=40), 1, 0),               # more sums than the backward kernel holds
    (dict(reach=1000), 1, 0),                   # 2 heads * 2129 floats of bias
    (dict(q=0x7F0000000008), 0, 0),             # not 16-byte aligned
    (dict(num_queries=0), 0, 0),
    (dict(width=-1), -1, -1),
])
def test_which_kernels_a_problem_takes(lib, kw, forward, backward):
    d = dict(batch=1, num_queries=4, num_keys=8, num_heads=4, num_kv_heads=2, width=32, value_width=64, dtype=1,
             num_buckets=8, reach=16, causal=0, scale=0.1, q=0x7F0000000000, k=0x7F0000000000, v=0x7F0000000000)
    d.update(kw)
    p = attention.DattnProblem(**d)
    p.q_stride[:] = (1024, 256, 64, 32)
    p.k_stride[:] = (1024, 128, 64, 32)
    p.v_stride[:] = (1024, 128, 64)
    assert lib.dattn_path(ctypes.byref(p), 0) == forward and lib.dattn_path(ctypes.byref(p), 1) == backward
    p.k_stride[1] = 0  # broadcast over the keys
    assert lib.dattn_path(ctypes.byref(p), 0) <= 0
