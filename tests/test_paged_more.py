"""More of the attention over a paged cache against 64 bits: what falls just
outside the tensor cores' rule at sizes of prompts, the first tile past 64 rows
of narrow heads, and the fp32 units' tiles with values at masked places that are
not finite."""
import pytest
import torch

import deformable_view_feature_gb300 as da
import test_paged
from operator_refs import check
from serving_refs import paged_reference


@pytest.fixture(scope="module", autouse=True)
def built():
    da.build.build()


CASES = [
    ("sixty-five rows of narrow heads", "tensor", dict(B=2, N=9, S=64, T=65, kind="bf16", lengths=[576, 300])),
    ("sixty-five rows of one narrow head", "tensor", dict(B=2, N=9, S=64, T=65, H=1, Hk=1, kind="f16", lengths=[576, 65])),
    ("narrowest heads", "tensor", dict(B=2, N=9, S=16, T=3, D=8, Dv=8, kind="bf16", lengths=[144, 77])),
    ("narrowest heads, many rows", "tensor", dict(B=2, N=9, S=8, T=70, D=8, Dv=16, kind="f16", lengths=[72, 71])),
    ("wide heads, a prompt's part", "general", dict(B=2, N=20, S=32, T=150, H=4, Hk=2, D=128, kind="bf16", lengths=[640, 201])),
    ("wide heads, few rows", "general", dict(B=2, N=20, S=32, T=2, H=4, Hk=2, D=128, kind="bf16", lengths=[640, 201])),
    ("a little wider than the tiles", "general", dict(B=2, N=20, S=32, T=70, H=4, Hk=2, D=72, kind="f16", lengths=[640, 201], tree="random")),
    ("wide values", "general", dict(B=2, N=20, S=32, T=70, H=4, Hk=2, D=64, Dv=136, kind="bf16", lengths=[640, 201])),
    ("pages of 20, a prompt's part", "general", dict(B=2, N=40, S=20, T=150, H=4, Hk=2, D=64, kind="bf16", lengths=[800, 333], counts=[150, 77])),
    ("pages of 20, one token", "general", dict(B=3, N=40, S=20, T=1, H=8, Hk=2, D=64, kind="f16", lengths=[800, 333, 1])),
    ("a bias of 48 heads, one token", "general", dict(B=2, N=20, S=16, T=1, H=48, Hk=12, D=32, kind="bf16", lengths=[320, 101], buckets=32, reach=128)),
    ("a bias of 48 heads, a prompt's part", "general", dict(B=2, N=20, S=16, T=90, H=48, Hk=12, D=32, kind="bf16", lengths=[320, 101], buckets=32, reach=128)),
    ("a bias as large as there is room for", "tensor", dict(B=2, N=20, S=16, T=20, H=40, Hk=10, D=32, kind="bf16", lengths=[320, 101], buckets=32, reach=255)),
]
assert len({name for name, *_ in CASES}) == len(CASES), "a name twice"


@pytest.mark.gpu
@pytest.mark.parametrize("name,path,kw", CASES, ids=[c[0] for c in CASES])
def test_against_64_bits(name, path, kw):
    t, opt = test_paged._attention_case(**kw)
    assert da.paged_path(**t, **opt) == path
    got = da.paged_attention(**t, **opt)
    check({"out": got}, *paged_reference(**t, **opt))
    assert torch.equal(got, da.paged_attention(**t, **opt)), "results vary from run to run"


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T,D", [("f32", 30, 64), ("f32", 30, 32), ("f32", 30, 100), ("f32", 5, 32), ("bf16", 30, 17), ("f16", 30, 100)])
def test_what_masked_places_hold_is_not_used_in_tiles(kind, T, D):
    test_paged.test_what_masked_places_hold_is_not_used(kind, T, D)
