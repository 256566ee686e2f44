"""Which device the group norm and the differential attention run on: their
tensors', which is made current; tensors of several devices are refused. On
the CPU, with tensors without storage and a recorded torch.cuda."""
import types
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import deformable_view_feature_gb300 as da


@pytest.fixture(scope="module", autouse=True)
def lib():
    da.build.build()
    return da.load_library()


class _Context:
    def __init__(self, log, what):
        self.log, self.what = log, what

    def __enter__(self):
        self.log.append(("enter", self.what))

    def __exit__(self, *exc):
        self.log.append(("exit", self.what))


@pytest.fixture
def cuda(monkeypatch):
    """torch.cuda with device 0 current; the log of what was made current."""
    log = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda index: _Context(log, index))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: _Context(log, s.device.index))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: _stream(0 if index is None else index))
    return log


def _stream(index):
    return types.SimpleNamespace(device=torch.device("cuda", index), cuda_stream=100 + index)


def test_the_tensors_device_is_current_during_a_call(cuda):
    with da._on_stream(None, torch.device("cuda", 1)) as handle:
        assert handle == 101 and cuda == [("enter", 1)]
    assert cuda == [("enter", 1), ("exit", 1)]
    del cuda[:]
    with da._on_stream(None, torch.device("cuda", 0)) as handle:
        assert handle == 100
    with da._on_stream(_stream(1), torch.device("cuda", 1)) as handle:
        assert handle == 101 and cuda == [("enter", 1)]
    del cuda[:]
    with pytest.raises(ValueError, match="one CUDA device"):
        with da._on_stream(_stream(1), torch.device("cuda", 0)):
            pass
    assert not cuda


def test_the_status_of_waits_is_read_on_the_streams_device(cuda, monkeypatch):
    lib, seen = types.SimpleNamespace(), []

    def status(word, handle):
        seen.append((handle, list(cuda)))
        return 0

    lib.gn_device_status = lib.dattn_device_status = status
    monkeypatch.setattr(da, "load_library", lambda: lib)
    assert not da.waits_gave_up(_stream(1)) and not da.waits_gave_up()
    assert [s[0] for s in seen] == [101, 101, 100, 100] and seen[0][1] == [("enter", 1)]


NORM = dict(feat=(1, 16, 8), gamma=(8,), beta=(8,), out=(1, 16, 8))
NORM_BACK = dict(feat=(1, 16, 8), gamma=(8,), beta=(8,), stats=(1, 1, 1, 2, 2), grad_out=(1, 16, 8), grad_feat=(1, 16, 8))
ATTENTION = dict(q=(1, 3, 2, 2, 8), k=(1, 5, 2, 2, 8), v=(1, 5, 2, 16), lam=(2,), bias_table=(4, 2), bucket_map=(5,),
                 pos_q=(1, 3), pos_k=(1, 5), key_mask=(1, 5), key_lengths=(1,), out=(1, 3, 2, 16))
ATTENTION_BACK = {**ATTENTION, "out1": (1, 3, 2, 16), "lse": (1, 2, 2, 3), "grad_out": (1, 3, 2, 16)}
KINDS = dict(bucket_map=torch.int32, pos_q=torch.int32, pos_k=torch.int32, key_mask=torch.bool, key_lengths=torch.int32)


def _gn_forward(ss, ls, a):
    return da.gn_forward(a["feat"], ss, ls, a["gamma"], a["beta"], 2, out=a["out"])


def _gn_backward(ss, ls, a):
    return da.gn_backward(a["feat"], ss, ls, a["gamma"], a["beta"], a["stats"], a["grad_out"], 2, grad_feat=a["grad_feat"])


def _dattn_forward(ss, ls, a):
    return da.dattn_forward(**a)


def _dattn_backward(ss, ls, a):
    return da.dattn_backward(saved=(a.pop("out1"), a.pop("lse")), **a)


CASES = [(call, shapes, other) for call, shapes in ((_gn_forward, NORM), (_gn_backward, NORM_BACK), (_dattn_forward, ATTENTION),
                                                    (_dattn_backward, ATTENTION_BACK)) for other in list(shapes)[1:]]


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU there, tensors without storage need its devices")
@pytest.mark.parametrize("call,shapes,other", CASES, ids=[f"{c[0].__name__[1:]}-{c[2]}" for c in CASES])
def test_tensors_of_two_devices_are_refused(cuda, call, shapes, other):
    ss, ls = torch.tensor([[[4, 4]]], dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")
        a = {n: torch.empty(s, dtype=KINDS.get(n, torch.float32), device="cuda:0" if n == other else "cuda:1") for n, s in shapes.items()}
        with pytest.raises(ValueError, match="one CUDA device"):
            call(ss, ls, a)
