"""Which device the group norm and the differential attention run on: their
tensors', which is made current; tensors of several devices are refused. On
the CPU, with tensors without storage and a recorded torch.cuda."""
import types
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import deformable_view_feature_gb300 as da

FAKE = FakeTensorMode()


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


def _cases():
    ss, ls = torch.tensor([[[4, 4]]], dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32)
    with FAKE, warnings.catch_warnings():
        def new(*shape, kind=torch.float32, on=1):
            return torch.empty(*shape, dtype=kind, device=f"cuda:{on}")

        norm = dict(feat=(1, 16, 8), gamma=(8,), beta=(8,), out=(1, 16, 8))
        back = dict(feat=(1, 16, 8), gamma=(8,), beta=(8,), stats=(1, 1, 1, 2, 2), grad_out=(1, 16, 8), grad_feat=(1, 16, 8))
        att = dict(q=((1, 3, 2, 2, 8),), k=((1, 5, 2, 2, 8),), v=((1, 5, 2, 16),), lam=((2,),), bias_table=((4, 2),),
                   bucket_map=((5,), torch.int32), pos_q=((1, 3), torch.int32), pos_k=((1, 5), torch.int32),
                   key_mask=((1, 5), torch.bool), key_lengths=((1,), torch.int32), out=((1, 3, 2, 16),))
        for other in norm:
            if other != "feat":
                a = {n: new(*s, on=0 if n == other else 1) for n, s in norm.items()}
                yield f"gn_forward {other}", lambda a=a: da.gn_forward(a["feat"], ss, ls, a["gamma"], a["beta"], 2, out=a["out"])
        for other in back:
            if other != "feat":
                a = {n: new(*s, on=0 if n == other else 1) for n, s in back.items()}
                yield f"gn_backward {other}", lambda a=a: da.gn_backward(a["feat"], ss, ls, a["gamma"], a["beta"], a["stats"],
                                                                         a["grad_out"], 2, grad_feat=a["grad_feat"])
        for other in att:
            if other != "q":
                a = {n: new(*s[0], kind=s[1] if len(s) > 1 else torch.float32, on=0 if n == other else 1) for n, s in att.items()}
                yield f"dattn_forward {other}", lambda a=a: da.dattn_forward(**a)
        a = {n: new(*s[0], kind=s[1] if len(s) > 1 else torch.float32) for n, s in att.items()}
        out, near, far = a.pop("out"), new(1, 2, 2, 3), new(1, 3, 2, 16, on=0)
        yield "dattn_backward grad_out", lambda: da.dattn_backward(out=out, saved=(out, near), grad_out=far, **a)
        yield "dattn_backward out", lambda: da.dattn_backward(out=far, saved=(out, near), grad_out=out, **a)
        yield "dattn_backward saved", lambda: da.dattn_backward(out=out, saved=(far, near), grad_out=out, **a)


CASES = dict(_cases())


@pytest.mark.parametrize("name", list(CASES))
def test_tensors_of_two_devices_are_refused(cuda, name):
    with FAKE, warnings.catch_warnings():
        warnings.simplefilter("ignore")
        with pytest.raises(ValueError, match="one CUDA device"):
            CASES[name]()
