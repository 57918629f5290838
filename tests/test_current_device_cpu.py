"""Calls whose tensors or stream are not the current device's: the binding refuses
them before anything is allocated or launched.  Nothing here touches a GPU: the
tensors are CPU tensors that say they are CUDA tensors, the current device is a
number, and the library is a recorder."""
import pytest
import torch

import layout_folding_gb300 as lf
from layout_folding_gb300 import ffn

BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


class OnCuda(torch.Tensor):
    """A CPU tensor that calls itself a tensor of cuda:`index`."""
    index = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


class Stream:
    cuda_stream = 77

    def __init__(self, index):
        self.device = torch.device("cuda", index)


class Recorder:
    """Stands for the library: every call is noted and succeeds."""
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


def on(index, shape, dtype=BF16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(OnCuda)
    t.index = index
    return t


@pytest.fixture
def library(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(ffn, "_L", rec)
    monkeypatch.setattr(ffn, "_raw_stream", lambda device: 1000 + device)
    return rec


def current(monkeypatch, index):
    monkeypatch.setattr(ffn, "_current_device", lambda: index)


def add_rms_norm(i, stream=None):
    x = on(i, (4, 64))
    return lf.add_rms_norm(x, on(i, (64,)), residual=x, h=on(i, (4, 64)), y=on(i, (4, 64)), stream=stream)


def add_rms_norm_backward(i, stream=None):
    x = on(i, (4, 64))
    return lf.add_rms_norm_backward(x, x, on(i, (64,)), dx=on(i, (4, 64)), want_dweight=False, stream=stream)


def gated_ffn(i, stream=None):
    return lf.gated_ffn(on(i, (4, 32)), on(i, (128, 32)), out=on(i, (4, 64)), stream=stream)


def gated_ffn_e4m3(i, stream=None):
    return lf.gated_ffn(on(i, (4, 32), E4M3), on(i, (128, 32), E4M3), x_scale=on(i, (4,), FP32),
                        w_scale=on(i, (128,), FP32), out=on(i, (4, 64)), stream=stream)


def gated_ffn_backward(i, stream=None):
    # (the recorder's scratch size is 0)
    return lf.gated_ffn_backward(on(i, (4, 64)), on(i, (4, 32)), on(i, (128, 32)), on(i, (4, 128)), dgu=on(i, (4, 128)),
                                 dx=on(i, (4, 32)), dw=on(i, (128, 32)), stream=stream)


FFN = [add_rms_norm, add_rms_norm_backward, gated_ffn, gated_ffn_e4m3, gated_ffn_backward]


@pytest.mark.parametrize("call", FFN, ids=lambda f: f.__name__)
@pytest.mark.parametrize("tensors,device", [(1, 0), (0, 1)])
def test_feed_forward_tensors_of_another_device(monkeypatch, library, call, tensors, device):
    current(monkeypatch, device)
    with pytest.raises(ValueError, match="cuda:%d.*current device is cuda:%d" % (tensors, device)):
        call(tensors)
    assert not library.calls


@pytest.mark.parametrize("call", FFN, ids=lambda f: f.__name__)
def test_feed_forward_stream_of_another_device(monkeypatch, library, call):
    current(monkeypatch, 0)
    with pytest.raises(ValueError, match="stream.*cuda:1"):
        call(0, stream=Stream(1))
    assert not library.calls


@pytest.mark.parametrize("call", FFN, ids=lambda f: f.__name__)
def test_feed_forward_on_the_current_device(monkeypatch, library, call):
    """Any device may be the current one; the call goes to its stream, or to the given one."""
    current(monkeypatch, 1)
    call(1)
    call(1, stream=Stream(1))
    calls = [(name, args) for name, args in library.calls if not name.endswith("_scratch")]
    assert [args[-1] for _, args in calls] == [1001, 77]


def test_feed_forward_calls_without_rows_are_refused_too(monkeypatch, library):
    current(monkeypatch, 0)
    with pytest.raises(ValueError):
        lf.add_rms_norm(on(1, (0, 64)), on(1, (64,)))
    with pytest.raises(ValueError):
        lf.gated_ffn(on(1, (0, 32)), on(1, (128, 32)))
