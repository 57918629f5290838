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
    monkeypatch.setattr(lf, "lib", lambda: rec)
    monkeypatch.setattr(ffn, "_raw_stream", lambda device: 1000 + device)
    return rec


def current(monkeypatch, index):
    monkeypatch.setattr(ffn, "_current_device", lambda: index)
    monkeypatch.setattr(lf, "_current_device", lambda: index)


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


# ---------------------------------------------------------------- the other entry points
def gemm_nt(i, stream=None):
    return lf.gemm_nt(on(i, (16, 64)), on(i, (32, 64)), out=on(i, (16, 32)), stream=stream)


def gemm_nt_xent(i, stream=None, **layout):
    x, w = (64, 16) if layout else (16, 64), (64, 32) if layout else (32, 64)
    return lf.gemm_nt_xent(on(i, x), on(i, w), on(i, (16,), torch.int32), loss=on(i, (16,), FP32), stream=stream, **layout)


def gemm_nt_xent_layout(i, stream=None):
    return gemm_nt_xent(i, stream, x_mn=True, w_mn=True)


def matmul_k1(i, stream=None):
    return lf.matmul_k1(on(i, (8, 1), FP32), on(i, (1, 8), FP32), out=on(i, (8, 8), FP32), stream=stream)


def fp8_cast_dual(i, stream=None):
    return lf.fp8_cast_dual(on(i, (16, 32)), on(i, (1,), FP32), out=on(i, (16, 32), E4M3), out_t=on(i, (32, 16), E4M3),
                            stream=stream)


def rope_cos_sin(i, stream=None):
    return lf.rope_cos_sin(on(i, (8,)), on(i, (16,), torch.int64), cos_out=on(i, (16, 16)), sin_out=on(i, (16, 16)),
                           stream=stream)


def gemm_layout(i, stream=None):
    return lf.gemm_layout(on(i, (64, 16)), on(i, (32, 64)), x_mn=True, out=on(i, (16, 32)), stream=stream)


def matmul(i, stream=None):
    return lf.matmul(on(i, (16, 64)), on(i, (64, 32)), out=on(i, (16, 32)), stream=stream)


def gemm_batched(i, stream=None):
    return lf.gemm_batched(on(i, (2, 16, 64)), False, 64, 1024, on(i, (32, 64)), False, 64, 0, on(i, (2, 16, 32)), 32, 512,
                           2, 16, 32, 64, stream=stream)


def bmm(i, stream=None):
    # (a slice keeps the class, not the index, so the output is three-dimensional)
    return lf.bmm(on(i, (2, 16, 64)), on(i, (2, 64, 32)), out=on(i, (2, 16, 32)), stream=stream)


OTHERS = [gemm_nt, gemm_nt_xent, gemm_nt_xent_layout, matmul_k1, fp8_cast_dual, rope_cos_sin, gemm_layout, matmul,
          gemm_batched, bmm]


@pytest.mark.parametrize("call", OTHERS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("tensors,device", [(1, 0), (0, 1)])
def test_tensors_of_another_device(monkeypatch, library, call, tensors, device):
    current(monkeypatch, device)
    with pytest.raises(ValueError, match="cuda:%d.*current device is cuda:%d" % (tensors, device)):
        call(tensors, stream=Stream(device))
    assert not library.calls


@pytest.mark.parametrize("call", OTHERS + [lambda i, stream: lf.check_device_error(stream)], ids=lambda f: f.__name__)
def test_stream_of_another_device(monkeypatch, library, call):
    current(monkeypatch, 0)
    with pytest.raises(ValueError, match="stream.*cuda:1"):
        call(0, stream=Stream(1))
    assert not library.calls


@pytest.mark.parametrize("call", OTHERS, ids=lambda f: f.__name__)
def test_on_the_current_device(monkeypatch, library, call):
    current(monkeypatch, 1)
    call(1, stream=Stream(1))
    assert [args[-1].value for _, args in library.calls] == [77]


def test_operands_of_two_devices(monkeypatch, library):
    current(monkeypatch, 0)
    for x, w, out in ((0, 1, 0), (0, 0, 1), (1, 0, 0)):
        with pytest.raises(ValueError):
            lf.gemm_nt(on(x, (16, 64)), on(w, (32, 64)), out=on(out, (16, 32)), stream=Stream(0))
    assert not library.calls
