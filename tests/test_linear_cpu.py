"""Host-side checks of linear and linear_backward that need no GPU: arguments that the C
ABI refuses before any CUDA call, and calls whose tensors or stream are not the current
device's (CPU tensors that say they are CUDA tensors, and a library that records)."""
import pytest
import torch

import layout_folding_gb300 as lf
from layout_folding_gb300 import build as lfbuild
from test_current_device_cpu import BF16, E4M3, FP32, Stream, current, library, on  # noqa: F401

A, B, C = (i << 24 for i in (1, 2, 3))  # distinct, 16-byte aligned, never used: validation fails before
NULL, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    lfbuild.build()
    return lf.lib()


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL),
    (dict(act=4), SHAPE), (dict(act=-1), SHAPE), (dict(bias_dtype=1), SHAPE), (dict(bias_dtype=3), SHAPE),
    (dict(M=0), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(N=1 << 31), SHAPE), (dict(M=1 << 31), SHAPE),
    (dict(x=A + 8), ALIGN), (dict(w=A + 8), ALIGN), (dict(out=A + 8), ALIGN), (dict(pre=B + 8), ALIGN),
    (dict(bias=A + 8), ALIGN), (dict(bias=A + 4, bias_dtype=2), ALIGN), (dict(residual=A + 8), ALIGN),
    (dict(N=60), ALIGN), (dict(K=60), ALIGN), (dict(K=1), ALIGN),
    (dict(pre=A), SHAPE), (dict(pre=C), SHAPE),      # over out, over the residual
])
def test_linear_rejects_on_host(L, kw, want):
    a = dict(x=A, w=A, bias=A, bias_dtype=0, act=3, residual=C, out=A, pre=B, M=4, N=64, K=64)
    a.update(kw)
    assert L.linear(*[a[k] for k in ("x", "w", "bias", "bias_dtype", "act", "residual", "out", "pre", "M", "N", "K")],
                    None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(xs=None), NULL), (dict(w=None), NULL), (dict(ws=None), NULL), (dict(out=None), NULL),
    (dict(act=7), SHAPE), (dict(bias_dtype=1), SHAPE), (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(x=A + 8), ALIGN), (dict(xs=A + 2), ALIGN), (dict(w=A + 8), ALIGN), (dict(ws=A + 4), ALIGN),
    (dict(bias=A + 8), ALIGN), (dict(residual=A + 8), ALIGN), (dict(out=A + 2), ALIGN), (dict(N=60), ALIGN),
    (dict(K=72), ALIGN),
])
def test_linear_e4m3_rejects_on_host(L, kw, want):
    a = dict(x=A, xs=A, w=A, ws=A, bias=A, bias_dtype=2, act=0, residual=C, out=A, M=4, N=64, K=64)
    a.update(kw)
    assert L.linear_e4m3(*[a[k] for k in ("x", "xs", "w", "ws", "bias", "bias_dtype", "act", "residual", "out", "M", "N",
                                          "K")], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dout=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(pre=None), NULL), (dict(dz=None), NULL),
    (dict(scratch=None, M=64, N=8192), NULL), (dict(scratch=None, M=4096, N=13824, K=5120), NULL),
    (dict(scratch=A + 8), ALIGN), (dict(act=4), SHAPE), (dict(bias_dtype=1), SHAPE), (dict(M=0), SHAPE),
    (dict(N=1 << 31), SHAPE), (dict(K=1 << 31), SHAPE),
    (dict(dout=A + 8), ALIGN), (dict(x=A + 8), ALIGN), (dict(w=A + 8), ALIGN), (dict(pre=A + 8), ALIGN),
    (dict(dz=A + 8), ALIGN), (dict(dx=A + 8), ALIGN), (dict(dw=A + 8), ALIGN), (dict(db=A + 8), ALIGN),
    (dict(N=12), ALIGN), (dict(K=12), ALIGN),
])
def test_linear_backward_rejects_on_host(L, kw, want):
    a = dict(dout=A, x=A, w=A, pre=A, act=0, dz=A, dx=A, dw=A, db=A, bias_dtype=0, scratch=A, M=4, N=64, K=64)
    a.update(kw)
    assert L.linear_backward(*[a[k] for k in ("dout", "x", "w", "pre", "act", "dz", "dx", "dw", "db", "bias_dtype",
                                              "scratch", "M", "N", "K")], None) == want


def test_the_gated_operators_still_refuse_no_activation(L):
    assert L.gated_ffn(A, A, 3, A, None, 4, 64, 64, None) == SHAPE
    with pytest.raises(ValueError):
        lf.gated_ffn(torch.zeros(4, 16, dtype=BF16), torch.zeros(16, 16, dtype=BF16), act=None)


def test_scratch_size(L):
    size = L.linear_backward_scratch
    assert size(0, 64, 64) == size(64, 0, 64) == size(64, 64, -1) == size(64, 1 << 31, 64) == 0
    assert size(64, 64, 64) == 0                     # one block has all rows, one pair each product
    # enough tiles: only the bias's partial sums
    assert 0 < size(4096, 13824, 5120) <= 64 * 13824 * 4
    for M, N, K in ((1, 13824, 5120), (333, 5632, 2048), (64, 8192, 64), (100000, 64, 64)):
        assert 0 < size(M, N, K) < 200 << 20


# ---------------------------------------------------------------- the current device
def linear(i, stream=None):
    return lf.linear(on(i, (4, 32)), on(i, (64, 32)), bias=on(i, (64,)), residual=on(i, (4, 64)), out=on(i, (4, 64)),
                     stream=stream)


def linear_e4m3(i, stream=None):
    return lf.linear(on(i, (4, 32), E4M3), on(i, (64, 32), E4M3), x_scale=on(i, (4,), FP32), w_scale=on(i, (64,), FP32),
                     out=on(i, (4, 64)), stream=stream)


def linear_backward(i, stream=None):
    # (the recorder's scratch size is 0)
    return lf.linear_backward(on(i, (4, 64)), on(i, (4, 32)), on(i, (64, 32)), pre=on(i, (4, 64)), act="silu",
                              dz=on(i, (4, 64)), dx=on(i, (4, 32)), dw=on(i, (64, 32)), dbias=on(i, (64,)), stream=stream)


CALLS = [linear, linear_e4m3, linear_backward]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("tensors,device", [(1, 0), (0, 1)])
def test_tensors_of_another_device(monkeypatch, library, call, tensors, device):  # noqa: F811
    current(monkeypatch, device)
    with pytest.raises(ValueError, match="cuda:%d.*current device is cuda:%d" % (tensors, device)):
        call(tensors)
    assert not library.calls


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_stream_of_another_device(monkeypatch, library, call):  # noqa: F811
    current(monkeypatch, 0)
    with pytest.raises(ValueError, match="stream.*cuda:1"):
        call(0, stream=Stream(1))
    assert not library.calls


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_on_the_current_device(monkeypatch, library, call):  # noqa: F811
    current(monkeypatch, 1)
    call(1)
    call(1, stream=Stream(1))
    calls = [(name, args) for name, args in library.calls if not name.endswith("_scratch")]
    assert [args[-1] for _, args in calls] == [1001, 77]


def test_operands_of_two_devices(monkeypatch, library):  # noqa: F811
    current(monkeypatch, 0)
    good = dict(x=(4, 32), w=(64, 32), bias=(64,), residual=(4, 64), out=(4, 64), pre=(4, 64))
    for other in good:
        with pytest.raises(ValueError):
            lf.linear(**{k: on(1 if k == other else 0, s) for k, s in good.items()})
    assert not library.calls
