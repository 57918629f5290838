"""Host-side checks of the feed-forward operators that need no GPU: arguments
that the C ABI refuses before any CUDA call, arguments that the binding refuses,
and the references that the GPU tests compare with."""
import ctypes

import pytest
import torch

import ffn_reference as ref
import layout_folding_gb300 as lf
from layout_folding_gb300 import build as lfbuild

A = 1 << 20  # a 16-byte aligned fake address: validation fails before it is used
NULL, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    lfbuild.build()
    return lf.lib()


def norm_args(**kw):
    a = dict(x=A, ldx=64, res=A, ldr=64, w=A, h=A, y=A, scale=None, dtype=0, wdtype=0, ydtype=0, eps=1e-6, M=4, D=64)
    a.update(kw)
    return [a[k] for k in ("x", "ldx", "res", "ldr", "w", "h", "y", "scale", "dtype", "wdtype", "ydtype", "eps", "M",
                           "D")] + [None]


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL),
    (dict(w=None), NULL),
    (dict(y=None), NULL),
    (dict(h=None), NULL),                        # a residual is added: its sum has to go somewhere
    (dict(ydtype=3), NULL),                      # e4m3 without scales
    (dict(ydtype=3, scale=A, dtype=3), SHAPE),   # the stream is not kept in e4m3
    (dict(scale=A), SHAPE),                      # scales without an e4m3 output
    (dict(dtype=-1), SHAPE),
    (dict(dtype=0, wdtype=1), SHAPE),
    (dict(dtype=2, wdtype=0, ydtype=2), SHAPE),
    (dict(dtype=0, ydtype=2), SHAPE),
    (dict(M=0), SHAPE),
    (dict(D=0), SHAPE),
    (dict(M=1 << 31), SHAPE),
    (dict(D=1 << 31, ldx=1 << 31, ldr=1 << 31), SHAPE),
    (dict(ldx=63), SHAPE),
    (dict(ldr=63), SHAPE),
    (dict(eps=-1e-6), SHAPE),
    (dict(eps=float("nan")), SHAPE),
    (dict(x=A + 1), ALIGN),
    (dict(res=A + 1), ALIGN),
    (dict(h=A + 1), ALIGN),
    (dict(y=A + 1), ALIGN),
    (dict(w=A + 2, wdtype=2), ALIGN),
    (dict(x=A + 2, dtype=2, wdtype=2, ydtype=2), ALIGN),
    (dict(ydtype=3, scale=A + 2), ALIGN),
])
def test_add_rms_norm_rejects_on_host(L, kw, want):
    assert L.add_rms_norm(*norm_args(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), NULL), (dict(h=None), NULL), (dict(w=None), NULL), (dict(dx=None), NULL),
    (dict(scratch=None), NULL),                  # dweight without scratch
    (dict(dtype=3), SHAPE), (dict(wdtype=1), SHAPE), (dict(M=0), SHAPE), (dict(D=-1), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(dy=A + 1), ALIGN), (dict(h=A + 1), ALIGN), (dict(dh=A + 1), ALIGN), (dict(dx=A + 1), ALIGN),
    (dict(dw=A + 1), ALIGN), (dict(scratch=A + 2), ALIGN),
])
def test_add_rms_norm_backward_rejects_on_host(L, kw, want):
    a = dict(dy=A, h=A, w=A, dh=A, dx=A, dw=A, scratch=A, dtype=0, wdtype=0, eps=1e-6, M=4, D=64)
    a.update(kw)
    assert L.add_rms_norm_backward(*[a[k] for k in ("dy", "h", "w", "dh", "dx", "dw", "scratch", "dtype", "wdtype",
                                                    "eps", "M", "D")], None) == want


def test_scratch_size(L):
    assert L.add_rms_norm_backward_scratch(0, 64) == 0
    assert L.add_rms_norm_backward_scratch(64, 0) == 0
    assert L.add_rms_norm_backward_scratch(1 << 31, 64) == 0
    assert L.add_rms_norm_backward_scratch(1, 100) >= 400
    # rows of partial sums are bounded however many tokens there are, and never fewer for more of them
    sizes = [L.add_rms_norm_backward_scratch(m, 64) for m in (1, 10, 1000, 100000, (1 << 31) - 1)]
    assert sizes == sorted(sizes) and sizes[-1] == sizes[-2]


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL),
    (dict(act=3), SHAPE), (dict(act=-1), SHAPE), (dict(M=0), SHAPE), (dict(F=0), SHAPE), (dict(K=0), SHAPE),
    (dict(F=1 << 30), SHAPE), (dict(M=1 << 31), SHAPE),
    (dict(x=A + 8), ALIGN), (dict(w=A + 8), ALIGN), (dict(out=A + 8), ALIGN), (dict(gu=A + 8), ALIGN),
    (dict(F=60), ALIGN), (dict(K=60), ALIGN), (dict(K=1), ALIGN),
])
def test_gated_ffn_rejects_on_host(L, kw, want):
    a = dict(x=A, w=A, act=0, out=A, gu=A, M=4, F=64, K=64)
    a.update(kw)
    assert L.gated_ffn(*[a[k] for k in ("x", "w", "act", "out", "gu", "M", "F", "K")], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(xs=None), NULL), (dict(w=None), NULL), (dict(ws=None), NULL), (dict(out=None), NULL),
    (dict(act=7), SHAPE), (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(F=1 << 30), SHAPE),
    (dict(x=A + 8), ALIGN), (dict(xs=A + 2), ALIGN), (dict(w=A + 8), ALIGN), (dict(ws=A + 4), ALIGN),
    (dict(out=A + 2), ALIGN), (dict(F=60), ALIGN), (dict(K=72), ALIGN),
])
def test_gated_ffn_e4m3_rejects_on_host(L, kw, want):
    a = dict(x=A, xs=A, w=A, ws=A, act=0, out=A, M=4, F=64, K=64)
    a.update(kw)
    assert L.gated_ffn_e4m3(*[a[k] for k in ("x", "xs", "w", "ws", "act", "out", "M", "F", "K")], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dout=None), NULL), (dict(x=None), NULL), (dict(w=None), NULL), (dict(gu=None), NULL), (dict(dgu=None), NULL),
    (dict(scratch=None, M=64, F=8192), NULL), (dict(scratch=A + 8), ALIGN),
    (dict(act=3), SHAPE), (dict(M=0), SHAPE), (dict(F=1 << 30), SHAPE),
    (dict(dout=A + 8), ALIGN), (dict(gu=A + 8), ALIGN), (dict(dgu=A + 8), ALIGN), (dict(dx=A + 8), ALIGN),
    (dict(dw=A + 8), ALIGN), (dict(F=12), ALIGN), (dict(K=12), ALIGN),
])
def test_gated_ffn_backward_rejects_on_host(L, kw, want):
    a = dict(dout=A, x=A, w=A, gu=A, act=0, dgu=A, dx=A, dw=A, scratch=A, M=4, F=64, K=64)
    a.update(kw)
    assert L.gated_ffn_backward(*[a[k] for k in ("dout", "x", "w", "gu", "act", "dgu", "dx", "dw", "scratch", "M", "F", "K")],
                                None) == want


def test_gated_ffn_backward_scratch_size(L):
    size = L.gated_ffn_backward_scratch
    assert size(0, 64, 64) == size(64, 0, 64) == size(64, 64, -1) == size(64, 1 << 30, 64) == 0
    assert size(4096, 13824, 5120) == 0          # tiles enough: no sum is split
    for M, F, K in ((1, 13824, 5120), (333, 5632, 2048), (64, 8192, 64), (100000, 64, 64)):
        assert 0 < size(M, F, K) < 200 << 20     # a few parts of 256 x 256 floats for each pair of SMs


def test_binding_refuses_cpu_tensors_and_unknown_activations():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    w = torch.zeros(16, 16, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        lf.add_rms_norm(x, x[0])
    with pytest.raises(TypeError):
        lf.add_rms_norm(None, x[0])
    with pytest.raises(TypeError):
        lf.add_rms_norm_backward(x, x, x[0])
    with pytest.raises(TypeError):
        lf.gated_ffn(x, w)
    with pytest.raises(TypeError):
        lf.gated_ffn_backward(x, x, w, x)
    with pytest.raises(ValueError):
        lf.gated_ffn(x, w, act="relu")


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_reference_gradients_against_differences(name):
    """The 64-bit gradients that the GPU tests use, against central differences of
    the 64-bit forward: step 1e-5, so the truncation (step^2 times a third
    derivative of order one) and the rounding (2^-53 / step) are both below 1e-9."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(3, 8, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(12, 8, generator=g, dtype=torch.float64, requires_grad=True)
    dout = torch.randn(3, 6, generator=g, dtype=torch.float64)
    dx, dw = ref.grads(ref.gated(x, w, name)[0], (x, w), dout)
    for t, dt in ((x, dx), (w, dw)):
        v = torch.randn(t.shape, generator=g, dtype=torch.float64)
        def at(s):
            a, b = (x + s * v, w) if t is x else (x, w + s * v)
            return float((ref.gated(a, b, name)[0] * dout).sum())
        diff = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(diff - float((dt * v).sum())) < 1e-7 * (1 + abs(diff))


def test_reference_norm_gradient_against_its_formula():
    g = torch.Generator().manual_seed(4)
    h = torch.randn(5, 24, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(24, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(5, 24, generator=g, dtype=torch.float64)
    dh, dw = ref.grads(ref.rms_norm(h, w, 1e-5), (h, w), dy)
    r = ref.norm_factor(h, 1e-5)
    gr = dy * w
    want = r * gr - h * r ** 3 * (gr * h).mean(-1, keepdim=True)
    assert torch.allclose(dh, want, rtol=1e-12, atol=1e-12)
    assert torch.allclose(dw, (dy * h * r).sum(0), rtol=1e-12, atol=1e-12)
