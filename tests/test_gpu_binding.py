"""The compiled part of the binding: it is built and takes the plain calls, its results are
those of the Python functions, and what it does not take is done or refused by those."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import layout_folding_gb300 as lf
from layout_folding_gb300 import compiled

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def normal(shape, seed, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


@pytest.fixture
def taken(monkeypatch):
    """Counts the calls that the compiled functions take."""
    module = compiled.load()
    assert module is not None, "the compiled part of the binding is not built"
    count = []
    for name in compiled._NAMES:
        def call(*args, f=getattr(module, name), name=name):
            made = f(*args)
            if made is not None:
                count.append(name)
            return made
        monkeypatch.setattr(compiled, name, call)
    return count


def same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        if x is None or y is None:
            assert x is None and y is None
            continue
        assert x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride() and x.device == y.device
        assert not x.requires_grad and not y.requires_grad
        assert torch.equal(x.flatten().view(torch.uint8), y.flatten().view(torch.uint8))


def block_calls(dtype, wdtype, shape):
    D = shape[-1]
    x, res, dy, h, dh = (normal(shape, i, dtype) for i in range(5))
    w, v = normal((D,), 6, wdtype), normal((D,), 7, wdtype)
    rows = x.numel() // D
    for gate in (None, normal((D,), 8, dtype), normal((1, D), 9, FP32), normal((rows, D), 10, dtype)):
        for post, pre in ((w, v), (None, v), (w, None), (None, None)):
            kw = dict(post=post, pre=pre, gate=gate, branch_scale=0.5, residual_scale=2)
            for fp8 in (False, True) if pre is not None else (False,):
                yield lambda fp8=fp8, kw=kw, **k: lf.block_norm(x, res, fp8=fp8, **kw, **k)
            for want in (True, False):
                yield lambda want=want, kw=kw, **k: lf.block_norm_backward(dy, x, h, dh=dh, want_dparams=want, **kw, **k)
    yield lambda **k: lf.block_norm_backward(dy, x, h, pre=w, **k)


def linear_calls(lead):
    N, K = 72, 48
    x, w, res, dout = normal((*lead, K), 1), normal((N, K), 2), normal((*lead, N), 3), normal((*lead, N), 4)
    M = x.numel() // K
    s, t = torch.rand(M, device=DEV) + 0.5, torch.rand(N, device=DEV) + 0.5
    for b in (None, normal((N,), 5), normal((N,), 6, FP32)):
        for act in (None, "silu", "gelu", "gelu_tanh"):
            for r in (None, res):
                yield lambda b=b, act=act, r=r, **k: lf.linear(x, w, bias=b, act=act, residual=r, want_pre=r is None, **k)
                yield lambda b=b, act=act, r=r, **k: lf.linear(x.to(E4M3), w.to(E4M3), bias=b, act=act, residual=r,
                                                              x_scale=s, w_scale=t, **k)
            for dx, dw in ((True, True), (False, True), (True, False)):
                yield lambda b=b, act=act, dx=dx, dw=dw, **k: lf.linear_backward(dout, x, w, pre=res, act=act, bias=b,
                                                                               want_dx=dx, want_dw=dw, **k)


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, FP32), (FP16, FP16), (FP32, FP32)])
@pytest.mark.parametrize("shape", [(6, 64), (2, 3, 33), (1, 1, 5, 64), (64,)])
def test_block_norm_as_in_python(taken, dtype, wdtype, shape):
    n = 0
    for call in block_calls(dtype, wdtype, shape):
        got = call()
        n += 1
        assert len(taken) == n
        same(got, call(stream=torch.cuda.current_stream()))  # (a stream: the Python function)
        assert len(taken) == n
    lf.check_device_error()


@pytest.mark.parametrize("lead", [(5,), (2, 3), ()])
def test_linear_as_in_python(taken, lead):
    n = 0
    for call in linear_calls(lead):
        got = call()
        n += 1
        assert len(taken) == n
        same(got, call(stream=torch.cuda.current_stream()))
        assert len(taken) == n
    lf.check_device_error()


def test_parameters_and_leaves_that_require_gradients(taken):
    x, w = normal((4, 64), 1), torch.nn.Parameter(normal((64,), 2))
    same(lf.block_norm(x.clone().requires_grad_(), x, w, w), lf.block_norm(x, x, w.detach(), w.detach()))
    assert len(taken) == 2


def test_on_the_current_stream_and_captured(taken):
    x, w = normal((700, 520), 1), normal((520,), 2)
    want = lf.block_norm(x, x, w, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late = x * 1                                   # ready only after the sleep, on the side stream
        got = lf.block_norm(late, late, w, w)
    side.synchronize()
    same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = lf.block_norm(x, x, w, w)
        grad = lf.block_norm_backward(x, x, x, w, w)
    graph.replay()
    torch.cuda.synchronize()
    same(got, want)
    same(grad, lf.block_norm_backward(x, x, x, w, w))
    lf.check_device_error()


def test_a_dispatch_mode_sees_the_outputs(taken):
    class Count(TorchDispatchMode):
        made = 0

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.made += func.overloadpacket.__name__ == "empty"
            return func(*args, **(kwargs or {}))
    x, w = normal((6, 64), 1), normal((64,), 2)
    W = normal((64, 64), 3)
    with Count() as count:
        lf.block_norm(x, x, w, w, fp8=True)
        lf.block_norm_backward(x, x, x, w, w)
        lf.linear(x, W, want_pre=True)
    assert count.made >= 3 + 5 + 2 and len(taken) == 3


def test_what_is_not_plain_is_left_to_python(taken):
    x, w, W = normal((6, 64), 1), normal((64,), 2), normal((64, 64), 3)
    wide = normal((6, 128), 4)[:, :64]
    lf.block_norm(wide, x, w, w)                                  # rows of a wider tensor
    lf.block_norm(x[:0], x[:0], w, w)                             # no rows
    lf.block_norm(x.view(2, 3, 64), x.view(2, 3, 64), w, w, gate=normal((2, 1, 64), 5))
    lf.linear(x[:0], W)
    lf.linear(x, W, out=torch.empty_like(x))
    for call in (lambda: lf.block_norm(x, x[:3], w, w), lambda: lf.block_norm(x, x, w, w.float()),
                 lambda: lf.block_norm(x, x.float(), w, w), lambda: lf.block_norm(x, x, w[:32], w),
                 lambda: lf.block_norm(x, x, w, None, fp8=True), lambda: lf.block_norm(x.cpu(), x, w, w),
                 lambda: lf.block_norm(x, x, w, w, gate=normal((4, 64), 6)), lambda: lf.block_norm(x, x, w, w, gate=w.half()),
                 lambda: lf.block_norm_backward(None, x, x, w, w), lambda: lf.block_norm_backward(x, x, x, w),
                 lambda: lf.linear(x, W[:, :32]), lambda: lf.linear(x.half(), W.half()), lambda: lf.linear(x, W, bias=w[:8]),
                 lambda: lf.linear(x, W, residual=x[:3]), lambda: lf.linear(x.to(E4M3), W.to(E4M3), x_scale=w.float()),
                 lambda: lf.linear_backward(x, x, W, act="silu"), lambda: lf.linear_backward(x[:3], x, W)):
        with pytest.raises((ValueError, TypeError)):
            call()
    assert not taken
    with pytest.raises(lf.LayoutFoldError) as info:               # refused by the library itself
        lf.block_norm(x, x, w, w, eps=-1.0)
    assert info.value.status == 2 and taken == ["block_norm"]
    with pytest.raises(lf.LayoutFoldError) as info:
        lf.linear(normal((4, 60), 1), normal((64, 60), 2))
    assert info.value.status == 3
