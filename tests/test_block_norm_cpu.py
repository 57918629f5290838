"""Host-side checks of block_norm and its gradient that need no GPU: arguments that the C
ABI refuses before any CUDA call, outputs in an input's memory, and calls whose tensors or
stream are not the current device's."""
import pytest
import torch

import layout_folding_gb300 as lf
from layout_folding_gb300 import build as lfbuild
from test_current_device_cpu import BF16, E4M3, FP32, Stream, current, library, on  # noqa: F401

# distinct, 16-byte aligned, never used: validation fails before
X, R, POST, PRE, GATE, H, Y, S, DY, DH, DX, DR, DPO, DPR, DGA, W = (i << 24 for i in range(1, 17))
NULL, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    lfbuild.build()
    return lf.lib()


def forward(L, **kw):
    a = dict(x=X, ldx=64, residual=R, ldr=64, post=POST, pre=PRE, gate=GATE, rows=2, gtype=0, h=H, y=Y, scale=None, dtype=0,
             wdtype=0, ydtype=0, eps=1e-6, b=1.0, a=1.0, M=4, D=64)
    a.update(kw)
    return L.block_norm(*a.values(), None)


def backward(L, **kw):
    a = dict(dy=DY, x=X, h=H, post=POST, pre=PRE, gate=GATE, rows=2, gtype=0, dh=DH, dx=DX, dr=DR, dpost=DPO, dpre=DPR,
             dgate=DGA, scratch=W, dtype=0, wdtype=0, eps=1e-6, b=1.0, a=1.0, M=4, D=64)
    a.update(kw)
    return L.block_norm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(residual=None), NULL), (dict(h=None), NULL), (dict(y=None), NULL),
    (dict(ydtype=3), NULL),                                          # codes without scales
    (dict(scale=S), SHAPE), (dict(pre=None, scale=S), SHAPE), (dict(pre=None, ydtype=3, scale=S), SHAPE),
    (dict(ydtype=1), SHAPE), (dict(dtype=3), SHAPE), (dict(dtype=-1), SHAPE), (dict(wdtype=1), SHAPE),
    (dict(gtype=1), SHAPE), (dict(gtype=3), SHAPE), (dict(dtype=2, ydtype=2), SHAPE),
    (dict(rows=0), SHAPE), (dict(rows=3), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=8), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(M=0), SHAPE), (dict(D=0), SHAPE),
    (dict(M=1 << 31), SHAPE), (dict(D=1 << 31, ldx=1 << 32, ldr=1 << 32), SHAPE), (dict(ldx=63), SHAPE),
    (dict(ldr=63), SHAPE),
    (dict(x=X + 1), ALIGN), (dict(residual=R + 1), ALIGN), (dict(post=POST + 1), ALIGN), (dict(pre=PRE + 1), ALIGN),
    (dict(gate=GATE + 1), ALIGN), (dict(h=H + 1), ALIGN), (dict(y=Y + 1), ALIGN), (dict(gtype=2, gate=GATE + 2), ALIGN),
    (dict(wdtype=2, pre=PRE + 2), ALIGN), (dict(ydtype=3, scale=S + 2), ALIGN),
    # outputs whose rows would lie over other rows' input, or each other's
    (dict(y=H), SHAPE), (dict(h=X, ldx=72), SHAPE), (dict(h=R, ldr=72), SHAPE), (dict(y=X, ldx=72), SHAPE),
    (dict(y=R, ldr=72), SHAPE), (dict(y=X, ydtype=3, scale=S), SHAPE), (dict(y=R, ydtype=3, scale=S), SHAPE),
    (dict(y=R, ydtype=3, scale=S, M=2), SHAPE),
])
def test_forward_rejects_on_host(L, kw, want):
    assert forward(L, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(), dict(post=None), dict(pre=None), dict(pre=None, y=None, ydtype=77), dict(gate=None, rows=0, gtype=9),
    dict(post=None, pre=None, gate=None), dict(h=X), dict(h=R), dict(h=X, y=R), dict(h=R, y=X), dict(y=X, h=H),
    dict(ydtype=3, scale=S), dict(h=R, ldx=72), dict(M=1, rows=1, h=R, ldr=72), dict(gtype=2), dict(rows=4), dict(x=X + 2),
    dict(ydtype=3, scale=S, y=Y + 1),
])
def test_forward_goes_on_to_the_device(L, kw):
    if torch.cuda.is_available():
        pytest.skip("fake addresses, which a call that is not refused would use")
    assert forward(L, **kw) not in (0, NULL, SHAPE, ALIGN)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), NULL), (dict(h=None), NULL), (dict(x=None), NULL), (dict(x=None, post=None, dpost=None), NULL),
    (dict(pre=None, dpre=None, dh=None), NULL), (dict(dx=None), NULL), (dict(dr=None), NULL), (dict(scratch=None), NULL),
    (dict(scratch=None, dpost=None, dpre=None), NULL),
    (dict(post=None), SHAPE), (dict(pre=None), SHAPE), (dict(gate=None), SHAPE), (dict(dx=DR), SHAPE),
    (dict(dtype=3), SHAPE), (dict(wdtype=1), SHAPE), (dict(gtype=1), SHAPE), (dict(rows=3), SHAPE), (dict(rows=0), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(M=0), SHAPE), (dict(D=0), SHAPE), (dict(D=1 << 31), SHAPE),
    (dict(dy=DY + 1), ALIGN), (dict(x=X + 1), ALIGN), (dict(h=H + 1), ALIGN), (dict(dh=DH + 1), ALIGN),
    (dict(dx=DX + 1), ALIGN), (dict(dr=DR + 1), ALIGN), (dict(post=POST + 1), ALIGN), (dict(pre=PRE + 1), ALIGN),
    (dict(gate=GATE + 1), ALIGN), (dict(dpost=DPO + 1), ALIGN), (dict(dpre=DPR + 1), ALIGN), (dict(dgate=DGA + 1), ALIGN),
    (dict(gtype=2, dgate=DGA + 2), ALIGN), (dict(scratch=W + 8), ALIGN),
])
def test_backward_rejects_on_host(L, kw, want):
    assert backward(L, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(), dict(dh=None), dict(dx=DY, dr=DH), dict(dx=X, dr=H), dict(pre=None, dpre=None, dy=None, h=None),
    dict(post=None, dpost=None), dict(post=None, dpost=None, gate=None, dgate=None, x=None),
    dict(dpost=None, dpre=None, dgate=None, scratch=None),
])
def test_backward_goes_on_to_the_device(L, kw):
    if torch.cuda.is_available():
        pytest.skip("fake addresses, which a call that is not refused would use")
    assert backward(L, **kw) not in (0, NULL, SHAPE, ALIGN)


def test_scratch_size(L):
    size = L.block_norm_backward_scratch
    assert size(0, 64, 0, 0) == size(64, 0, 0, 0) == size(64, 64, 3, 0) == size(64, 64, 0, -1) == size(64, 64, 0, 65) == 0
    for M in (1, 7, 8, 9, 151, 303, 304, 305, 607, 608, 5000, 100000):
        for D in (1, 33, 1024, 5121, 20000):
            for dtype in (0, 1, 2):
                lanes = min(M, 304)       # a row of sums for each block at least, two regions
                assert size(M, D, dtype, 0) >= 2 * 4 * lanes * D
                assert size(M, D, dtype, M) >= 4 * (2 * lanes + M - 1) * D
                assert size(M, D, dtype, 0) <= 2 * 4 * 1824 * (D + 4)


# ---------------------------------------------------------------- the current device
def block_norm(i, stream=None):
    return lf.block_norm(on(i, (4, 64)), on(i, (4, 64)), on(i, (64,)), on(i, (64,)), gate=on(i, (2, 64)), h=on(i, (4, 64)),
                         y=on(i, (4, 64)), stream=stream)


def block_norm_e4m3(i, stream=None):
    return lf.block_norm(on(i, (4, 64)), on(i, (4, 64)), None, on(i, (64,)), fp8=True, h=on(i, (4, 64)),
                         y=on(i, (4, 64), E4M3), scale=on(i, (4,), FP32), stream=stream)


def block_norm_backward(i, stream=None):
    x = on(i, (4, 64))
    return lf.block_norm_backward(x, x, x, on(i, (64,)), on(i, (64,)), dx=on(i, (4, 64)), dresidual=on(i, (4, 64)),
                                  want_dparams=False, stream=stream)


CALLS = [block_norm, block_norm_e4m3, block_norm_backward]


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
    assert [args[-1] for _, args in library.calls] == [1001, 77]


def test_operands_of_two_devices(monkeypatch, library):  # noqa: F811
    current(monkeypatch, 0)
    good = dict(x=(4, 64), residual=(4, 64), post=(64,), pre=(64,), gate=(2, 64), h=(4, 64), y=(4, 64))
    for other in good:
        with pytest.raises((ValueError, TypeError)):
            lf.block_norm(**{k: on(1 if k == other else 0, s) for k, s in good.items()})
    good = dict(dy=(4, 64), x=(4, 64), h=(4, 64), post=(64,), pre=(64,), gate=(2, 64), dh=(4, 64), dx=(4, 64),
                dresidual=(4, 64), dpost=(64,), dpre=(64,), dgate=(2, 64))
    for other in good:
        with pytest.raises((ValueError, TypeError)):
            lf.block_norm_backward(**{k: on(1 if k == other else 0, s) for k, s in good.items()})
    assert not library.calls


# ---------------------------------------------------------------- gates
@pytest.mark.parametrize("shape,gate,rows", [
    ((6, 64), (64,), 1), ((6, 64), (1, 64), 1), ((6, 64), (3, 64), 3), ((6, 64), (6, 64), 6), ((2, 3, 64), (2, 64), 2),
    ((2, 3, 64), (2, 1, 64), 2), ((2, 3, 64), (1, 1, 64), 1), ((2, 3, 64), (2, 3, 64), 6), ((2, 3, 64), (6, 64), 6),
    ((2, 3, 5, 64), (2, 1, 1, 64), 2), ((2, 3, 5, 64), (2, 3, 1, 64), 6), ((64,), (64,), 1), ((64,), (1, 64), 1),
    ((2, 3, 64), (1, 3, 64), None), ((2, 3, 64), (4, 64), None), ((6, 64), (1, 1, 64), None), ((2, 3, 64), (2, 2, 64), None),
    ((6, 64), (0, 64), None), ((6, 64), (2, 32), None), ((6, 64), (), None), ((2, 3, 5, 64), (2, 1, 5, 64), None),
])
def test_rows_of_a_gate(monkeypatch, library, shape, gate, rows):  # noqa: F811
    """One row, rows for as many consecutive tokens each, or one that x's first dimensions
    choose: what would mean another order (a gate shared by a batch) is refused."""
    current(monkeypatch, 0)

    def call():
        return lf.block_norm(on(0, shape), on(0, shape), gate=on(0, gate), h=on(0, shape))
    if rows is None:
        with pytest.raises(ValueError, match="gate"):
            call()
        assert not library.calls
    else:
        call()
        assert library.calls[0][1][7] == rows


def test_binding_refusals(monkeypatch, library):  # noqa: F811
    current(monkeypatch, 0)
    x, w = on(0, (4, 64)), on(0, (64,))
    out = dict(h=on(0, (4, 64)), y=on(0, (4, 64)))
    ok = dict(x=x, residual=x, post=w, pre=w)
    for bad, error in ((dict(x=on(0, (4, 64), torch.float64)), TypeError), (dict(x=torch.zeros(4, 64)), TypeError),
                       (dict(residual=on(0, (4, 64), FP32)), TypeError), (dict(residual=on(0, (2, 64))), ValueError),
                       (dict(residual=None), TypeError), (dict(post=on(0, (64,), torch.float16)), TypeError),
                       (dict(post=on(0, (64,), FP32)), TypeError),              # two types of weights
                       (dict(pre=on(0, (32,))), ValueError), (dict(gate=on(0, (64,), torch.float16)), TypeError),
                       (dict(gate=0.5), TypeError), (dict(gate=on(0, (128,))[::2]), ValueError),
                       (dict(fp8=True), TypeError), (dict(scale=on(0, (4,), FP32)), ValueError), (dict(pre=None), ValueError),
                       (dict(pre=None, y=None, fp8=True), ValueError), (dict(h=on(0, (4, 32))), ValueError),
                       (dict(h=on(0, (64, 4)).t()), ValueError), (dict(x=on(0, (64, 4)).t()), ValueError)):
        with pytest.raises(error):
            lf.block_norm(**{**ok, **out, **bad})
    grad = dict(dy=x, x=x, h=x, post=w, pre=w, dx=on(0, (4, 64)), dresidual=on(0, (4, 64)), want_dparams=False)
    for bad, error in ((dict(dy=None), ValueError), (dict(h=None), ValueError), (dict(pre=None), ValueError),
                       (dict(dgate=on(0, (64,))), ValueError), (dict(dpre=on(0, (64,), FP32)), TypeError),
                       (dict(dy=on(0, (2, 64))), ValueError), (dict(dh=on(0, (4, 64), FP32)), TypeError),
                       (dict(x=on(0, (4, 128))[:, :64]), ValueError), (dict(gate=w, dgate=on(0, (1, 64))), ValueError)):
        with pytest.raises(error):
            lf.block_norm_backward(**{**grad, **bad})
    assert not library.calls
