"""gated_ffn, its e4m3 form and gated_ffn_backward against the 64-bit reference.

Bounds, element by element.  An fp32 accumulation of K products is off by at
most K 2^-23 times the sum of the products' magnitudes (2^-23: the tensor cores
may cut where an fp32 addition rounds).  With dg and du those bounds for the
projections, |act'| <= 1.13 for the three activations and FAST = 2^-18 for the
activation's own fp32 evaluation,
  |out - act(g) u| <= 1.13 |u| dg + |act(g)| du + 1.13 dg du + (half_step + FAST)(|act(g) u|).
In the backward pass the gradients of the projections are rounded to bf16 once
(half_step), then summed over 2F (dx) or M (dw) products, then rounded again.
"""
import math

import pytest
import torch

import ffn_reference as ref
import layout_folding_gb300 as lf

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
E4M3 = torch.float8_e4m3fn
HALF = ref.half_step(BF16)
TINY = 2.0 ** -126
FAST = 2.0 ** -18
ACC = 2.0 ** -23
ACTS = ["silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module", autouse=True)
def _device():
    lf.lib()
    torch.cuda.set_device(0)
    lf.check_device_error()
    yield
    lf.set_test_hooks(False, 0)
    torch.cuda.synchronize()
    lf.check_device_error()


def normal(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * std


def inputs(M, F, K, seed=1):
    return normal((M, K), seed).to(BF16), normal((2 * F, K), seed + 1, 1 / math.sqrt(K)).to(BF16)


def close(got, want, bound, what):
    got = got.detach().double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %g of its bound, first at %s" % (
        what, int(bad.sum()), bad.numel(), float(((got - want).abs() / bound).max()), bad.nonzero()[0].tolist())


def check_forward(x64, w64, name, out, gu=None):
    """x64, w64: what the operands stand for, in 64 bits on the CPU."""
    want, p = ref.gated(x64, w64, name)
    F, K = w64.shape[0] // 2, w64.shape[1]
    d = (K * ACC + 4 * ref.F32) * (x64.abs() @ w64.abs().t())
    g, u, dg, du = p[..., :F], p[..., F:], d[..., :F], d[..., F:]
    a = ref.act(g, name)
    bound = 1.13 * u.abs() * dg + a.abs() * du + 1.13 * dg * du + (HALF + FAST) * want.abs() + TINY
    close(out, want, bound, "out")
    if gu is not None:
        close(gu, p, d + HALF * p.abs() + TINY, "gu")


def check_backward(dout, x, w, gu, name, dx, dw):
    x64, w64, gu64 = x.double(), w.double(), gu.double().requires_grad_()
    (dgu,) = ref.grads(ref.gated_from_gu(gu64, name), (gu64,), dout.double())
    F2, M = w.shape[0], x.shape[0]
    for got, a, b, n, what in ((dx, dgu, w64, F2, "dx"), (dw, dgu.t(), x64, M, "dw")):
        if got is None:
            continue
        want, size = a @ b, a.abs() @ b.abs()
        # dgu: its own fp32 evaluation (its factors are of order one) and the rounding
        close(got, want, (HALF + 4 * FAST + n * ACC) * 1.02 * size + HALF * want.abs() + 1e-6 * b.abs().sum(0), what)
        # independent roundings: norm-wise well below one half step each for dgu and the result
        assert float((got.double().cpu() - want).norm()) <= HALF * float(want.norm()) * 1.1, what


SHAPES = [(1, 8, 8), (1, 1416, 520), (2, 128, 64), (3, 136, 72), (17, 264, 1032), (64, 520, 2048), (127, 8, 256),
          (128, 128, 128), (129, 392, 136), (200, 1416, 520), (256, 256, 64), (257, 248, 1000), (520, 1000, 264),
          (1030, 136, 192),
          # few tokens: whole K loops and K loops split over 2, 4 and 8 CTAs, one and two CTAs per SM
          (5, 40000, 256), (33, 9000, 520), (16, 4104, 1024), (65, 2056, 2048), (100, 20000, 136), (113, 520, 2048),
          # more tokens in groups: split in eight, four and two, ragged groups; and just not
          (130, 264, 1032), (333, 1408, 1040), (200, 4104, 4096), (1000, 520, 2048), (512, 512, 1024), (700, 2056, 512)]


@pytest.mark.parametrize("M,F,K", SHAPES)
def test_forward(M, F, K):
    x, w = inputs(M, F, K, M + F + K)
    xd, wd = x.to(DEV), w.to(DEV)
    for name in ACTS:
        out, gu = lf.gated_ffn(xd, wd, act=name, want_gu=True)
        only, none = lf.gated_ffn(xd, wd, act=name)
        lf.check_device_error()
        assert none is None and torch.equal(out, only)
        check_forward(x.double(), w.double(), name, out, gu)


def quantised(t):
    s = ref.row_scale(t.double()).float()
    return (t / s[:, None]).clamp(-448, 448).to(E4M3), s


@pytest.mark.parametrize("M,F,K", [(1, 8, 16), (1, 1416, 528), (3, 136, 80), (48, 520, 2048), (128, 128, 128),
                                   (129, 392, 144), (300, 1000, 272), (1030, 136, 192), (5, 20000, 256),
                                   (33, 4104, 1040), (65, 2056, 4096), (113, 520, 4096),
                                   (130, 264, 2064), (333, 1408, 2064), (150, 4104, 8208), (1000, 520, 4096)])
def test_forward_e4m3(M, F, K):
    x, xs = quantised(normal((M, K), 5) * torch.exp(normal((M, 1), 6)))
    w, ws = quantised(normal((2 * F, K), 7, 1 / math.sqrt(K)))
    for name in ACTS:
        out, gu = lf.gated_ffn(x.to(DEV), w.to(DEV), act=name, x_scale=xs.to(DEV), w_scale=ws.to(DEV))
        lf.check_device_error()
        assert gu is None
        check_forward(x.double() * xs.double()[:, None], w.double() * ws.double()[:, None], name, out)


# Pair tiles of 128, 112, 96, 80 and 64 columns (with 76 pairs: the widest of them that gives
# one wave), two waves of 96 and of 112, full and clipped last tiles
WIDTHS = [(1000, 2432, 72), (1000, 2120, 72), (1000, 1800, 72), (1000, 1512, 72), (1000, 1208, 72), (1024, 2128, 128),
          (257, 6912, 136), (520, 5544, 200), (140, 6160, 80), (4096, 1408, 64)]


@pytest.mark.parametrize("M,F,K", WIDTHS)
def test_forward_tile_widths(M, F, K):
    x, w = inputs(M, F, K, M + F + K)
    xd, wd = x.to(DEV), w.to(DEV)
    out, gu = lf.gated_ffn(xd, wd, want_gu=True)
    only, _ = lf.gated_ffn(xd, wd)
    assert torch.equal(out, only)
    check_forward(x.double(), w.double(), "silu", out, gu)
    x, xs = quantised(normal((M, 2 * K), 5))
    w, ws = quantised(normal((2 * F, 2 * K), 7, 1 / math.sqrt(K)))
    out, _ = lf.gated_ffn(x.to(DEV), w.to(DEV), act="gelu", x_scale=xs.to(DEV), w_scale=ws.to(DEV))
    lf.check_device_error()
    check_forward(x.double() * xs.double()[:, None], w.double() * ws.double()[:, None], "gelu", out)


@pytest.mark.parametrize("M,F,K", [(130, 264, 2056), (333, 1408, 2056), (200, 4104, 6152), (1000, 136, 4096)])
def test_forward_groups_of_tokens(M, F, K):
    """More than 128 tokens with long K loops: groups split in eight, four and two."""
    x, w = inputs(M, F, K, M + F + K)
    out, gu = lf.gated_ffn(x.to(DEV), w.to(DEV), want_gu=True)
    check_forward(x.double(), w.double(), "silu", out, gu)
    x, xs = quantised(normal((M, 2 * K), 5))
    w, ws = quantised(normal((2 * F, 2 * K), 7, 1 / math.sqrt(K)))
    out, _ = lf.gated_ffn(x.to(DEV), w.to(DEV), act="gelu_tanh", x_scale=xs.to(DEV), w_scale=ws.to(DEV))
    lf.check_device_error()
    check_forward(x.double() * xs.double()[:, None], w.double() * ws.double()[:, None], "gelu_tanh", out)


@pytest.mark.parametrize("M,F,K", [(1, 520, 72), (15, 136, 200), (33, 20000, 200), (64, 520, 1016), (64, 520, 1032),
                                   (90, 12000, 136), (112, 12000, 136), (128, 136, 2056), (128, 1000, 2000),
                                   (300, 1408, 2760)])
def test_forward_on_both_sides_of_the_choice(M, F, K):
    """Few tokens with short and long K loops, few and many tiles."""
    x, w = inputs(M, F, K, M + F + K)
    out, gu = lf.gated_ffn(x.to(DEV), w.to(DEV), want_gu=True)
    check_forward(x.double(), w.double(), "silu", out, gu)
    x, xs = quantised(normal((M, 2 * K), 5))
    w, ws = quantised(normal((2 * F, 2 * K), 7, 1 / math.sqrt(K)))
    out, _ = lf.gated_ffn(x.to(DEV), w.to(DEV), act="gelu_tanh", x_scale=xs.to(DEV), w_scale=ws.to(DEV))
    lf.check_device_error()
    check_forward(x.double() * xs.double()[:, None], w.double() * ws.double()[:, None], "gelu_tanh", out)


@pytest.mark.parametrize("M,F,K", [(1000, 2120, 72), (1000, 1512, 72)])
def test_narrow_tiles_stay_inside_their_buffers(M, F, K):
    """Two epilogue halves that overlap: nothing outside the output, nothing left out."""
    x, w = inputs(M, F, K)
    buf = torch.full((M * F + 8192,), 7.0, dtype=BF16, device=DEV)
    out = buf[4096:4096 + M * F].view(M, F)
    lf.gated_ffn(x.to(DEV), w.to(DEV), out=out)
    lf.check_device_error()
    assert bool((buf[:4096] == 7).all()) and bool((buf[4096 + M * F:] == 7).all())
    check_forward(x.double(), w.double(), "silu", out)


@pytest.mark.parametrize("M,F,K", SHAPES)
def test_backward(M, F, K):
    x, w = inputs(M, F, K, M + F + K)
    gu = ref.gated(x.double(), w.double(), "silu")[1].to(BF16)
    dout = normal((M, F), 9).to(BF16)
    dev = [t.to(DEV) for t in (dout, x, w, gu)]
    for name in ACTS:
        dx, dw = lf.gated_ffn_backward(*dev, act=name)
        lf.check_device_error()
        check_backward(dout, x, w, gu, name, dx, dw)
    only, none = lf.gated_ffn_backward(*dev, act=name, want_dw=False)
    assert none is None and torch.equal(only, dx)
    none, only = lf.gated_ffn_backward(*dev, act=name, want_dx=False)
    assert none is None and torch.equal(only, dw)
    dx2, dw2 = lf.gated_ffn_backward(*dev, act=name, dgu=dev[3])     # over gu
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_activations_far_from_zero():
    """g over the whole range that bf16 models reach, products with u = 1 exactly:
    x = (g, 1), one row of w selects each."""
    vals = torch.cat([torch.linspace(-120, 120, 481), torch.tensor([-3e4, 3e4, -1e-3, 1e-3, -0.0, 88.5, -88.5])]).to(BF16)
    M, K, F = vals.numel(), 8, 8
    x = torch.zeros(M, K)
    x[:, 0], x[:, 1] = vals.float(), 1.0
    w = torch.zeros(2 * F, K)
    w[:F, 0] = 1.0
    w[F:, 1] = 1.0
    x, w = x.to(BF16), w.to(BF16)
    dout = torch.ones(M, F).to(BF16)
    for name in ACTS:
        out, gu = lf.gated_ffn(x.to(DEV), w.to(DEV), act=name, want_gu=True)
        want = ref.act(vals.double(), name)[:, None].expand(M, F)
        # the far tails of the activations are below 2^-20 and may flush to zero there
        close(out, want, (HALF + 64 * FAST) * want.abs() + 2.0 ** -20, name)
        assert torch.equal(gu[:, :F].cpu(), vals[:, None].expand(M, F))
        dx, _ = lf.gated_ffn_backward(dout.to(DEV), x.to(DEV), w.to(DEV), gu, act=name)
        v = vals.double().requires_grad_()
        (slope,) = ref.grads(ref.act(v, name).sum(), (v,), None)
        ok = slope.isfinite()
        close(dx[:, 0][ok.to(DEV)], 8 * slope[ok], 8 * ((2 * HALF + 64 * FAST) * slope[ok].abs() + 2.0 ** -16), name + " slope")


def test_nan_and_infinity_stay_in_their_rows():
    M, F, K = 300, 136, 264
    x, w = inputs(M, F, K)
    x[5, 7] = float("nan")
    x[260, 0] = float("inf")
    out, gu = lf.gated_ffn(x.to(DEV), w.to(DEV), want_gu=True)
    fine = [i for i in range(M) if i not in (5, 260)]
    check_forward(x[fine].double(), w.double(), "silu", out[fine], gu[fine])
    assert torch.isnan(out[5]).all() and torch.isnan(gu[5]).all()
    assert not torch.isfinite(gu[260]).any()


def test_leading_dimensions_and_given_outputs():
    x, w = inputs(6 * 50, 72, 136)
    x3 = x.view(6, 50, 136).to(DEV)
    out = torch.empty(6, 50, 72, dtype=BF16, device=DEV)
    gu = torch.empty(6, 50, 144, dtype=BF16, device=DEV)
    a, b = lf.gated_ffn(x3, w.to(DEV), out=out, gu=gu)
    assert a is out and b is gu
    check_forward(x.double(), w.double(), "silu", out.view(300, 72), gu.view(300, 144))
    dx, dw = lf.gated_ffn_backward(out, x3, w.to(DEV), gu)
    assert dx.shape == x3.shape
    check_backward(out.cpu().view(300, 72), x, w, gu.cpu().view(300, 144), "silu", dx.view(300, 136), dw)


@pytest.mark.parametrize("M,F,K", [(1, 8, 8), (3, 136, 72), (45, 392, 520), (129, 8, 64), (300, 136, 264)])
def test_outputs_stay_inside_their_buffers(M, F, K):
    G = 4096
    x, w = inputs(M, F, K)
    xd, wd = x.to(DEV), w.to(DEV)

    def guarded(*shape):
        n = math.prod(shape)
        b = torch.full((n + 2 * G,), 7.0, dtype=BF16, device=DEV)
        return b, b[G:G + n].view(shape), n
    bufs = [guarded(M, F), guarded(M, 2 * F), guarded(M, 2 * F), guarded(M, K), guarded(2 * F, K)]
    out, gu, dgu, dx, dw = (b[1] for b in bufs)
    lf.gated_ffn(xd, wd, out=out, gu=gu)
    lf.gated_ffn_backward(out, xd, wd, gu, dgu=dgu, dx=dx, dw=dw)
    torch.cuda.synchronize()
    lf.check_device_error()
    check_forward(x.double(), w.double(), "silu", out, gu)
    check_backward(out.cpu(), x, w, gu.cpu(), "silu", dx, dw)
    if K % 16 == 0:
        q, s = quantised(x.float())
        qw, sw = quantised(w.float())
        b8 = guarded(M, F)
        bufs.append(b8)
        lf.gated_ffn(q.to(DEV), qw.to(DEV), x_scale=s.to(DEV), w_scale=sw.to(DEV), out=b8[1])
        check_forward(q.double() * s.double()[:, None], qw.double() * sw.double()[:, None], "silu", b8[1])
    for b, _, n in bufs:
        assert bool((b[:G] == 7.0).all()) and bool((b[G + n:] == 7.0).all())


def test_refusals():
    x, w = (t.to(DEV) for t in inputs(4, 16, 32))
    one = torch.ones(4, device=DEV)
    for bad in (dict(act="relu"), dict(act=None), dict(x_scale=one), dict(w_scale=one)):
        with pytest.raises((ValueError, TypeError)):
            lf.gated_ffn(x, w, **bad)
    with pytest.raises(TypeError):
        lf.gated_ffn(x.half(), w.half())
    with pytest.raises(ValueError):
        lf.gated_ffn(x, w[:, :16].contiguous())
    with pytest.raises(ValueError):
        lf.gated_ffn(x, w[:31])
    with pytest.raises(ValueError):
        lf.gated_ffn(x, w, out=torch.empty(4, 32, dtype=BF16, device=DEV))
    with pytest.raises(lf.LayoutFoldError) as info:
        lf.gated_ffn(x, w[:28].contiguous())          # F = 14
    assert info.value.status == 3
    q, qw = x.to(E4M3), w.to(E4M3)
    sw = torch.ones(32, device=DEV)
    with pytest.raises(ValueError):
        lf.gated_ffn(q, qw, x_scale=one, w_scale=sw, want_gu=True)
    with pytest.raises(ValueError):
        lf.gated_ffn(q, qw, x_scale=one[:3], w_scale=sw)
    with pytest.raises(TypeError):
        lf.gated_ffn(x, w, x_scale=one, w_scale=sw)
    with pytest.raises(TypeError):
        lf.gated_ffn(q, qw, x_scale=one.half(), w_scale=sw)
    with pytest.raises(ValueError):
        lf.gated_ffn_backward(x, x, w, x)


def test_no_rows():
    x, w = (t.to(DEV) for t in inputs(4, 16, 32))
    out, gu = lf.gated_ffn(x[:0], w, want_gu=True)
    assert out.shape == (0, 16) and gu.shape == (0, 32)
    dx, dw = lf.gated_ffn_backward(out, x[:0], w, gu)
    assert dx.shape == (0, 32) and not dw.any()


def test_on_side_streams_and_captured():
    M, F, K = 150, 264, 520
    x, w = inputs(M, F, K)
    xd, wd = x.to(DEV), w.to(DEV)
    dout = normal((M, F), 3).to(BF16).to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, gu = lf.gated_ffn(xd, wd, want_gu=True, stream=side)
    dx, dw = lf.gated_ffn_backward(dout, xd, wd, gu, stream=side)
    side.synchronize()
    check_forward(x.double(), w.double(), "silu", out, gu)
    check_backward(dout.cpu(), x, w, gu.cpu(), "silu", dx, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out, gu = lf.gated_ffn(xd, wd, want_gu=True)
            dx, dw = lf.gated_ffn_backward(dout, xd, wd, gu)
    for seed in (11, 12):
        x = normal((M, K), seed).to(BF16)
        xd.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        lf.check_device_error()
        check_forward(x.double(), w.double(), "silu", out, gu)
        check_backward(dout.cpu(), x, w, gu.cpu(), "silu", dx, dw)


def test_new_tensors_of_a_side_stream():
    """They are not memory that work of the current stream may still read."""
    M, F, K = 1024, 2048, 1024
    x, w = (t.to(DEV) for t in inputs(M, F, K))
    out, gu = lf.gated_ffn(x, w, want_gu=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for call, like in ((lambda: lf.gated_ffn(x, w, stream=side)[0], out),
                       (lambda: lf.gated_ffn_backward(out, x, w, gu, stream=side)[1], w)):
        freed = torch.empty_like(like)
        at = freed.data_ptr()
        del freed
        got = call()
        assert got.data_ptr() != at
        torch.cuda.synchronize()
        lf.check_device_error()


def test_repeatable():
    x, w = (t.to(DEV) for t in inputs(700, 392, 1032))
    dout = normal((700, 392), 3).to(BF16).to(DEV)
    out, gu = lf.gated_ffn(x, w, want_gu=True)
    first = (out, gu, *lf.gated_ffn_backward(dout, x, w, gu))
    for _ in range(3):
        out, gu = lf.gated_ffn(x, w, want_gu=True)
        for a, b in zip(first, (out, gu, *lf.gated_ffn_backward(dout, x, w, gu))):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [4, 300])
def test_stalled_wait_times_out_and_context_survives(M):
    x, w = inputs(M, 264, 520)
    xd, wd = x.to(DEV), w.to(DEV)
    lf.check_device_error()
    lf.set_test_hooks(True, 200_000_000)      # the first CTA never loads its first stage; 200 ms per wait
    try:
        lf.gated_ffn(xd, wd)
        with pytest.raises(lf.LayoutFoldError) as info:
            lf.check_device_error()
        assert info.value.status == 6 and lf.last_device_wait_code() in lf.WAIT_CODES
    finally:
        lf.set_test_hooks(False, 0)
    out, _ = lf.gated_ffn(xd, wd)
    lf.check_device_error()
    check_forward(x.double(), w.double(), "silu", out)


def test_block_training_and_generation():
    """The operators as a block uses them: norm, gated projections, down
    projection; the gradient of the whole against 64-bit autograd, norm-wise
    (each of the chain's five bf16 roundings is at most HALF of its value)."""
    M, D, F = 70, 136, 264
    x, res, w = normal((M, D), 1).to(BF16), normal((M, D), 2, 2.0).to(BF16), inputs(M, F, D, 3)[1]
    wn, wd = (1 + normal((D,), 5, 0.2)).to(BF16), normal((D, F), 6, 1 / math.sqrt(F)).to(BF16)
    dy = normal((M, D), 7).to(BF16)
    X, RES, W, WN, WD, DY = (t.to(DEV) for t in (x, res, w, wn, wd, dy))
    y, h, _ = lf.add_rms_norm(X, WN, residual=RES, eps=1e-6)
    a, gu = lf.gated_ffn(y, W, want_gu=True)
    out = lf.gemm_nt(a, WD)
    da = lf.gemm_layout(DY, WD, w_mn=True)
    dwd = lf.gemm_layout(DY, a, x_mn=True, w_mn=True)
    dyn, dw = lf.gated_ffn_backward(da, y, W, gu)
    dx, dwn = lf.add_rms_norm_backward(dyn, h, WN, dh=DY, eps=1e-6)
    lf.check_device_error()
    h64 = h.double().cpu().requires_grad_()
    p64 = [t.double().requires_grad_() for t in (wn, w, wd)]
    yn = ref.rms_norm(h64, p64[0], 1e-6)
    o64 = ref.gated(yn, p64[1], "silu")[0] @ p64[2].t()
    want = ref.grads(o64 + h64, (h64, *p64), dy.double())
    for got, ref64, what in ((out, o64, "out"), (dx, want[0], "dx"), (dwn, want[1], "dwn"), (dw, want[2], "dw"),
                             (dwd, want[3], "dwd")):
        err = float((got.double().cpu() - ref64.detach()).norm()) / float(ref64.detach().norm())
        assert err <= 5 * HALF, (what, err)
    # generation: one token, e4m3
    q, h1, s = lf.add_rms_norm(X[:1], WN, residual=RES[:1], fp8=True)
    if D % 16 == 0:
        qw, sw = quantised(w.float())
        lf.gated_ffn(q, qw.to(DEV), x_scale=s, w_scale=sw.to(DEV))


@pytest.mark.parametrize("M,F,K", [(300, 264, 520), (33, 2056, 264)])
def test_stalled_wait_in_the_gradient_times_out(M, F, K):
    x, w = inputs(M, F, K)
    gu = ref.gated(x.double(), w.double(), "silu")[1].to(BF16)
    dout = normal((M, F), 9).to(BF16)
    dev = [t.to(DEV) for t in (dout, x, w, gu)]
    lf.check_device_error()
    lf.set_test_hooks(True, 200_000_000)
    try:
        lf.gated_ffn_backward(*dev)
        with pytest.raises(lf.LayoutFoldError) as info:
            lf.check_device_error()
        assert info.value.status == 6 and lf.last_device_wait_code() in lf.WAIT_CODES
    finally:
        lf.set_test_hooks(False, 0)
    dx, dw = lf.gated_ffn_backward(*dev)
    lf.check_device_error()
    check_backward(dout, x, w, gu, "silu", dx, dw)


def test_tokens_and_sums_of_every_size():
    """Sizes around the tile, split and stage borders of every kernel, forward and
    backward, norm-wise (the element bounds are test_forward's and test_backward's):
    at most HALF for an output rounded once, 1.1 HALF where the gradient of the
    projections was rounded as well."""
    for M in (1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 511, 513):
        for F, K in ((8, 16), (120, 64), (128, 136), (136, 1040), (1000, 128)):
            x, w = inputs(M, F, K, M + F + K)
            xd, wd = x.to(DEV), w.to(DEV)
            out, gu = lf.gated_ffn(xd, wd, want_gu=True)
            want, p = ref.gated(x.double(), w.double(), "silu")
            for a, b in ((out, want), (gu, p)):
                assert float((a.double().cpu() - b).norm()) <= HALF * float(b.norm()), (M, F, K)
            dout = normal((M, F), M).to(BF16)
            dx, dw = lf.gated_ffn_backward(dout.to(DEV), xd, wd, gu)
            g64 = gu.double().cpu().requires_grad_()
            (dgu,) = ref.grads(ref.gated_from_gu(g64, "silu"), (g64,), dout.double())
            for a, b in ((dx, dgu @ w.double()), (dw, dgu.t() @ x.double())):
                assert float((a.double().cpu() - b).norm()) <= 1.1 * HALF * float(b.norm()), (M, F, K)
    lf.check_device_error()


def test_example_block_learns():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ffn_block.py")
    spec = importlib.util.spec_from_file_location("ffn_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, off = mod.main(["--tokens", "200", "--hidden", "256", "--ffn", "520", "--steps", "12"])
    assert losses[-1] < 0.7 * losses[0]
    # e4m3 activations and weights: each product is off by two roundings of at most
    # 2^-4, of random sign, so the block's output by well under sqrt(3) 2^-4 (gate, up and
    # their product)
    assert off < 3 ** 0.5 * 2 ** -4


def test_offsets_past_32_bits():
    """gu and dgu of more than 2^31 elements (M 2F): rows at both ends and at the border,
    and the weight gradient of a block of columns."""
    M, F, K = 300_000, 4096, 64
    w = inputs(1, F, K)[1]
    g = torch.Generator(device=DEV).manual_seed(1)
    xd = torch.empty(M, K, dtype=BF16, device=DEV).normal_(generator=g)
    wd = w.to(DEV)
    border = 2 ** 31 // (2 * F)
    rows = torch.tensor([0, 255, border - 1, border, border + 1, M - 1], device=DEV)
    out, gu = lf.gated_ffn(xd, wd, want_gu=True)
    x = xd[rows].cpu()
    gus = gu[rows].cpu()
    check_forward(x.double(), w.double(), "silu", out[rows], gus)
    dx, dw = lf.gated_ffn_backward(out, xd, wd, gu, dgu=gu)
    outs = out[rows].cpu()
    check_backward(outs, x, w, gus, "silu", dx[rows], None)
    # dgu now lies in gu: the weight gradient of its last 64 columns
    want = gu[:, -64:].double().t() @ xd.double()
    assert float((dw[-64:].double() - want).norm()) <= HALF * float(want.norm())
    lf.check_device_error()
