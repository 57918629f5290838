"""linear, its e4m3 form and linear_backward against the 64-bit reference.

Bounds, element by element.  An fp32 accumulation of K products is off by at
most K 2^-23 times the sum of the products' magnitudes (2^-23: the tensor cores
may cut where an fp32 addition rounds); e4m3 operands add two scalings, the bias
one addition, each half a step.  With dz that bound for z, |act'| <= 1.13 for
the three activations and FAST = 2^-18 for an activation's own fp32 evaluation,
  |out - (act(z) + residual)| <= 1.13 dz + FAST |act(z)| + F32 |out| + HALF |out|.
In the backward pass the slope is evaluated in fp32 (off by at most 8 FAST in all:
slopes are of order one), dz is rounded to bf16 once, then summed over N (dx) or M
(dw) products, then rounded again.  dbias: unrounded dz, at most M / 16 + M / 64 + 20
additions one after another (a thread's rows, the 16 rows of threads, the blocks).
"""
import math

import pytest
import torch

import ffn_reference as ref
import layout_folding_gb300 as lf

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
E4M3 = torch.float8_e4m3fn
HALF, F32 = ref.half_step(BF16), ref.F32
TINY = 2.0 ** -126
FAST = 2.0 ** -18
ACC = 2.0 ** -23
ACTS = [None, "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module", autouse=True)
def _device():
    lf.lib()
    torch.cuda.set_device(0)
    lf.check_device_error()
    yield
    lf.set_test_hooks(False, 0)
    torch.cuda.synchronize()
    lf.check_device_error()


def normal(shape, seed, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def inputs(M, N, K, seed=1):
    """x, w, bias, residual"""
    return (normal((M, K), seed), normal((N, K), seed + 1, 1 / math.sqrt(K)), normal((N,), seed + 2, 0.5),
            normal((M, N), seed + 3, 2.0))


def quantised(t):
    s = ref.row_scale(t.double()).float()
    return (t.float() / s[:, None]).clamp(-448, 448).to(E4M3), s


def act(v, name):
    return v if name is None else ref.act(v, name)


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def close(got, want, bound, what):
    got = got.detach().double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %g of its bound, first at %s" % (
        what, int(bad.sum()), bad.numel(), float(((got - want).abs() / bound).max()), bad.nonzero()[0].tolist())


def check_forward(x64, w64, bias, res, name, out, pre=None):
    """x64, w64: what the operands stand for, in 64 bits on the CPU."""
    z = x64 @ w64.t()
    d = (w64.shape[1] * ACC + 4 * F32) * (x64.abs() @ w64.abs().t())
    if bias is not None:
        d = d + F32 * (z.abs() + bias.double().abs())
        z = z + bias.double()
    a = act(z, name)
    want = a if res is None else a + res.double()
    close(out, want, 1.13 * d + FAST * a.abs() + (HALF + F32) * want.abs() + TINY, "out")
    if pre is not None:
        close(pre, z, d + HALF * z.abs() + TINY, "pre")


def gradient(dout, pre, name):
    if name is None:
        return dout.double()
    z = pre.double().requires_grad_()
    return ref.grads(act(z, name), (z,), dout.double())[0]


def check_backward(dout, x, w, pre, name, dx, dw, db=None):
    dz = gradient(dout, pre, name)
    x64, w64 = x.double(), w.double()
    M, N = dz.shape
    slope = 0.0 if name is None else 8 * FAST
    once = 0.0 if name is None else HALF
    off = slope * dout.double().abs()  # of dz before its rounding
    for got, a, e, b, n, what in ((dx, dz, off, w64, N, "dx"), (dw, dz.t(), off.t(), x64, M, "dw")):
        if got is None:
            continue
        want, size = a @ b, a.abs() @ b.abs()
        close(got, want, (once + n * ACC) * 1.02 * size + 1.02 * (e @ b.abs()) + HALF * want.abs() + TINY, what)
        # independent roundings: norm-wise well below one half step each for dz and the result
        assert float((got.double().cpu() - want).norm()) <= HALF * float(want.norm()) * 1.1, what
    if db is not None:
        want = dz.sum(0)
        steps = M / 16 + M / 64 + 20
        close(db, want, off.sum(0) + steps * F32 * dz.abs().sum(0) + ref.half_step(db.dtype) * want.abs() + TINY, "dbias")


SHAPES = [(1, 8, 8), (1, 1416, 520), (2, 128, 64), (3, 136, 72), (17, 264, 1032), (64, 520, 2048), (127, 8, 256),
          (128, 128, 128), (129, 392, 136), (200, 1416, 520), (256, 256, 64), (257, 248, 1000), (520, 1000, 264),
          (1030, 136, 192), (33, 9000, 520), (16, 4104, 1024), (5, 40000, 256), (100, 2056, 2048), (333, 1408, 1040)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(M, N, K):
    x, w, b, res = inputs(M, N, K, M + N + K)
    xd, wd, bd, rd = dev(x, w, b, res)
    x64, w64 = x.double(), w.double()
    for name in ACTS:
        out, pre = lf.linear(xd, wd, bias=bd, act=name, residual=rd, want_pre=True)
        only, none = lf.linear(xd, wd, bias=bd, act=name, residual=rd)
        lf.check_device_error()
        assert none is None and torch.equal(out, only)
        check_forward(x64, w64, b, res, name, out, pre)
        out, _ = lf.linear(xd, wd, act=name)
        check_forward(x64, w64, None, None, name, out)
    b32 = normal((N,), 5, 0.5, FP32)
    out, _ = lf.linear(xd, wd, bias=b32.to(DEV), act="silu")
    check_forward(x64, w64, b32, None, "silu", out)
    out, _ = lf.linear(xd, wd, residual=rd)
    lf.check_device_error()
    check_forward(x64, w64, None, res, None, out)


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 1416, 528), (3, 136, 80), (48, 520, 2048), (128, 128, 128),
                                   (129, 392, 144), (300, 1000, 272), (1030, 136, 192), (5, 20000, 256),
                                   (33, 4104, 1040), (65, 2056, 4096), (333, 1408, 2064)])
def test_forward_e4m3(M, N, K):
    x, xs = quantised(normal((M, K), 5, dtype=FP32) * torch.exp(normal((M, 1), 6, dtype=FP32)))
    w, ws = quantised(normal((N, K), 7, 1 / math.sqrt(K), FP32))
    b, res = normal((N,), 8, 0.5), normal((M, N), 9, 2.0)
    xd, sd, wd, td, bd, rd = dev(x, xs, w, ws, b, res)
    x64, w64 = x.double() * xs.double()[:, None], w.double() * ws.double()[:, None]
    for name in ACTS:
        out, pre = lf.linear(xd, wd, bias=bd, act=name, residual=rd, x_scale=sd, w_scale=td)
        lf.check_device_error()
        assert pre is None
        check_forward(x64, w64, b, res, name, out)
    out, _ = lf.linear(xd, wd, bias=b.float().to(DEV), x_scale=sd, w_scale=td)
    check_forward(x64, w64, b, None, None, out)


# Tiles of 256, 192, 128 and 64 columns in one wave of 76 pairs and in two, full and clipped last tiles
WIDTHS = [(1000, 4864, 72), (1000, 3640, 72), (1000, 2424, 72), (1000, 1208, 72), (1024, 5120, 128), (257, 9736, 136),
          (520, 5544, 200), (140, 6160, 80), (4096, 1408, 64)]


@pytest.mark.parametrize("M,N,K", WIDTHS)
def test_forward_tile_widths(M, N, K):
    x, w, b, res = inputs(M, N, K, M + N + K)
    xd, wd, bd, rd = dev(x, w, b, res)
    out, pre = lf.linear(xd, wd, bias=bd, act="gelu", residual=rd, want_pre=True)
    only, _ = lf.linear(xd, wd, bias=bd, act="gelu", residual=rd)
    assert torch.equal(out, only)
    check_forward(x.double(), w.double(), b, res, "gelu", out, pre)
    x, xs = quantised(normal((M, 2 * K), 5))
    w, ws = quantised(normal((N, 2 * K), 7, 1 / math.sqrt(K)))
    xd, sd, wd, td = dev(x, xs, w, ws)
    out, _ = lf.linear(xd, wd, bias=bd, residual=rd, x_scale=sd, w_scale=td)
    lf.check_device_error()
    check_forward(x.double() * xs.double()[:, None], w.double() * ws.double()[:, None], b, res, None, out)


@pytest.mark.parametrize("M,N,K", [(256, 2048, 4096), (520, 1000, 8192), (300, 264, 8200), (140, 4104, 2056),
                                   (129, 520, 1032), (1000, 1032, 2056), (256, 4096, 1024), (260, 200, 4104)])
def test_forward_shared_sums(M, N, K):
    """Few tiles and long K loops: the pairs of a cluster (two to four, tiles of every width)
    share a tile's K blocks."""
    x, w, b, res = inputs(M, N, K, M + N + K)
    xd, wd, bd, rd = dev(x, w, b, res)
    x64, w64 = x.double(), w.double()
    for name in ACTS:
        out, pre = lf.linear(xd, wd, bias=bd, act=name, residual=rd, want_pre=True)
        only, _ = lf.linear(xd, wd, bias=bd, act=name, residual=rd)
        assert torch.equal(out, only)
        check_forward(x64, w64, b, res, name, out, pre)
    out, _ = lf.linear(xd, wd)
    check_forward(x64, w64, None, None, None, out)
    over = rd.clone()
    lf.linear(xd, wd, bias=bd, act=name, residual=over, out=over)
    assert torch.equal(over, only)
    if K % 16 == 0:
        x, xs = quantised(x)
        w, ws = quantised(w)
        xd, sd, wd, td = dev(x, xs, w, ws)
        out, _ = lf.linear(xd, wd, bias=bd, act="silu", residual=rd, x_scale=sd, w_scale=td)
        check_forward(x.double() * xs.double()[:, None], w.double() * ws.double()[:, None], b, res, "silu", out)
    lf.check_device_error()


@pytest.mark.parametrize("M,N,K", [(1, 264, 136), (70, 1000, 520), (130, 264, 1032), (1000, 2424, 72), (2000, 5120, 64)])
def test_residual_updated_in_place(M, N, K):
    """out over the residual, several tiles for each pair among the shapes."""
    x, w, b, res = inputs(M, N, K, 3)
    xd, wd, bd, rd = dev(x, w, b, res)
    want, _ = lf.linear(xd, wd, bias=bd, act="silu", residual=rd)
    out, pre = lf.linear(xd, wd, bias=bd, act="silu", residual=rd, out=rd, want_pre=True)
    lf.check_device_error()
    assert out is rd and torch.equal(out, want)
    check_forward(x.double(), w.double(), b, res, "silu", out, pre)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_backward(M, N, K):
    x, w, b, _ = inputs(M, N, K, M + N + K)
    pre = (x.double() @ w.double().t() + b.double()).to(BF16)
    dout = normal((M, N), 9)
    dd, xd, wd, pd, bd = dev(dout, x, w, pre, b)
    for name in ACTS:
        p = None if name is None else pd
        dx, dw, db = lf.linear_backward(dd, xd, wd, pre=p, act=name, bias=bd)
        lf.check_device_error()
        assert db.dtype == BF16
        check_backward(dout, x, w, pre, name, dx, dw, db)
        _, _, db32 = lf.linear_backward(dd, xd, wd, pre=p, act=name, bias=bd.float(), want_dx=False, want_dw=False)
        assert db32.dtype == FP32 and torch.equal(db32.bfloat16(), db)
        check_backward(dout, x, w, pre, name, None, None, db32)
    only, none, nob = lf.linear_backward(dd, xd, wd, pre=pd, act=name, want_dw=False)
    assert none is None and nob is None and torch.equal(only, dx)
    none, only, _ = lf.linear_backward(dd, xd, wd, pre=pd, act=name, want_dx=False)
    assert none is None and torch.equal(only, dw)
    over = pd.clone()
    for dz in (over, dd):     # over pre, then over dout
        dx2, dw2, db2 = lf.linear_backward(dd, xd, wd, pre=pd if dz is dd else over, act=name, bias=bd, dz=dz)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("name", ACTS)
def test_gradient_against_differences(name):
    """Directional derivative of L = sum(dout out) in 64 bits by central differences:
    truncation and rounding are below 1e-8, so the kernels' own bound (two bf16
    roundings, of random sign over N or M products) is what is left: 4 HALF of the
    root sum of squares of the terms."""
    M, N, K = 40, 72, 56
    x, w, b, _ = inputs(M, N, K, 31)
    pre = (x.double() @ w.double().t() + b.double()).to(BF16)
    dout = normal((M, N), 9)
    dd, xd, wd, pd, bd = dev(dout, x, w, pre, b)
    got = lf.linear_backward(dd, xd, wd, pre=None if name is None else pd, act=name, bias=bd.float())

    def loss(x64, w64, b64):
        # (around the kept z, which the gradient is taken at)
        z = pre.double() + (x64 - x.double()) @ w.double().t() + x.double() @ (w64 - w.double()).t() + (b64 - b.double())
        return float((act(z, name) * dout.double()).sum())
    args = [x.double(), w.double(), b.double()]
    for i, g in enumerate(got):
        v = normal(args[i].shape, 40 + i, dtype=FP32).double()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * v, args[i] - 1e-5 * v
        want = (loss(*up) - loss(*down)) / 2e-5
        terms = g.double().cpu() * v
        assert abs(float(terms.sum()) - want) <= 4 * HALF * float(terms.norm()) + 1e-6


def test_activations_far_from_zero():
    """z over the whole range that bf16 models reach: x selects one column of w."""
    vals = torch.cat([torch.linspace(-120, 120, 481), torch.tensor([-3e4, 3e4, -1e-3, 1e-3, -0.0, 88.5, -88.5])]).to(BF16)
    M, K, N = vals.numel(), 8, 8
    x = torch.zeros(M, K, dtype=BF16)
    x[:, 0] = vals
    w = torch.zeros(N, K, dtype=BF16)
    w[:, 0] = 1.0
    dout = torch.ones(M, N, dtype=BF16)
    for name in ACTS:
        out, pre = lf.linear(x.to(DEV), w.to(DEV), act=name, want_pre=True)
        want = act(vals.double(), name)[:, None].expand(M, N)
        # the far tails of the activations are below 2^-20 and may flush to zero there
        close(out, want, (HALF + 64 * FAST) * want.abs() + 2.0 ** -20, str(name))
        assert torch.equal(pre.cpu(), vals[:, None].expand(M, N))
        dx, _, _ = lf.linear_backward(*dev(dout, x, w), pre=None if name is None else pre, act=name)
        slope = gradient(dout, pre.cpu(), name)[:, 0]
        ok = slope.isfinite()
        close(dx[:, 0][ok.to(DEV)], 8 * slope[ok], 8 * ((2 * HALF + 64 * FAST) * slope[ok].abs() + 2.0 ** -16),
              "%s slope" % name)


@pytest.mark.parametrize("M,rows", [(300, (5, 260)), (7, (2, 6))])
def test_nan_and_infinity_stay_in_their_rows(M, rows):
    N, K = 136, 264
    x, w, b, res = inputs(M, N, K)
    x[rows[0], 7] = float("nan")
    res[rows[1], 3] = float("inf")
    out, pre = lf.linear(*dev(x, w), bias=b.to(DEV), act="silu", residual=res.to(DEV), want_pre=True)
    fine = [i for i in range(M) if i not in rows]
    check_forward(x[fine].double(), w.double(), b, res[fine], "silu", out[fine], pre[fine])
    assert torch.isnan(out[rows[0]]).all() and torch.isnan(pre[rows[0]]).all()
    assert out[rows[1], 3] == float("inf") and int((~torch.isfinite(out[rows[1]])).sum()) == 1


def test_leading_dimensions_and_given_outputs():
    x, w, b, res = inputs(6 * 50, 72, 136)
    xd, wd, bd, rd = dev(x.view(6, 50, 136), w, b, res.view(6, 50, 72))
    out, pre = (torch.empty(6, 50, 72, dtype=BF16, device=DEV) for _ in range(2))
    a, p = lf.linear(xd, wd, bias=bd, act="gelu", residual=rd, out=out, pre=pre)
    assert a is out and p is pre
    check_forward(x.double(), w.double(), b, res, "gelu", out.view(300, 72), pre.view(300, 72))
    db = torch.empty(72, device=DEV)
    dx, dw, db2 = lf.linear_backward(out, xd, wd, pre=pre, act="gelu", dbias=db)
    assert dx.shape == xd.shape and db2 is db
    check_backward(out.cpu().view(300, 72), x, w, pre.cpu().view(300, 72), "gelu", dx.view(300, 136), dw, db)
    row, _ = lf.linear(xd[0, 0], wd, bias=bd)
    assert row.shape == (72,)
    check_forward(x[:1].double(), w.double(), b, None, None, row[None])


@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (3, 136, 72), (45, 392, 520), (129, 8, 64), (300, 136, 264), (1000, 2424, 72)])
def test_outputs_stay_inside_their_buffers(M, N, K):
    G = 4096
    x, w, b, res = inputs(M, N, K)
    xd, wd, bd, rd = dev(x, w, b, res)

    def guarded(*shape):
        n = math.prod(shape)
        buf = torch.full((n + 2 * G,), 7.0, dtype=BF16, device=DEV)
        return buf, buf[G:G + n].view(shape), n
    bufs = [guarded(M, N), guarded(M, N), guarded(M, N), guarded(M, K), guarded(N, K), guarded(N), guarded(M, N)]
    out, pre, dz, dx, dw, db, out8 = (t[1] for t in bufs)
    lf.linear(xd, wd, bias=bd, act="silu", residual=rd, out=out, pre=pre)
    lf.linear_backward(out, xd, wd, pre=pre, act="silu", dz=dz, dx=dx, dw=dw, dbias=db)
    torch.cuda.synchronize()
    lf.check_device_error()
    check_forward(x.double(), w.double(), b, res, "silu", out, pre)
    check_backward(out.cpu(), x, w, pre.cpu(), "silu", dx, dw, db)
    if K % 16 == 0:
        q, s = quantised(x)
        qw, sw = quantised(w)
        lf.linear(q.to(DEV), qw.to(DEV), bias=bd, x_scale=s.to(DEV), w_scale=sw.to(DEV), out=out8)
        check_forward(q.double() * s.double()[:, None], qw.double() * sw.double()[:, None], b, None, None, out8)
    for buf, _, n in bufs:
        assert bool((buf[:G] == 7.0).all()) and bool((buf[G + n:] == 7.0).all())


def test_refusals():
    x, w, b, res = dev(*inputs(4, 16, 32))
    one = torch.ones(4, device=DEV)
    for bad in (dict(act="relu"), dict(act=0), dict(x_scale=one), dict(w_scale=one), dict(bias=b.half()),
                dict(bias=b[:8]), dict(residual=res[:3]), dict(residual=res.float()), dict(residual=res.t()),
                dict(out=torch.empty(4, 32, dtype=BF16, device=DEV)), dict(bias=b.cpu()), dict(residual=res.cpu())):
        with pytest.raises((ValueError, TypeError)):
            lf.linear(x, w, **bad)
    with pytest.raises(TypeError):
        lf.linear(x.half(), w.half())
    with pytest.raises(ValueError):
        lf.linear(x, w[:, :16].contiguous())
    with pytest.raises(ValueError):
        lf.linear(x[:, ::2], w[:, :16].contiguous())
    for bad in (dict(w=w[:12].contiguous()), dict(x=x[:, :28].contiguous(), w=w[:, :28].contiguous()), dict(out=res, pre=res),
                dict(residual=res, pre=res)):
        with pytest.raises(lf.LayoutFoldError):
            lf.linear(**{**dict(x=x, w=w), **bad})
    q, qw, sw = x.to(E4M3), w.to(E4M3), torch.ones(16, device=DEV)
    with pytest.raises(ValueError):
        lf.linear(q, qw, x_scale=one, w_scale=sw, want_pre=True)
    with pytest.raises(ValueError):
        lf.linear(q, qw, x_scale=one[:3], w_scale=sw)
    with pytest.raises(TypeError):
        lf.linear(x, w, x_scale=one, w_scale=sw)
    with pytest.raises(ValueError):
        lf.linear_backward(res, x, w, act="silu")            # no pre
    with pytest.raises(ValueError):
        lf.linear_backward(res, x, w, dz=res)                # nothing to write there
    with pytest.raises(ValueError):
        lf.linear_backward(x, x, w)
    with pytest.raises(TypeError):
        lf.linear_backward(res, x, w, bias=b, dbias=b.float())


def test_no_rows():
    x, w, b, res = dev(*inputs(4, 16, 32))
    out, pre = lf.linear(x[:0], w, bias=b, residual=res[:0], want_pre=True)
    assert out.shape == (0, 16) and pre.shape == (0, 16)
    dx, dw, db = lf.linear_backward(out, x[:0], w, pre=pre, act="silu", bias=b)
    assert dx.shape == (0, 32) and not dw.any() and not db.any()


@pytest.mark.parametrize("M", [5, 150])
def test_on_side_streams_and_captured(M):
    N, K = 264, 520
    x, w, b, res = inputs(M, N, K)
    dout = normal((M, N), 3)
    xd, wd, bd, rd, dd = dev(x, w, b, res, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, pre = lf.linear(xd, wd, bias=bd, act="gelu", residual=rd, want_pre=True, stream=side)
    dx, dw, db = lf.linear_backward(dd, xd, wd, pre=pre, act="gelu", bias=bd, stream=side)
    side.synchronize()
    check_forward(x.double(), w.double(), b, res, "gelu", out, pre)
    check_backward(dout, x, w, pre.cpu(), "gelu", dx, dw, db)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out, pre = lf.linear(xd, wd, bias=bd, act="gelu", residual=rd, want_pre=True)
            dx, dw, db = lf.linear_backward(dd, xd, wd, pre=pre, act="gelu", bias=bd)
    for seed in (11, 12):
        x = normal((M, K), seed)
        xd.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        lf.check_device_error()
        check_forward(x.double(), w.double(), b, res, "gelu", out, pre)
        check_backward(dout, x, w, pre.cpu(), "gelu", dx, dw, db)


def test_new_tensors_of_a_side_stream():
    """They are not memory that work of the current stream may still read."""
    x, w, _, res = dev(*inputs(1024, 2048, 1024))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for call, like in ((lambda: lf.linear(x, w, stream=side)[0], res),
                       (lambda: lf.linear_backward(res, x, w, stream=side)[1], w)):
        freed = torch.empty_like(like)
        at = freed.data_ptr()
        del freed
        got = call()
        assert got.data_ptr() != at
        torch.cuda.synchronize()
        lf.check_device_error()


def test_repeatable_and_on_two_streams_at_once():
    x, w, b, res = dev(*inputs(700, 392, 1032))
    dout = normal((700, 392), 3).to(DEV)
    out, pre = lf.linear(x, w, bias=b, act="silu", residual=res, want_pre=True)
    first = (out, pre, *lf.linear_backward(dout, x, w, pre=pre, act="silu", bias=b))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        s = streams[i % 2]
        out, pre = lf.linear(x, w, bias=b, act="silu", residual=res, want_pre=True, stream=s)
        got.append((out, pre, *lf.linear_backward(dout, x, w, pre=pre, act="silu", bias=b, stream=s)))
    torch.cuda.synchronize()
    for again in got:
        for a, c in zip(first, again):
            assert torch.equal(a, c)


@pytest.mark.parametrize("M,K", [(4, 520), (300, 136), (300, 4104)])
def test_stalled_wait_times_out_and_context_survives(M, K):
    x, w, b, res = inputs(M, 264, K)
    xd, wd, bd, rd = dev(x, w, b, res)
    lf.check_device_error()
    for residual in (None, rd):
        lf.set_test_hooks(True, 200_000_000)      # the first CTA never loads its first stage; 200 ms per wait
        try:
            lf.linear(xd, wd, residual=residual)
            with pytest.raises(lf.LayoutFoldError) as info:
                lf.check_device_error()
            assert info.value.status == 6 and lf.last_device_wait_code() in lf.WAIT_CODES
        finally:
            lf.set_test_hooks(False, 0)
        out, _ = lf.linear(xd, wd, bias=bd, residual=rd)
        lf.check_device_error()
        check_forward(x.double(), w.double(), b, res, None, out)


def test_tokens_and_sums_of_every_size():
    """Sizes around the tile, split and stage borders of every kernel, forward and
    backward, norm-wise (the element bounds are test_forward's and test_backward's):
    at most HALF for an output rounded once, 1.1 HALF where dz was rounded as well."""
    for M in (1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 511, 513):
        for N, K in ((8, 16), (56, 64), (128, 136), (136, 1040), (1000, 128), (264, 2064)):
            x, w, b, res = inputs(M, N, K, M + N + K)
            xd, wd, bd, rd = dev(x, w, b, res)
            z = x.double() @ w.double().t() + b.double()
            out, pre = lf.linear(xd, wd, bias=bd, act="silu", residual=rd, want_pre=True)
            for a, c in ((out, act(z, "silu") + res.double()), (pre, z)):
                assert float((a.double().cpu() - c).norm()) <= HALF * float(c.norm()), (M, N, K)
            dout = normal((M, N), M)
            dx, dw, _ = lf.linear_backward(dout.to(DEV), xd, wd, pre=pre, act="silu")
            dz = gradient(dout, pre.cpu(), "silu")
            for a, c in ((dx, dz @ w.double()), (dw, dz.t() @ x.double())):
                assert float((a.double().cpu() - c).norm()) <= 1.1 * HALF * float(c.norm()), (M, N, K)
    lf.check_device_error()


def test_offsets_past_32_bits():
    """out, pre and dz of more than 2^31 elements: rows at both ends and at the border, the
    bias gradient and the weight gradient of the last columns."""
    M, N, K = 300_000, 8192, 64
    w = normal((N, K), 2, 1 / math.sqrt(K))
    b = normal((N,), 4, 0.5)
    g = torch.Generator(device=DEV).manual_seed(1)
    xd = torch.empty(M, K, dtype=BF16, device=DEV).normal_(generator=g)
    wd, bd = dev(w, b)
    border = 2 ** 31 // N
    rows = torch.tensor([0, 255, border - 1, border, border + 1, M - 1], device=DEV)
    out, pre = lf.linear(xd, wd, bias=bd, act="gelu_tanh", want_pre=True)
    x, outs, pres = xd[rows].cpu(), out[rows].cpu(), pre[rows].cpu()
    check_forward(x.double(), w.double(), b, None, "gelu_tanh", outs, pres)
    added, _ = lf.linear(xd, wd, residual=out)
    check_forward(x.double(), w.double(), None, outs, None, added[rows])
    del added
    dx, dw, db = lf.linear_backward(out, xd, wd, pre=pre, act="gelu_tanh", bias=bd.float(), dz=pre)
    check_backward(outs, x, w, pres, "gelu_tanh", dx[rows], None)
    # dz now lies in pre: the weight gradient of its last 64 columns, and the bias's (of dz
    # before its rounding, M roundings of random sign)
    tail = pre[:, -64:].double()
    want = tail.t() @ xd.double()
    assert float((dw[-64:].double() - want).norm()) <= HALF * float(want.norm())
    assert float((db[-64:].double() - tail.sum(0)).abs().max()) <= 8 * HALF * float(tail.norm(dim=0).max())
    lf.check_device_error()
