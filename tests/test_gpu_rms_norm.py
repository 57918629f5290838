"""add_rms_norm and add_rms_norm_backward against the 64-bit reference.

Bounds, element by element.  F32 = 2^-24 is half a step of fp32; a fp32 sum
whose terms pass through at most S additions one after another is off by at
most S F32 times the sum of the terms' magnitudes.
  r: the sum of squares (S <= 128: what one thread adds, then the block's tree,
     64 + 16 with room) gives half its error in r; rsqrt, the mean and the two
     products add a few F32.  R = 96 F32 covers all of f = h r w.
  y: R |f| plus the rounding to the type, half_step |f| (or half the spacing of
     the type's subnormals).
  e4m3: |y scale - f| <= (half_step + R + a few F32) |f| + scale 2^-10.
  dx = r g - h r^3 mean(g h) + dh: each term R of its own magnitude (the mean
     R of mean |g h|), plus the rounding.
  dweight: the rows' terms d h r are each R off; they are added M / blocks by one
     thread, then over the blocks.
"""
import numpy as np
import pytest
import torch

import ffn_reference as ref
import layout_folding_gb300 as lf

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
R = 96 * ref.F32
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _device():
    lf.lib()
    torch.cuda.set_device(0)
    lf.check_device_error()
    yield
    torch.cuda.synchronize()


def normal(shape, seed, std=1.0, dtype=BF16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def close(got, want, bound, what):
    got = got.detach().double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %g of its bound, first at %s" % (
        what, int(bad.sum()), bad.numel(), float(((got - want).abs() / bound).max()), bad.nonzero()[0].tolist())


def kept(x, res):
    return x if res is None else (x.float() + res.float()).to(x.dtype)


def check_forward(x, w, res, fp8, got):
    y, h, scale = got
    hk = kept(x, res)
    if res is None:
        assert h is None or h.shape == x.shape
    else:
        assert torch.equal(h.cpu().view(torch.int16 if h.element_size() == 2 else torch.int32),
                           hk.view(torch.int16 if hk.element_size() == 2 else torch.int32))  # one fp32 addition, one rounding
    f = ref.rms_norm(hk.double(), w.double(), EPS)
    if not fp8:
        assert scale is None and y.dtype == x.dtype and y.shape == x.shape
        close(y, f, (ref.half_step(y.dtype) + R) * f.abs() + ref.smallest(y.dtype), "y")
        return
    assert y.dtype == E4M3 and scale.dtype == FP32 and scale.shape == x.shape[:-1]
    s = ref.row_scale(f)
    close(scale, s, (R + 4 * ref.F32) * s, "scale")
    v = y.float().cpu().double() * scale.cpu().double()[..., None]
    close(v, f, (2.0 ** -4 + R + 8 * ref.F32) * f.abs() + (s * 2.0 ** -10 * 1.001)[..., None], "y scale")


def forward(x, w, res=None, fp8=False, **kw):
    dev = [None if t is None else t.to(DEV) for t in (x, w, res)]
    out = lf.add_rms_norm(dev[0], dev[1], residual=dev[2], eps=EPS, fp8=fp8, **kw)
    torch.cuda.synchronize()
    return out


SIZES = [(1, 1), (1, 5120), (2, 7), (3, 8), (5, 31), (4, 32), (7, 256), (9, 1000), (3, 1027), (5, 1530), (6, 4096),
         (2, 8192), (3, 8200), (2, 10001), (1, 16384), (1, 40000), (2, 65536), (1, 70000)]
TYPES = [(BF16, BF16), (BF16, FP32), (FP16, FP16), (FP16, FP32), (FP32, FP32)]
IDS = ["bf16", "bf16_w32", "fp16", "fp16_w32", "fp32"]


@pytest.mark.parametrize("M,D", SIZES)
@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=IDS)
def test_forward(M, D, dtype, wdtype):
    x, w = normal((M, D), M + D, 1.0, dtype), 1 + normal((D,), D, 0.2, wdtype)
    res = normal((M, D), 77 + D, 2.0, dtype)
    for r in (None, res):
        for fp8 in (False, True):
            check_forward(x, w, r, fp8, forward(x, w, r, fp8))


def test_many_rows_and_leading_dimensions():
    x, w = normal((3, 701, 264), 1), 1 + normal((264,), 2, 0.2)
    res = normal((3, 701, 264), 3, 2.0)
    check_forward(x, w, res, True, forward(x, w, res, True))
    check_forward(x, w, res, False, forward(x, w, res, False))


# enough rows for the persistent kernels: one warp per row and many groups of them,
# several warps, rows that leave room for one group only, rows too long for it
MANY = [(609, 8), (1000, 136), (2500, 264), (700, 1032), (1300, 2056), (640, 5120), (613, 12296), (610, 20000),
        # rows that are not a multiple of 16 bytes
        (700, 33), (611, 37), (900, 250), (1333, 1027), (777, 1530), (650, 5121), (609, 9999), (608, 12301),
        # the longest rows that fit, weights in shared memory or not; few phased rows
        (620, 16384), (609, 16383), (100, 1027), (153, 515), (303, 2050),
        (1, 5121), (4, 10303), (7, 1031), (9, 2047), (33, 13611)]


@pytest.mark.parametrize("M,D", MANY)
@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=IDS)
def test_many_rows(M, D, dtype, wdtype):
    x, w = normal((M, D), M + D, 1.0, dtype), 1 + normal((D,), D, 0.2, wdtype)
    res = normal((M, D), 77 + D, 2.0, dtype)
    check_forward(x, w, None, True, forward(x, w, None, True))
    check_forward(x, w, res, True, forward(x, w, res, True))
    check_forward(x, w, res, False, forward(x, w, res, False))
    check_backward(x, res, w, None, backward(x, res, w))
    check_backward(x, res, w, x, backward(x, res, w, x))
    lf.check_device_error()


def test_many_rows_of_wider_tensors_in_place_and_with_nan():
    M, D = 900, 1024
    wide, w = normal((M, 1040), 4), 1 + normal((D,), 6, 0.2)
    wide[17, 100] = float("nan")
    res = normal((M, D), 5, 2.0)
    rd = res.to(DEV)
    y, h, _ = lf.add_rms_norm(wide.to(DEV)[:, 8:8 + D], w.to(DEV), residual=rd, eps=EPS, h=rd)
    fine = [i for i in range(M) if i != 17]
    x = wide[:, 8:8 + D].contiguous()
    check_forward(x[fine], w, res[fine], False, (y[fine], h[fine], None))
    assert torch.isnan(y[17]).all()


def test_stalled_wait_times_out_and_context_survives():
    M, D = 1000, 1024
    x, w, res = normal((M, D), 1), 1 + normal((D,), 2, 0.2), normal((M, D), 3, 2.0)
    for call, check in ((lambda: forward(x, w, res), lambda out: check_forward(x, w, res, False, out)),
                        (lambda: backward(x, res, w), lambda out: check_backward(x, res, w, None, out))):
        lf.check_device_error()
        lf.set_test_hooks(True, 100_000_000)   # the first group's first row never lands; 100 ms per wait
        try:
            call()
            with pytest.raises(lf.LayoutFoldError) as info:
                lf.check_device_error()
            assert info.value.status == 6 and lf.last_device_wait_code() in lf.WAIT_CODES
        finally:
            lf.set_test_hooks(False, 0)
        check(call())
        lf.check_device_error()


@pytest.mark.parametrize("pitch,off", [(1032, 8), (1031, 3), (1030, 2)])
def test_rows_of_wider_tensors(pitch, off):
    wide, wide_r = normal((6, pitch), 4).to(DEV), normal((6, pitch), 5, 2.0).to(DEV)
    D = 1000
    w = 1 + normal((D,), 6, 0.2)
    x, res = wide[:, off:off + D], wide_r[:, off:off + D]
    assert not x.is_contiguous()
    for fp8 in (False, True):
        got = lf.add_rms_norm(x, w.to(DEV), residual=res, eps=EPS, fp8=fp8)
        check_forward(x.cpu().contiguous(), w, res.cpu().contiguous(), fp8, got)


@pytest.mark.parametrize("D", [264, 1027, 70000])
def test_in_place_stream(D):
    x, w, res = normal((5, D), 8), 1 + normal((D,), 9, 0.2), normal((5, D), 10, 2.0)
    for alias in ("residual", "x"):
        xd, rd = x.to(DEV), res.to(DEV)
        h = rd if alias == "residual" else xd
        y, h2, _ = lf.add_rms_norm(xd, w.to(DEV), residual=rd, eps=EPS, h=h)
        assert h2.data_ptr() == h.data_ptr()
        check_forward(x, w, res, False, (y, h2, None))
    xd = x.to(DEV)
    y, _, _ = lf.add_rms_norm(xd, w.to(DEV), eps=EPS, y=xd)      # y over x
    check_forward(x, w, None, False, (y, y, None))


@pytest.mark.parametrize("D", [64, 1027])
def test_rows_of_zeros_and_of_other_magnitudes(D):
    x = normal((8, D), 11, dtype=FP32)
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4] = 0
    x[4, D // 2] = 3.0                      # one channel only
    w = 1 + normal((D,), 12, 0.2, FP32)
    check_forward(x, w, None, False, forward(x, w))
    y, _, scale = forward(x, w, fp8=True)
    check_forward(x, w, None, True, (y, None, scale))
    assert float(scale[1]) == 1.0 and not y[1].float().any()
    assert float(y[4].float().abs().max()) == 448.0


@pytest.mark.parametrize("D", [64, 1027, 70000])
def test_nan_and_infinity_stay_in_their_rows(D):
    x = normal((6, D), 13)
    x[1, 3] = float("nan")
    x[3, D - 1] = float("inf")
    x[4, 0] = float("-inf")
    w = 1 + normal((D,), 14, 0.2)
    y, _, _ = forward(x, w)
    q, _, scale = forward(x, w, fp8=True)
    fine = [0, 2, 5]
    check_forward(x[fine], w, None, False, (y[fine], x[fine], None))
    check_forward(x[fine], w, None, True, (q[fine], None, scale[fine]))
    assert torch.isnan(y[1]).all() and torch.isnan(y[3, D - 1]) and torch.isnan(y[4, 0])
    assert not y[3, :D - 1].any() and not y[4, 1:].any()     # 1 / rms is 0
    for r in (1, 3, 4):
        assert torch.isnan(scale[r]) and torch.isnan(q[r].float()).all()


def test_eps_zero_and_single_channel():
    x = torch.tensor([[3.0], [-2.0]], dtype=FP32)
    y, _, _ = lf.add_rms_norm(x.to(DEV), torch.tensor([0.5], device=DEV), eps=0.0)
    close(y, torch.tensor([[0.5], [-0.5]], dtype=torch.float64), 4 * ref.F32, "sign")


# ---------------------------------------------------------------- gradient
def check_backward(dy, h, w, dh, got):
    dx, dw = got
    M, D = h.shape
    h64 = h.double().requires_grad_()
    w64 = w.double().requires_grad_()
    dy64 = dy.double()
    gx, gw = ref.grads(ref.rms_norm(h64, w64, EPS), (h64, w64), dy64)
    h64, w64 = h64.detach(), w64.detach()
    r = ref.norm_factor(h64, EPS)
    g = dy64 * w64
    size = (r * g).abs() + h64.abs() * r ** 3 * (g * h64).abs().mean(-1, keepdim=True)
    if dh is not None:
        gx = gx + dh.double()
        size = size + dh.double().abs()
    close(dx, gx, 2 * R * size + ref.half_step(h.dtype) * gx.abs() + ref.smallest(h.dtype), "dx")
    if dw is not None:
        terms = (dy64 * h64 * r).abs().sum(0)
        chain = M / min(M, 304) + 64
        close(dw, gw, (R + chain * ref.F32) * terms + ref.half_step(w.dtype) * gw.abs() + ref.smallest(w.dtype), "dw")


def backward(dy, h, w, dh=None, **kw):
    dev = [None if t is None else t.to(DEV) for t in (dy, h, w, dh)]
    out = lf.add_rms_norm_backward(dev[0], dev[1], dev[2], dh=dev[3], eps=EPS, **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("M,D", SIZES + [(305, 72), (1000, 33), (911, 520)])
@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=IDS)
def test_backward(M, D, dtype, wdtype):
    h, w = normal((M, D), M * 3 + D, 2.0, dtype), 1 + normal((D,), D + 1, 0.2, wdtype)
    dy, dh = normal((M, D), 21 + D, 0.5, dtype), normal((M, D), 22 + D, 0.5, dtype)
    for d in (None, dh):
        check_backward(dy, h, w, d, backward(dy, h, w, d))


def test_backward_without_dweight_and_repeatable():
    h, w, dy = normal((700, 136), 31, 2.0), 1 + normal((136,), 32, 0.2), normal((700, 136), 33, 0.5)
    dx, none = backward(dy, h, w, want_dweight=False)
    assert none is None
    first = backward(dy, h, w)
    again = backward(dy, h, w)
    assert torch.equal(dx.view(torch.int16), first[0].view(torch.int16))
    assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16))
    assert torch.equal(first[1].view(torch.int16), again[1].view(torch.int16))


@pytest.mark.parametrize("D", [136, 1027, 70000])
def test_backward_in_place(D):
    h, w, dy, dh = normal((9, D), 34, 2.0), 1 + normal((D,), 35, 0.2), normal((9, D), 36, 0.5), normal((9, D), 37, 0.5)
    dyd = dy.to(DEV)
    check_backward(dy, h, w, dh, lf.add_rms_norm_backward(dyd, h.to(DEV), w.to(DEV), dh=dh.to(DEV), eps=EPS, dx=dyd))
    dhd = dh.to(DEV)
    check_backward(dy, h, w, dh, lf.add_rms_norm_backward(dy.to(DEV), h.to(DEV), w.to(DEV), dh=dhd, eps=EPS, dx=dhd))


def test_gradient_against_differences():
    """Directional derivative of L = sum(dy * y) in fp32: central difference with
    step t of the forward kernel.  Truncation ~ t^2 |L'''| and rounding ~ F32 |y dy| /
    t summed over N independent errors: with t = 2^-6 both are below 1e-3 of the scale of
    the terms' root sum of squares, which the bound takes as 4e-3."""
    M, D, t = 16, 200, 2.0 ** -6
    h, w, dy = normal((M, D), 41, 1.0, FP32), 1 + normal((D,), 42, 0.2, FP32), normal((M, D), 43, 1.0, FP32)
    v, vw = normal((M, D), 44, 1.0, FP32), normal((D,), 45, 1.0, FP32)
    dx, dw = backward(dy, h, w)

    def loss(hh, ww):
        return float((forward(hh, ww)[0].double().cpu() * dy.double()).sum())
    got = float((dx.double().cpu() * v.double()).sum())
    want = (loss(h + t * v, w) - loss(h - t * v, w)) / (2 * t)
    assert abs(got - want) < 4e-3 * np.sqrt(M * D)
    got = float((dw.double().cpu() * vw.double()).sum())
    want = (loss(h, w + t * vw) - loss(h, w - t * vw)) / (2 * t)
    assert abs(got - want) < 4e-3 * np.sqrt(M * D)


def test_backward_nan_stays_in_its_row():
    h, w, dy = normal((6, 264), 51, 2.0), 1 + normal((264,), 52, 0.2), normal((6, 264), 53, 0.5)
    dy[2, 5] = float("nan")
    dx, _ = backward(dy, h, w)
    fine = [0, 1, 3, 4, 5]
    check_backward(dy[fine], h[fine], w, None, (dx[fine], None))
    assert torch.isnan(dx[2]).all()


# ---------------------------------------------------------------- use
def test_refusals():
    x, w = normal((4, 64), 61).to(DEV), normal((64,), 62).to(DEV)
    for bad in (dict(weight=w.half()), dict(weight=w.double()), dict(weight="w")):
        with pytest.raises(TypeError):
            lf.add_rms_norm(x, **bad)
    with pytest.raises(TypeError):
        lf.add_rms_norm(x.double(), w.double())
    with pytest.raises(TypeError):
        lf.add_rms_norm(x, w, residual=x.float())
    for bad in (dict(weight=w[:32]), dict(weight=w, residual=x[:2]), dict(weight=w, h=x), dict(weight=w, y=x[:2]),
                dict(weight=w, scale=torch.empty(4, device=DEV)),
                dict(weight=w, residual=x, h=torch.empty(64, 4, device=DEV, dtype=BF16).t())):
        with pytest.raises(ValueError):
            lf.add_rms_norm(x, **bad)
    with pytest.raises(ValueError):
        lf.add_rms_norm(x.t(), w[:4].contiguous())           # no unit column stride
    with pytest.raises(ValueError):
        lf.add_rms_norm(x[:1].expand(4, 64), w)              # rows that overlap
    with pytest.raises(lf.LayoutFoldError):
        lf.add_rms_norm(x[:, :0], w[:0])                     # rows without channels
    with pytest.raises(ValueError):
        lf.add_rms_norm_backward(x[:2], x, w)
    with pytest.raises(TypeError):
        lf.add_rms_norm_backward(x.float(), x, w)
    with pytest.raises(lf.LayoutFoldError):
        lf.add_rms_norm_backward(x[:, :0].contiguous(), x[:, :0].contiguous(), w[:0])


def test_no_rows():
    x, w = normal((4, 64), 61).to(DEV), normal((64,), 62).to(DEV)
    y, h, scale = lf.add_rms_norm(x[:0], w, residual=x[:0], fp8=True)
    assert y.shape == (0, 64) and h.shape == (0, 64) and scale.shape == (0,)
    dx, dw = lf.add_rms_norm_backward(x[:0], x[:0], w)
    assert dx.shape == (0, 64) and not dw.any()


def test_outputs_stay_inside_their_buffers():
    """Every output lies between guard bands that must not change."""
    G = 4096
    for M, D, dtype in ((3, 1027, BF16), (5, 264, FP16), (2, 1530, FP32), (1, 70000, BF16), (700, 1027, BF16),
                        (613, 53, FP16), (801, 131, FP32), (608, 264, BF16)):
        x, w, res = normal((M, D), 71, 1.0, dtype), 1 + normal((D,), 72, 0.2, dtype), normal((M, D), 73, 1.0, dtype)
        n = M * D
        bufs = {k: torch.full((n + 2 * G,), 7.0, dtype=dtype, device=DEV) for k in ("h", "y", "dx")}
        view = {k: b[G:G + n].view(M, D) for k, b in bufs.items()}
        y, h, _ = lf.add_rms_norm(x.to(DEV), w.to(DEV), residual=res.to(DEV), eps=EPS, h=view["h"], y=view["y"])
        dwb = torch.full((D + 2 * G,), 7.0, dtype=dtype, device=DEV)  # (G elements keep 16-byte alignment)
        lf.add_rms_norm_backward(res.to(DEV), h, w.to(DEV), eps=EPS, dx=view["dx"], dweight=dwb[G:G + D])
        torch.cuda.synchronize()
        for b, size in [(b, n) for b in bufs.values()] + [(dwb, D)]:
            assert bool((b[:G] == 7.0).all()) and bool((b[G + size:] == 7.0).all())
        check_forward(x, w, res, False, (y, h, None))
        qb = torch.full((n + 2 * G,), 0x5A, dtype=torch.uint8, device=DEV)
        q = qb[G:G + n].view(E4M3).view(M, D)
        _, _, s = lf.add_rms_norm(x.to(DEV), w.to(DEV), residual=res.to(DEV), eps=EPS, fp8=True, y=q)
        assert bool((qb[:G] == 0x5A).all()) and bool((qb[G + n:] == 0x5A).all())
        check_forward(x, w, res, True, (q, h, s))


def test_unaligned_bases_take_the_scalar_path():
    M, D = 4, 256
    for off in (1, 3):
        x = normal((M * D + 8,), 81).to(DEV)[off:off + M * D].view(M, D)
        w = (1 + normal((D + 8,), 82, 0.2)).to(DEV)[off:off + D]
        y, h, _ = lf.add_rms_norm(x, w, eps=EPS)
        check_forward(x.cpu(), w.cpu(), None, False, (y, h, None))
        check_backward(x.cpu(), x.cpu(), w.cpu(), None, lf.add_rms_norm_backward(x, x, w, eps=EPS))


def test_on_a_side_stream_and_captured():
    x, w, res = (t.to(DEV) for t in (normal((33, 520), 91), 1 + normal((520,), 92, 0.2), normal((33, 520), 93, 2.0)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lf.add_rms_norm(x, w, residual=res, eps=EPS, stream=side)
    grad = lf.add_rms_norm_backward(x, got[1], w, eps=EPS, stream=side)
    side.synchronize()
    check_forward(x.cpu(), w.cpu(), res.cpu(), False, got)
    check_backward(x.cpu(), got[1].cpu(), w.cpu(), None, grad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            q = lf.add_rms_norm(x, w, residual=res, eps=EPS, fp8=True)
            grad = lf.add_rms_norm_backward(res, q[1], w, dh=x, eps=EPS)
    for seed in (94, 95):
        x.copy_(normal((33, 520), seed))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_forward(x.cpu(), w.cpu(), res.cpu(), True, q)
        check_backward(res.cpu(), q[1].cpu(), w.cpu(), x.cpu(), grad)


def test_new_tensors_of_a_side_stream():
    """They are neither memory that work of the current stream may still read, nor handed
    out again while the current stream may still read them."""
    M, D = 512, 4096
    x, w = normal((M, D), 96).to(DEV), torch.ones(D, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    calls = (lambda: lf.add_rms_norm(x, w, stream=side)[0], lambda: lf.add_rms_norm_backward(x, x, w, stream=side)[0])
    for call in calls:
        freed = torch.empty_like(x)
        at = freed.data_ptr()
        del freed
        got = call()
        assert got.data_ptr() != at
        at = got.data_ptr()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(50_000_000)  # the current stream is at work, and could be reading got
        del got
        again = call()
        assert again.data_ptr() != at
        torch.cuda.synchronize()


@pytest.mark.parametrize("M,D", [(525_000, 4104), (300_001, 7171)])
def test_offsets_past_32_bits(M, D):
    """More than 2^31 elements: rows at both ends and around the border."""
    w = 1 + normal((D,), 3, 0.2)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(M, D, dtype=BF16, device=DEV).normal_(generator=g)
    res = torch.empty(M, D, dtype=BF16, device=DEV).normal_(generator=g)
    border = 2 ** 31 // D
    rows = torch.tensor([0, 1, border - 1, border, border + 1, M - 2, M - 1], device=DEV)
    xs, rs = x[rows].cpu(), res[rows].cpu()
    q, h, s = lf.add_rms_norm(x, w.to(DEV), residual=res, eps=EPS, fp8=True)
    hs = h[rows]
    check_forward(xs, w, rs, True, (q.view(torch.uint8)[rows].view(E4M3), hs, s[rows]))
    del q, s
    dx, _ = lf.add_rms_norm_backward(x, h, w.to(DEV), dh=res, eps=EPS, dx=res)
    check_backward(xs, hs.cpu(), w, rs, (dx[rows], None))
    lf.check_device_error()


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("M", [5, 700])
def test_sums_of_subnormal_and_of_far_apart_numbers(dtype, M):
    """The packed 16-bit addition against one fp32 addition rounded once, over
    exponents from the type's subnormals to its largest."""
    D = 512
    g = torch.Generator().manual_seed(5)
    fi = torch.finfo(dtype)
    lo, hi = np.log2(fi.tiny * fi.eps), np.log2(fi.max) - 2

    def spread():
        e = torch.rand(M, D, generator=g, dtype=torch.float64) * (hi - lo) + lo
        return (torch.sign(torch.randn(M, D, generator=g)).double() * 2.0 ** e).to(dtype)
    x, res = spread(), spread()
    res[:, ::3] = (-x[:, ::3].float() * (1 + 2.0 ** -7)).to(dtype)      # cancellation
    y, h, _ = lf.add_rms_norm(x.to(DEV), torch.ones(D, dtype=dtype, device=DEV), residual=res.to(DEV), eps=EPS)
    assert torch.equal(h.cpu().view(torch.int16), kept(x, res).view(torch.int16))
