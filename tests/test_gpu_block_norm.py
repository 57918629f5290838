"""block_norm and block_norm_backward against the 64-bit reference.

Bounds, element by element.  F32 = 2^-24 is half a step of fp32; a sum of fp32 terms that
pass through at most S additions one after another is off by at most S F32 times the sum
of the terms' magnitudes.  A row's sums have S <= 128 (what one thread adds, at most 69,
the tree of a warp, at most 32 warps), so a factor r = rsqrt(mean + eps) is off by (S / 2
+ 3) F32 <= 67 F32 of itself, and R = 96 F32 covers r with the few products around it.
  h: R |beta p u|, 2 F32 of each summand, and the rounding.
  y, scale, codes: those of add_rms_norm on the kept h.
Backward, with size = |r2 g| + |h| r2^3 mean|g h| + |dh| and cu = beta u post:
  H: its mean term is off by S + 3 (S / 2 + 3) + a few F32, less than 4 R of it, the other
     terms by less: 4 R size.  dresidual: that times alpha, and the rounding.
  dx: H's error and r1's with the products: 5 R r1 |cu| size.  Its mean term: the three
     sums are off by S F32 of their terms' magnitudes, r2 twice, m2 and r1^3 by their
     factors, in all S + 5 (S / 2 + 3) + S: less than 6 R |x| r1^3 mean(|cu x| size).
  Parameters' gradients: a row's terms are off by 5 R, and are added one after another
     along at most M / min(M, 152) rows of a lane, 12 groups, and the blocks' and gate rows'
     sums by 32 threads each and a tree: CHAIN below.
"""
import math

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
TYPES = [(BF16, BF16), (BF16, FP32), (FP16, FP16), (FP16, FP32), (FP32, FP32)]
IDS = ["bf16", "bf16_w32", "fp16", "fp16_w32", "fp32"]


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


def dev(t):
    return None if t is None else t.to(DEV)


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)


def close(got, want, bound, what):
    got = got.detach().double().cpu()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %g of its bound, first at %s" % (
        what, int(bad.sum()), bad.numel(), float(((got - want).abs() / bound).max()), bad.nonzero()[0].tolist())


def rounding(want, dtype):
    return ref.half_step(dtype) * 1.001 * want.abs() + ref.smallest(dtype)


class Case:
    """Inputs of both passes on the CPU.  gates: 0, 1 ([D]) or more ([G, D])."""
    def __init__(self, M, D, dtype=BF16, wdtype=None, post=True, pre=True, gates=0, gate_dtype=None, a=0.75, b=0.5, seed=0):
        wdtype = wdtype or dtype
        s = 1000 * seed + M + D
        self.M, self.D, self.a, self.b = M, D, a, b
        self.x, self.res = normal((M, D), s, 1.5, dtype), normal((M, D), s + 1, 2.0, dtype)
        self.post = 1 + normal((D,), s + 2, 0.2, wdtype) if post else None
        self.pre = 1 + normal((D,), s + 3, 0.2, wdtype) if pre else None
        self.gate = None
        if gates:
            self.gate = normal((D,) if gates == 1 else (gates, D), s + 4, 0.7, gate_dtype or wdtype)
        self.h = normal((M, D), s + 5, 2.0, dtype)         # (of the backward pass, where no forward pass came before)
        self.dy = normal((M, D), s + 6, 0.5, dtype) if pre else None
        self.dh = normal((M, D), s + 7, 0.5, dtype)

    def kw(self):
        return dict(post=dev(self.post), pre=dev(self.pre), gate=dev(self.gate), branch_scale=self.b, residual_scale=self.a,
                    eps=EPS)

    def rows_gate(self):
        """The gate of every row in 64 bits, or 1."""
        if self.gate is None:
            return torch.ones(1, self.D, dtype=torch.float64)
        g = self.gate.double().reshape(-1, self.D)
        return g if g.shape[0] == 1 else g.repeat_interleave(self.M // g.shape[0], 0)

    def branch(self):
        x = self.x.double()
        return x if self.post is None else ref.rms_norm(x, self.post.double(), EPS)

    def forward(self, fp8=False, **kw):
        out = lf.block_norm(dev(self.x), dev(self.res), fp8=fp8, **{**self.kw(), **kw})
        lf.check_device_error()
        return out

    def check_forward(self, got, fp8=False, rows=slice(None)):
        y, h, scale = got
        M, D, t = self.M, self.D, self.x.dtype
        assert h.dtype == t and h.shape == (M, D)
        p = self.b * (self.branch() * self.rows_gate()).expand(M, D)
        want = self.a * self.res.double() + p
        close(h[rows], want[rows], ((R + 6 * ref.F32) * p.abs() + 2 * ref.F32 * (want.abs() + (self.a * self.res.double()).abs())
                                    + rounding(want, t))[rows], "h")
        if self.pre is None:
            assert y is None and scale is None
            return
        f = ref.rms_norm(h.cpu().double(), self.pre.double(), EPS)
        if not fp8:
            assert scale is None and y.dtype == t and y.shape == (M, D)
            close(y[rows], f[rows], (R * f.abs() + rounding(f, t))[rows], "y")
            return
        assert y.dtype == E4M3 and scale.dtype == FP32 and scale.shape == (M,)
        s = ref.row_scale(f)
        close(scale[rows], s[rows], ((R + 4 * ref.F32) * s)[rows], "scale")
        v = y.float().cpu().double() * scale.cpu().double()[:, None]
        close(v[rows], f[rows], ((2.0 ** -4 + R + 8 * ref.F32) * f.abs() + (s * 2.0 ** -10 * 1.001)[:, None])[rows], "y scale")

    def backward(self, dh=True, **kw):
        out = lf.block_norm_backward(dev(self.dy), dev(self.x), dev(self.h), dh=dev(self.dh) if dh else None,
                                     **{**self.kw(), **kw})
        lf.check_device_error()
        return out

    def check_backward(self, got, dh=True, rows=slice(None), sums=True):
        dx, dres, dpost, dpre, dgate = got
        M, D, t = self.M, self.D, self.x.dtype
        H = self.dh.double() if dh else torch.zeros(M, D, dtype=torch.float64)
        size = H.abs()
        if self.pre is not None:
            h = self.h.double().requires_grad_()
            w = self.pre.double().requires_grad_()
            dy = self.dy.double()
            gh, want_dpre = ref.grads(ref.rms_norm(h, w, EPS), (h, w), dy)
            h, w = h.detach(), w.detach()
            r2 = ref.norm_factor(h, EPS)
            H = H + gh
            size = size + (r2 * dy * w).abs() + h.abs() * r2 ** 3 * (dy * w * h).abs().mean(1, keepdim=True)
        close(dres[rows], (self.a * H)[rows], (self.a * 4 * R * size + rounding(self.a * H, t))[rows], "dresidual")
        x = self.x.double().requires_grad_()
        post = None if self.post is None else self.post.double().requires_grad_()
        gate = None if self.gate is None else self.gate.double().requires_grad_()
        p = x if post is None else ref.rms_norm(x, post, EPS)
        if gate is not None:
            g = gate.reshape(-1, D)
            p = p * (g if g.shape[0] == 1 else g.repeat_interleave(M // g.shape[0], 0))
        wanted = [v for v in (x, post, gate) if v is not None]
        grads = dict(zip([id(v) for v in wanted], ref.grads(self.b * p, wanted, H)))
        u = self.rows_gate()
        x64 = x.detach()
        cu = self.b * u * (1 if post is None else post.detach())
        want = grads[id(x)]
        if post is None:
            bound, xh = 5 * R * cu.abs() * size, x64
        else:
            r1 = ref.norm_factor(x64, EPS)
            xh = x64 * r1
            bound = 5 * R * r1 * cu.abs() * size + 6 * R * x64.abs() * r1 ** 3 * ((cu * x64).abs() * size).mean(1, keepdim=True)
        close(dx[rows], want[rows], (bound + rounding(want, t))[rows], "dx")
        if not sums:
            return
        chain = M / min(M, 152) + M / 32 + 160

        def summed(g, param, want, terms, what):
            assert (g is None) == (param is None), what
            if g is not None:
                assert g.dtype == param.dtype and g.shape == param.shape
                close(g, want, (5 * R + chain * ref.F32) * terms + rounding(want, g.dtype), what)
        if self.pre is not None:
            summed(dpre, self.pre, want_dpre, (dy * h * r2).abs().sum(0), "dpre")
        else:
            assert dpre is None
        summed(dpost, self.post, grads.get(id(post)), (self.b * u * xh).abs().mul(size).sum(0), "dpost")
        if gate is None:
            assert dgate is None
        else:
            terms = (self.b * xh * (1 if post is None else post.detach())).abs() * size
            terms = terms.reshape(-1 if gate.dim() > 1 else 1, M // (gate.shape[0] if gate.dim() > 1 else 1), D).sum(1)
            summed(dgate, self.gate, grads[id(gate)], terms.reshape(gate.shape), "dgate")


# what a call can have: post, pre, gate rows (as a rule of M)
def divisors(M):
    return [g for g in range(2, M + 1) if M % g == 0]


def forms(M):
    few, many = (divisors(M) or [1])[0], (divisors(M) or [1])[-1]
    mid = ([g for g in divisors(M) if g * g >= M] or [1])[0]
    return [dict(), dict(gates=1), dict(gates=few), dict(gates=many), dict(gates=mid), dict(post=False, gates=1),
            dict(post=False, gates=few), dict(pre=False, gates=1), dict(pre=False, gates=mid), dict(post=False),
            dict(pre=False), dict(post=False, pre=False), dict(post=False, pre=False, gates=few)]


SIZES = [(1, 1), (1, 5120), (2, 7), (3, 8), (5, 31), (4, 32), (6, 256), (9, 1000), (4, 1027), (6, 1530), (6, 4096),
         (2, 8192), (3, 8200), (2, 10001), (1, 16384), (2, 40000), (1, 70000)]


@pytest.mark.parametrize("M,D", SIZES)
@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=IDS)
def test_few_rows(M, D, dtype, wdtype):
    all_forms = D <= 1027 or dtype == BF16
    for i, form in enumerate(forms(M)):
        if not all_forms and i % 4:
            continue
        c = Case(M, D, dtype, wdtype, gate_dtype=dtype if i % 2 else FP32, **form)
        c.check_forward(c.forward())
        if c.pre is not None:
            c.check_forward(c.forward(fp8=True), fp8=True)
        for dh in (True, False) if c.pre is not None else (True,):
            c.check_backward(c.backward(dh=dh), dh=dh)


# Enough rows for the rings: one warp per row and many groups of them, several warps, one
# group only, rows too long; rows that are not a multiple of 16 bytes; few of those
MANY = [(610, 8), (1000, 136), (2500, 264), (700, 1032), (1300, 2056), (640, 5120), (612, 12296), (610, 20000),
        (700, 33), (612, 37), (900, 250), (1332, 1027), (777, 1530), (650, 5121), (609, 9999), (608, 12301),
        (620, 16384), (609, 16383), (100, 1027), (153, 515), (303, 2050), (1, 5121), (4, 10303), (33, 13611),
        # rows on two and four CTAs
        (40, 12288), (160, 16383), (310, 11416), (78, 22000), (90, 14337), (620, 9000)]


@pytest.mark.parametrize("M,D", MANY)
@pytest.mark.parametrize("dtype,wdtype", TYPES, ids=IDS)
def test_many_rows(M, D, dtype, wdtype):
    big = M * D > 3_000_000
    for i, form in enumerate(forms(M)):
        if (big or dtype != BF16) and i not in ((2,) if dtype != BF16 else (0, 1, 4, 8)):
            continue
        c = Case(M, D, dtype, wdtype, gate_dtype=FP32 if i % 2 else dtype, **form)
        c.check_forward(c.forward())
        if c.pre is not None:
            c.check_forward(c.forward(fp8=True), fp8=True)
        dh = c.pre is None or i % 2 == 0
        c.check_backward(c.backward(dh=dh), dh=dh)


@pytest.mark.parametrize("M,gates", [(608, 608), (1216, 2), (1216, 76), (1216, 304), (4560, 15), (4560, 1520), (20000, 4),
                                     (20000, 20000)])
def test_gate_rows_across_lanes(M, gates):
    """Gate rows shorter and longer than a lane's share of the rows, and of the same size."""
    c = Case(M, 136, gates=gates)
    c.check_forward(c.forward())
    c.check_backward(c.backward())
    c = Case(M, 77, FP32, gates=gates, post=False)
    c.check_forward(c.forward())
    c.check_backward(c.backward(dh=False), dh=False)


def test_leading_dimensions_and_gates_of_their_rows():
    c = Case(6 * 35, 264, gates=6)
    for gate in (c.gate.view(6, 1, 264), c.gate):
        y, h, s = lf.block_norm(dev(c.x).view(6, 35, 264), dev(c.res).view(6, 35, 264),
                                **{**c.kw(), "gate": dev(gate)}, fp8=True)
        assert y.shape == h.shape == (6, 35, 264) and s.shape == (6, 35)
        c.check_forward((y.view(210, 264), h.view(210, 264), s.view(210)), fp8=True)
        view = [dev(t).view(6, 35, 264) for t in (c.dy, c.x, c.h)]
        dx, dres, dpost, dpre, dgate = lf.block_norm_backward(*view, **{**c.kw(), "gate": dev(gate)})
        assert dgate.shape == gate.shape and dx.shape == dres.shape == (6, 35, 264)
        c.check_backward((dx.view(210, 264), dres.view(210, 264), dpost, dpre, dgate.view(6, 264)), dh=False)
    one = Case(1, 264, gates=1)
    y, h, _ = lf.block_norm(dev(one.x)[0], dev(one.res)[0], **one.kw())
    assert y.shape == (264,)
    one.check_forward((y[None], h[None], None))


@pytest.mark.parametrize("M", [6, 700])
@pytest.mark.parametrize("pitch,off", [(1032, 8), (1031, 3), (1030, 2)])
def test_rows_of_wider_tensors(M, pitch, off):
    c = Case(M, 1000, gates=2)
    wide = [torch.full((M, pitch), float("nan"), dtype=BF16, device=DEV) for _ in range(2)]
    for w, t in zip(wide, (c.x, c.res)):
        w[:, off:off + 1000] = dev(t)
    x, res = (w[:, off:off + 1000] for w in wide)
    for fp8 in (False, True):
        c.check_forward(lf.block_norm(x, res, fp8=fp8, **c.kw()), fp8=fp8)
        c.check_forward(lf.block_norm(x, dev(c.res), fp8=fp8, **c.kw()), fp8=fp8)
    lf.check_device_error()


@pytest.mark.parametrize("M,D", [(5, 264), (5, 1027), (2, 70000), (700, 264), (700, 1027)])
def test_in_place(M, D):
    c = Case(M, D, gates=1)
    want = c.forward()
    c.check_forward(want)
    for over in ("res", "x", "both", "crossed"):
        x, res = dev(c.x), dev(c.res)
        out = {"res": dict(h=res), "x": dict(h=x), "both": dict(h=res, y=x), "crossed": dict(h=x, y=res)}[over]
        y, h, _ = lf.block_norm(x, res, **c.kw(), **out)
        assert torch.equal(bits(y), bits(want[0])) and torch.equal(bits(h), bits(want[1])), over
    grads = c.backward()
    c.check_backward(grads)
    for a, b in ((0, 3), (1, 2), (2, 1), (3, 0)):
        t = [dev(v) for v in (c.dy, c.x, c.h, c.dh)]
        got = lf.block_norm_backward(t[0], t[1], t[2], dh=t[3], **c.kw(), dx=t[a], dresidual=t[b])
        for g, w in zip(got, grads):
            assert torch.equal(bits(g), bits(w))


def test_unaligned_bases_take_the_scalar_path():
    c = Case(4, 256, gates=2)

    def shifted(t, off):
        buf = torch.empty(t.numel() + off, dtype=t.dtype, device=DEV)
        buf[off:] = dev(t).flatten()
        return buf[off:].view(t.shape)
    for off in (1, 3):
        x, res, dy, h, dh = (shifted(t, off) for t in (c.x, c.res, c.dy, c.h, c.dh))
        kw = {k: shifted(v.cpu(), off) if torch.is_tensor(v) else v for k, v in c.kw().items()}
        c.check_forward(lf.block_norm(x, res, **kw))
        c.check_forward(lf.block_norm(x, res, fp8=True, **kw), fp8=True)
        c.check_backward(lf.block_norm_backward(dy, x, h, dh=dh, **kw))


@pytest.mark.parametrize("M,D", [(6, 64), (6, 1027), (6, 70000), (1000, 264)])
def test_nan_and_infinity_stay_in_their_rows(M, D):
    c = Case(M, D)
    c.x[1, 3] = float("nan")
    c.res[3, D - 1] = float("inf")
    fine = [i for i in range(M) if i not in (1, 3)]
    y, h, _ = got = c.forward()
    c.check_forward(got, rows=fine)
    assert torch.isnan(h[1]).all() and torch.isnan(y[1]).all() and h[3, D - 1] == float("inf")
    assert torch.isnan(y[3, D - 1]) and not y[3, :D - 1].any()
    q, _, s = got = c.forward(fp8=True)
    c.check_forward(got, fp8=True, rows=fine)
    assert torch.isnan(s[1]) and torch.isnan(s[3]) and torch.isnan(q[[1, 3]].float()).all()
    c = Case(M, D)
    c.dy[1, 3] = float("nan")
    c.x[3, 5] = float("nan")
    got = c.backward()
    c.check_backward(got, rows=fine, sums=False)
    assert torch.isnan(got[0][1]).all() and torch.isnan(got[0][3]).all() and not torch.isnan(got[1][3]).any()


@pytest.mark.parametrize("M,D", [(8, 64), (8, 1027), (800, 264)])
def test_rows_of_zeros_and_of_other_magnitudes(M, D):
    c = Case(M, D, FP32, gates=1, a=1.0)
    for t in (c.x, c.res, c.h):
        t[1] = 0
        t[2] *= 1e-15
        t[3] *= 1e15
    c.x[4] = 0
    c.res[5] = 0
    c.dy[6] = 0
    c.check_forward(c.forward())
    y, _, s = got = c.forward(fp8=True)
    c.check_forward(got, fp8=True)
    assert float(s[1]) == 1.0 and not y[1].float().any()
    got = c.backward()
    rows = [i for i in range(M) if i != 3]          # (whose gradient of h is a difference of its dh alone)
    c.check_backward(got, rows=rows, sums=False)


@pytest.mark.parametrize("M", [5, 700])
def test_codes_of_products_outside_fp32(M):
    """Rows whose products h pre leave fp32's range, although (h r2) pre does not: the same
    codes and scales as add_rms_norm's on the kept h."""
    D = 264
    g = torch.Generator().manual_seed(3)
    res = torch.randn(M, D, generator=g) * 2.0 ** torch.randint(-60, 60, (M, 1), generator=g).float()
    x = torch.randn(M, D, generator=g)
    for e in (100, 0, -110):
        pre = (1 + 0.2 * torch.randn(D, generator=g)) * 2.0 ** e
        y, h, s = lf.block_norm(dev(x), dev(res), pre=dev(pre), fp8=True, branch_scale=0.0)
        want, _, ws = lf.add_rms_norm(h, dev(pre), fp8=True)
        assert torch.equal(h.cpu(), res)
        # (the two sums of squares may be added in another order)
        assert torch.allclose(s.cpu(), ws.cpu(), rtol=2 * R, atol=0)
        v, w = y.float().cpu().double() * s.cpu().double()[:, None], want.float().cpu().double() * ws.cpu().double()[:, None]
        off = (v - w).abs() > 2 * (2.0 ** -4 * w.abs() + ws.cpu().double()[:, None] * 2.0 ** -10)
        assert not off.any()
    lf.check_device_error()


@pytest.mark.parametrize("M,D,dtype,form", [
    (3, 1027, BF16, dict(gates=3)), (5, 264, FP16, dict(gates=1)), (2, 1530, FP32, dict(gates=2)), (1, 70000, BF16, dict()),
    (700, 1027, BF16, dict(gates=1)), (613, 53, FP16, dict()), (801, 131, FP32, dict(gates=267)),
    (608, 264, BF16, dict(gates=8)), (100, 1027, BF16, dict(post=False, gates=1)), (620, 520, FP32, dict(pre=False, gates=620))])
def test_outputs_stay_inside_their_buffers(M, D, dtype, form):
    """Every output lies between guard bands that must not change."""
    G = 4096
    c = Case(M, D, dtype, **form)

    def guarded(t, fill=7.0):
        n = t.numel()
        buf = torch.full((n + 2 * G,), fill, dtype=t.dtype, device=DEV)
        return buf, buf[G:G + n].view(t.shape), n
    names = {"h": c.x, "y": c.x if c.pre is not None else None}
    grads = {"dx": c.x, "dresidual": c.x, "dpost": c.post, "dpre": c.pre, "dgate": c.gate}
    bufs = {k: guarded(t) for k, t in {**names, **grads}.items() if t is not None}
    got = c.forward(**{k: bufs[k][1] for k in names if k in bufs})
    grad = c.backward(**{k: bufs[k][1] for k in grads if k in bufs})
    c.check_forward(got)
    c.check_backward(grad)
    if c.pre is not None:
        codes, scale = torch.full((M * D + 2 * G,), 0x5A, dtype=torch.uint8, device=DEV), guarded(torch.empty(M))
        q = c.forward(fp8=True, y=codes[G:G + M * D].view(E4M3).view(M, D), scale=scale[1])
        c.check_forward(q, fp8=True)
        assert bool((codes[:G] == 0x5A).all()) and bool((codes[G + M * D:] == 0x5A).all())
        bufs["scale"] = scale
    for k, (buf, _, n) in bufs.items():
        assert bool((buf[:G] == 7.0).all()) and bool((buf[G + n:] == 7.0).all()), k


@pytest.mark.parametrize("M,D,form", [(700, 136, dict(gates=1)), (700, 136, dict(gates=7)), (40, 1027, dict(gates=4))])
def test_repeatable_parts_alone_and_on_two_streams(M, D, form):
    c = Case(M, D, **form)
    first, grads = c.forward(), c.backward()
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [dev(t) for t in (c.x, c.res, c.dy, c.h, c.dh)]
    kw = c.kw()
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        s = streams[i % 2]
        got.append((lf.block_norm(args[0], args[1], stream=s, **kw),
                    lf.block_norm_backward(args[2], args[0], args[3], dh=args[4], stream=s, **kw)))
    torch.cuda.synchronize()
    lf.check_device_error()
    for f, b in got:
        for x, w in zip((*f[:2], *b), (*first[:2], *grads)):
            assert torch.equal(bits(x), bits(w))
    # one output is the same with and without the others
    none = c.backward(want_dparams=False)
    assert none[2:] == (None, None, None)
    for i, name in ((2, "dpost"), (3, "dpre"), (4, "dgate")):
        only = c.backward(want_dparams=False, **{name: torch.empty_like(grads[i])})
        assert [g is None for g in only[2:]] == [j != i for j in (2, 3, 4)]
        assert torch.equal(bits(only[i]), bits(grads[i])) and torch.equal(bits(only[0]), bits(grads[0]))
    assert torch.equal(bits(none[0]), bits(grads[0])) and torch.equal(bits(none[1]), bits(grads[1]))


@pytest.mark.parametrize("M,D,gates", [(33, 520, 1), (700, 520, 1), (150, 1027, 1), (700, 520, 7), (330, 1027, 5), (60, 264, 60)])
def test_on_a_side_stream_and_captured(M, D, gates):
    c = Case(M, D, gates=gates)
    x, res, dy, h, dh = (dev(t) for t in (c.x, c.res, c.dy, c.h, c.dh))
    kw = c.kw()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lf.block_norm(x, res, stream=side, **kw)
    grad = lf.block_norm_backward(dy, x, h, dh=dh, stream=side, **kw)
    side.synchronize()
    c.check_forward(got)
    c.check_backward(grad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            got = lf.block_norm(x, res, fp8=True, **kw)
            grad = lf.block_norm_backward(dy, x, h, dh=dh, **kw)
    for seed in (94, 95):
        c.x = normal((M, D), seed)
        x.copy_(dev(c.x))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        lf.check_device_error()
        c.check_forward(got, fp8=True)
        c.check_backward(grad)


def test_new_tensors_of_a_side_stream():
    """They are not memory that work of the current stream may still read."""
    x, w = normal((512, 4096), 96).to(DEV), torch.ones(4096, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for call in (lambda: lf.block_norm(x, x, w, w, stream=side)[0],
                 lambda: lf.block_norm_backward(x, x, x, w, w, stream=side)[0]):
        freed = torch.empty_like(x)
        at = freed.data_ptr()
        del freed
        got = call()
        assert got.data_ptr() != at
        torch.cuda.synchronize()


@pytest.mark.parametrize("M,D,gates", [(1000, 1024, 4), (616, 4096, 1), (300, 1027, 1), (80, 12288, 2)])
def test_stalled_wait_times_out_and_context_survives(M, D, gates):
    """Rows of one warp, of several, phased, and on two CTAs."""
    c = Case(M, D, gates=gates)
    forward = M >= 300
    for call, check in ((lambda: lf.block_norm(dev(c.x), dev(c.res), **c.kw()), c.check_forward),
                        (lambda: lf.block_norm(dev(c.x), dev(c.res), fp8=True, **c.kw()),
                         lambda out: c.check_forward(out, fp8=True)),
                        (lambda: lf.block_norm_backward(dev(c.dy), dev(c.x), dev(c.h), dh=dev(c.dh), **c.kw()),
                         c.check_backward))[0 if forward else 2:]:
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


def test_no_rows():
    c = Case(4, 64, gates=2)
    kw = c.kw()
    x = dev(c.x)[:0]
    y, h, s = lf.block_norm(x, x, fp8=True, **kw)
    assert y.shape == h.shape == (0, 64) and s.shape == (0,)
    dx, dres, *params = lf.block_norm_backward(x, x, x, **kw)
    assert dx.shape == dres.shape == (0, 64) and all(not p.any() for p in params)
    with pytest.raises(lf.LayoutFoldError):
        lf.block_norm(dev(c.x)[:, :0], dev(c.res)[:, :0], h=torch.empty(4, 0, dtype=BF16, device=DEV))


@pytest.mark.parametrize("form", [dict(gates=1), dict(gates=4), dict(post=False, gates=4), dict(pre=False, gates=1)])
def test_gradient_against_differences(form):
    """Directional derivatives of L = sum(dy y) + sum(dh h) in fp32 by central differences
    of the forward kernel with step t = 2^-7: truncation ~ t^2 |L'''| / 6 and rounding ~ R / t
    of independent terms are below 1e-3 of the terms' root sum of squares (M D terms of
    order dy, and as many of dh); the bound takes 4e-3 of 1.5 sqrt(M D)."""
    M, D, t = 16, 200, 2.0 ** -7
    c = Case(M, D, FP32, **form)
    c.h = None
    kw = c.kw()

    def out(x, res, kw):
        return lf.block_norm(x, res, **kw)
    x, res = dev(c.x), dev(c.res)
    _, h, _ = out(x, res, kw)
    got = lf.block_norm_backward(dev(c.dy), x, h, dh=dev(c.dh), **kw)

    def loss(x, res, kw):
        y, h, _ = out(x, res, kw)
        total = (h.double().cpu() * c.dh.double()).sum()
        return float(total if y is None else total + (y.double().cpu() * c.dy.double()).sum())
    for i, name in enumerate(("x", "res", "post", "pre", "gate")):
        at = {"x": x, "res": res}.get(name, kw.get(name))
        if at is None:
            assert got[i] is None
            continue
        v = normal(at.shape, 70 + i, 1.0, FP32).to(DEV)
        ends = []
        for sign in (1, -1):
            a = {"x": x, "res": res, **kw}
            a[name] = at + sign * t * v
            ends.append(loss(a.pop("x"), a.pop("res"), a))
        want = (ends[0] - ends[1]) / (2 * t)
        assert abs(float((got[i].double() * v.double()).sum()) - want) < 4e-3 * 1.5 * math.sqrt(M * D), name


def test_a_block_of_the_operators_together():
    """Serving and training a block: linear -> block_norm (e4m3 for the next projections)
    -> gated_ffn -> linear -> block_norm, and back, against the formulas in 64 bits on the
    rounded values that pass between the operators."""
    M, D, F = 300, 272, 528
    s = 1 / math.sqrt(D)
    x0, res = normal((M, D), 1), normal((M, D), 2, 2.0)
    wo, bo = normal((D, D), 3, s), normal((D,), 4, 0.3)
    wd = normal((D, F), 5, 1 / math.sqrt(F))
    wgu = normal((2 * F, D), 6, s)
    c = Case(M, D, gates=3, a=1.0, b=0.5)
    c.res = res
    kw = c.kw()
    attn, _ = lf.linear(dev(x0), dev(wo), bias=dev(bo))
    c.x = attn.cpu()
    y8, h, sc = lf.block_norm(attn, dev(res), fp8=True, **kw)
    c.check_forward((y8, h, sc), fp8=True)
    w8 = (wgu.float() / ref.row_scale(wgu.double()).float()[:, None]).to(E4M3)
    ws = ref.row_scale(wgu.double()).float()
    ff8, _ = lf.gated_ffn(y8, dev(w8), x_scale=sc, w_scale=dev(ws))
    y, h2, _ = lf.block_norm(attn, dev(res), **kw)
    assert torch.equal(bits(h2), bits(h))
    ff, gu = lf.gated_ffn(y, dev(wgu), want_gu=True)
    # e4m3 against bf16: each operand is off by 2^-4 at most, half of it typically, of random sign over D products
    assert float((ff8.float() - ff.float()).norm() / ff.float().norm()) < 0.1
    down, _ = lf.linear(ff, dev(wd))
    c2 = Case(M, D, gates=3, a=1.0, b=0.5)
    c2.x, c2.res = down.cpu(), h.cpu()
    got = lf.block_norm(down, h, **kw)
    c2.check_forward(got)
    # and back: the gradient of the second norm's y through both
    c2.h = got[1].cpu()
    g2 = lf.block_norm_backward(dev(c2.dy), down, got[1], dh=dev(c2.dh), **kw)
    c2.check_backward(g2)
    dff, dwd, _ = lf.linear_backward(g2[0], ff, dev(wd))
    want = g2[0].cpu().double() @ wd.double()
    assert float((dff.cpu().double() - want).norm()) <= ref.half_step(BF16) * float(want.norm())
    dy, dwgu = lf.gated_ffn_backward(dff, y, dev(wgu), gu)
    c.h, c.dy, c.dh = h.cpu(), dy.cpu(), g2[1].cpu()
    g1 = lf.block_norm_backward(dy, attn, h, dh=g2[1], **kw)
    c.check_backward(g1)
    dx0, dwo, dbo = lf.linear_backward(g1[0], dev(x0), dev(wo), bias=dev(bo))
    want = g1[0].cpu().double().t() @ x0.double()
    assert float((dwo.cpu().double() - want).norm()) <= ref.half_step(BF16) * float(want.norm())
    lf.check_device_error()


@pytest.mark.parametrize("M,D,gates", [(525_000, 4104, 1), (300_000, 7171, 4)])
def test_offsets_past_32_bits(M, D, gates):
    """More than 2^31 elements: rows at both ends and around the border."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(M, D, dtype=BF16, device=DEV).normal_(generator=g)
    res = torch.empty(M, D, dtype=BF16, device=DEV).normal_(generator=g)
    border = 2 ** 31 // D
    rows = torch.tensor([0, 1, border - 1, border, border + 1, M - 2, M - 1], device=DEV)
    c = Case(7, D, gates=1)
    c.gate = normal((D,) if gates == 1 else (gates, D), 5)
    kw = c.kw()
    if gates > 1:     # (the rows' own gates, for the check)
        c.gate = c.gate[(rows.cpu() * gates) // M]
    c.x, c.res = x[rows].cpu(), res[rows].cpu()
    q, h, s = lf.block_norm(x, res, fp8=True, **kw)
    c.check_forward((q.view(torch.uint8)[rows].view(E4M3), h[rows], s[rows]), fp8=True)
    del q, s
    c.h, c.dy = h[rows].cpu(), c.res
    dx, dres, *_ = lf.block_norm_backward(res, x, h, dx=res, dresidual=h, **kw)
    c.check_backward((dx[rows], dres[rows], None, None, None), dh=False, sums=False)
    lf.check_device_error()
