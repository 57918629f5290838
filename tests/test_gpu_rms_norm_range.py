"""add_rms_norm where products of the stream and the weights leave fp32's range, or
lie among its subnormal numbers, although h / rms(h) weight need not.

Bounds, element by element, with R as in test_gpu_rms_norm.py.  f32, the kernel's
f = (h r) w, is off by R |f|, and by 2^-150 more where it is subnormal.  Its row's
scale s is the largest |f32| / 448: off by (R + 4 F32) s, and by 2^-150 where it is
subnormal (2^-150 / 448 of f32's is the 1.01 below).  A code stands for f / s within
half a step (2^-4 relative, 2^-10 for the smallest), and a scale that was rounded down
by 2^-150 cuts the largest codes by at most 448 * 2^-150 (450 with the rest).  Where
the scale rounds to 0 it is 1 and all codes are 0, so f itself, at most 448 * 1.1 *
2^-150, is lost: 500 * 2^-150 covers both.
"""
import pytest
import torch

import ffn_reference as ref
import layout_folding_gb300 as lf

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
R = 96 * ref.F32
BF16, FP32 = torch.bfloat16, torch.float32
TINY = 2.0 ** -150


@pytest.fixture(scope="module", autouse=True)
def _device():
    lf.lib()
    torch.cuda.set_device(0)
    lf.check_device_error()
    yield
    torch.cuda.synchronize()


def row(M, D, exponent, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, D, generator=g, dtype=torch.float64) * 2.0 ** exponent
    x[:, ::3] = 0
    return x.to(dtype)


def weights(D, exponent, seed):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.2 * torch.randn(D, generator=g, dtype=torch.float64)) * 2.0 ** exponent).float()


def check_codes(h, w, eps, y, scale):
    f = ref.rms_norm(h.double(), w.double(), eps)
    # the statistics are fp32's: a sum of squares past its largest number has r = 0
    f[h.double().square().sum(-1) > torch.finfo(FP32).max] = 0
    s = f.abs().amax(-1) / ref.E4M3_MAX
    scale = scale.cpu().double()
    y = y.float().cpu().double()
    ok = ((scale - s).abs() <= (R + 4 * ref.F32) * s + 1.01 * TINY) & (s > 0.9 * TINY)
    ok |= (scale == 1) & (s < 1.1 * TINY)
    assert ok.all(), (scale[~ok], s[~ok])
    bound = (2.0 ** -4 + R + 8 * ref.F32) * f.abs() + (s * 2.0 ** -10 * 1.001)[:, None] + 500 * TINY
    bad = ~((y * scale[:, None] - f).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())
    assert not y[h.expand_as(y) == 0].any()


# one block a row, phased rows, rings of each kind, rows that are read twice
SIZES = [(3, 7), (5, 64), (5, 1027), (3, 5120), (700, 264), (700, 1027), (610, 5120), (4, 70000)]
# exponents of the stream and of the weights, eps
RANGES = [(0, -143, 1e-5),    # scales that round to 0
          (0, -140, 1e-5),    # scales of one or a few times 2^-149
          (60, -130, 1e-5),   # the same from ordinary products
          (50, 90, 1e-5),     # products past the largest fp32 number
          (62, 100, 1e-5),
          (-50, -90, 0.0),    # subnormal products of an ordinary f
          (-60, -100, 0.0)]   # products that are 0


@pytest.mark.parametrize("M,D", SIZES)
@pytest.mark.parametrize("hexp,wexp,eps", RANGES)
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_e4m3_of_products_outside_the_range(M, D, hexp, wexp, eps, dtype):
    x, w = row(M, D, hexp, 1, dtype), weights(D, wexp, 2)
    res = row(M, D, hexp, 3, dtype)
    x[1::3] = row(M, D, 0, 4, dtype)[1::3]       # ordinary rows among them
    res[1::3] = row(M, D, 0, 5, dtype)[1::3]
    y, _, scale = lf.add_rms_norm(x.to(DEV), w.to(DEV), eps=eps, fp8=True)
    check_codes(x, w, eps, y, scale)
    y, h, scale = lf.add_rms_norm(x.to(DEV), w.to(DEV), residual=res.to(DEV), eps=eps, fp8=True)
    check_codes(h.cpu(), w, eps, y, scale)
    lf.check_device_error()


@pytest.mark.parametrize("M,D", [(5, 1027), (700, 264)])
def test_zeros_and_nan_among_them(M, D):
    x, w = row(M, D, 50, 1, FP32), weights(D, 90, 2)
    x[0] = 0
    x[2, 5] = float("nan")
    x[4, 1] = float("inf")
    y, _, scale = lf.add_rms_norm(x.to(DEV), w.to(DEV), fp8=True)
    fine = [i for i in range(M) if i not in (2, 4)]
    check_codes(x[fine], w, 1e-6, y.view(torch.uint8)[fine].view(y.dtype), scale[fine])
    assert float(scale[0]) == 1.0
    for r in (2, 4):
        assert torch.isnan(scale[r]) and torch.isnan(y[r].float()).all()
    # weights of zero: nothing to scale
    y, _, scale = lf.add_rms_norm(x[fine].to(DEV), torch.zeros(D, device=DEV), fp8=True)
    assert not y.float().any() and bool((scale == 1).all())


@pytest.mark.parametrize("M,D", SIZES)
@pytest.mark.parametrize("hexp,wexp,eps", [(40, -120, 1e-5),    # r weight is 0 in fp32
                                           (40, -100, 1e-5),    # subnormal
                                           (-50, 90, 0.0)])     # infinite; h / rms(h) weight is not
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_factors_outside_the_range(M, D, hexp, wexp, eps, dtype):
    x, w = row(M, D, hexp, 1, dtype), weights(D, wexp, 2)
    y, _, _ = lf.add_rms_norm(x.to(DEV), w.to(DEV), eps=eps)
    f = ref.rms_norm(x.double(), w.double(), eps)
    bad = ~((y.cpu().double() - f).abs() <= (ref.half_step(dtype) + R) * f.abs() + ref.smallest(dtype))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())
    lf.check_device_error()
