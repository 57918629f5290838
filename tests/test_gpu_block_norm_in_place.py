"""block_norm and its gradient over their inputs' memory where rows are shared by the CTAs of
a cluster, and where odd rows with one or several gate rows run in rings, whose copies read
a neighbour's elements beside a row while its owner overwrites them.  The results have to
be those of new tensors, bit for bit; bounds of those: test_gpu_block_norm's."""
import pytest
import torch

import layout_folding_gb300 as lf
from test_gpu_block_norm import BF16, FP16, FP32, Case, _device, bits, dev  # noqa: F401

pytestmark = pytest.mark.gpu

#        M, D, dtype, gates
SIZES = [(40, 12288, BF16, 0), (40, 12288, BF16, 4), (160, 16383, BF16, 1), (256, 16383, BF16, 4), (78, 22000, BF16, 2),
         (78, 21999, FP16, 1), (64, 9000, FP32, 1), (64, 12289, FP32, 2), (700, 1027, BF16, 0), (700, 1027, BF16, 7),
         (1020, 4097, FP16, 4), (640, 517, FP32, 5), (1216, 5120, BF16, 8), (2432, 264, BF16, 76)]


def same(got, want):
    for g, w in zip(got, want):
        assert (g is None) == (w is None)
        assert g is None or torch.equal(bits(g), bits(w))


@pytest.mark.parametrize("M,D,dtype,gates", SIZES)
def test_gradient_over_its_inputs(M, D, dtype, gates):
    c = Case(M, D, dtype, gates=gates)
    want = c.backward()
    c.check_backward(want)
    for a, b in ((0, 3), (1, 2), (2, 1), (3, 0), (0, 1), (2, 3)):
        for _ in range(3):  # (neighbours meet at another time in each)
            t = [dev(v) for v in (c.dy, c.x, c.h, c.dh)]
            got = lf.block_norm_backward(t[0], t[1], t[2], dh=t[3], **c.kw(), dx=t[a], dresidual=t[b])
            assert got[0] is t[a] and got[1] is t[b]
            same(got, want)
    lf.check_device_error()


@pytest.mark.parametrize("post,pre,dh", [(False, True, True), (True, False, True), (False, False, True), (True, True, False)])
def test_gradient_of_a_part_over_its_inputs(post, pre, dh):
    for M, D, dtype, gates in ((256, 16383, BF16, 4), (700, 1027, BF16, 7), (40, 12288, BF16, 1)):
        c = Case(M, D, dtype, gates=gates, post=post, pre=pre)
        want = c.backward(dh=dh)
        c.check_backward(want, dh=dh)
        t = {"dy": dev(c.dy), "x": dev(c.x), "h": dev(c.h), "dh": dev(c.dh) if dh else None}
        over = [k for k in ("x", "dy", "dh") if t[k] is not None][:2]
        got = lf.block_norm_backward(t["dy"], t["x"], t["h"], dh=t["dh"], **c.kw(), dx=t[over[0]], dresidual=t[over[1]])
        same(got, want)
    lf.check_device_error()


@pytest.mark.parametrize("M,D,dtype,gates", SIZES)
def test_forward_over_its_inputs(M, D, dtype, gates):
    c = Case(M, D, dtype, gates=gates)
    want, want8 = c.forward(), c.forward(fp8=True)
    c.check_forward(want)
    c.check_forward(want8, fp8=True)
    for over in ("res", "x", "both", "crossed"):
        x, res = dev(c.x), dev(c.res)
        out = {"res": dict(h=res), "x": dict(h=x), "both": dict(h=res, y=x), "crossed": dict(h=x, y=res)}[over]
        same(lf.block_norm(x, res, **c.kw(), **out), want)
    for over in ("res", "x"):
        x, res = dev(c.x), dev(c.res)
        same(lf.block_norm(x, res, fp8=True, **c.kw(), h=res if over == "res" else x), want8)
    lf.check_device_error()
