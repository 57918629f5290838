"""linear where its kernels have more than one way: stages of the few-token kernel's ring used
again and again, two of its CTAs on an SM, K loops shared by every number of CTAs or pairs,
shared tiles of every width.  The way a call took is read back.  Bounds: test_gpu_linear's.

How many CTAs or pairs share a tile depends on the clusters that the device holds; those
below are of 152 SMs as they were found (seven never came up there: clusters of seven fit
no more often than clusters of eight).  On a device that holds others a case is checked all
the same and then skipped, and the last test says that enough of them were met."""
import os

import pytest
import torch

import layout_folding_gb300 as lf
from test_gpu_linear import BF16, DEV, _device, check_forward, dev, inputs, normal, quantised  # noqa: F401

pytestmark = pytest.mark.gpu

# (M, N, K, e4m3), the MMA's N, split, stages
FEW = [((1, 5120, 5120, False), 16, 3, 6), ((1, 5120, 13824, False), 16, 3, 12), ((1, 5120, 13824, True), 16, 3, 6),
       ((17, 5120, 2560, False), 32, 3, 5), ((48, 5120, 13824, True), 48, 3, 9), ((33, 5120, 2056, False), 48, 3, 9),
       ((64, 20000, 1024, False), 64, 1, 4), ((64, 32000, 4096, True), 64, 1, 4), ((40, 20000, 2056, False), 48, 1, 5),
       ((3, 20000, 4096, False), 16, 1, 6), ((64, 6000, 2056, False), 64, 2, 9), ((31, 4104, 8200, False), 32, 4, 5),
       ((20, 3848, 2056, False), 32, 4, 5), ((9, 3200, 4096, True), 16, 5, 6), ((65, 3000, 4104, False), 80, 5, 8),
       ((3, 2560, 4096, False), 16, 6, 6), ((5, 2048, 16384, False), 16, 6, 12), ((100, 2600, 4104, False), 112, 6, 7),
       ((128, 2568, 4104, False), 128, 6, 6), ((1, 264, 4104, False), 16, 8, 6), ((30, 1920, 4104, False), 32, 8, 5),
       ((130, 2600, 2056, False), 80, 3, 8), ((200, 2600, 4104, False), 112, 3, 7)]
# (M, N, K, e4m3), columns of a tile, split
PAIRS = [((256, 5120, 4104, False), 256, 3), ((300, 2568, 8208, True), 256, 3), ((300, 2048, 4104, False), 192, 3),
         ((300, 2048, 8208, True), 192, 3), ((300, 4104, 8200, False), 256, 2), ((520, 2048, 4104, False), 192, 2),
         ((520, 1000, 4104, False), 256, 4), ((1000, 520, 4104, False), 192, 4), ((1000, 520, 8208, True), 192, 4),
         ((5000, 56, 4104, False), 64, 3), ((4864, 120, 4104, False), 128, 3), ((6000, 56, 4104, False), 64, 2),
         ((8000, 128, 8200, False), 128, 2)]
met = {"few": set(), "pairs": set(), "widths": set()}


def operands(M, N, K, e4m3):
    x, w, b, res = inputs(M, N, K, M + N + K)
    if not e4m3:
        return (x, w, b, res), dict(x=x.to(DEV), w=w.to(DEV)), x.double(), w.double()
    (x, xs), (w, ws) = quantised(x), quantised(w)
    kw = dict(x=x.to(DEV), w=w.to(DEV), x_scale=xs.to(DEV), w_scale=ws.to(DEV))
    return (x, w, b, res), kw, x.double() * xs.double()[:, None], w.double() * ws.double()[:, None]


def check(M, N, K, e4m3):
    (_, _, b, res), kw, x64, w64 = operands(M, N, K, e4m3)
    bd, rd = dev(b, res)
    out, pre = lf.linear(**kw, bias=bd, act="gelu", residual=rd, want_pre=not e4m3)
    plan = lf.last_linear_plan()
    lf.check_device_error()
    check_forward(x64, w64, b, res, "gelu", out, pre)
    over = rd.clone()
    again, _ = lf.linear(**kw, bias=bd, act="gelu", residual=over, out=over)
    assert again is over and torch.equal(over, out) and lf.last_linear_plan() == plan
    plain, _ = lf.linear(**kw)
    lf.check_device_error()
    check_forward(x64, w64, None, None, None, plain)
    return plan


@pytest.mark.parametrize("size,n,split,stages", FEW, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else None)
def test_few_tokens(size, n, split, stages):
    plan = check(*size)
    assert plan["few_tokens"] and plan["tile_n"] == n
    met["few"].add(plan["split"])
    if plan["split"] != split:
        pytest.skip("this device shares a tile between %d, not %d" % (plan["split"], split))
    k_blocks = -(-size[2] // (128 if size[3] else 64))
    assert plan["stages"] == stages and -(-k_blocks // split) > stages


@pytest.mark.parametrize("size,cols,split", PAIRS, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else None)
def test_pairs_that_share_a_tile(size, cols, split):
    plan = check(*size)
    assert not plan["few_tokens"] and plan["stages"] == 0
    if plan["split"] > 1:
        met["pairs"].add(plan["split"])
        met["widths"].add(plan["tile_n"])
    if (plan["tile_n"], plan["split"]) != (cols, split):
        pytest.skip("this device shares tiles of %(tile_n)d columns between %(split)d" % plan)


def test_enough_of_them_were_met(request):
    cases = sum(item.name.startswith(("test_few_tokens[", "test_pairs_that_share_a_tile[")) for item in request.session.items)
    if cases < len(FEW) + len(PAIRS) or "PYTEST_XDIST_WORKER" in os.environ:
        pytest.skip("not all of the cases were run before, in this process")
    assert len(met["few"]) >= 5 and len(met["pairs"]) >= 2 and len(met["widths"]) >= 3, met


@pytest.mark.parametrize("M,N,K", [(300, 2048, 4104), (520, 1000, 4104), (5000, 56, 4104), (1, 5120, 5120), (64, 20000, 1024)])
def test_a_stalled_wait_among_shared_tiles(M, N, K):
    """One pair's (or CTA's) wait runs out while those that share its tile are done."""
    x, w, b, res = inputs(M, N, K)
    xd, wd, bd, rd = dev(x, w, b, res)
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


def test_captured_and_on_two_streams():
    """Shared tiles replayed with new inputs, and two calls at once."""
    for M, N, K in ((300, 2048, 4104), (17, 5120, 2560)):
        x, w, b, res = inputs(M, N, K)
        xd, wd, bd, rd = dev(x, w, b, res)
        lf.linear(xd, wd)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, _ = lf.linear(xd, wd, bias=bd, act="silu", residual=rd)
        for seed in (11, 12):
            x = normal((M, K), seed)
            xd.copy_(x)
            graph.replay()
            lf.check_device_error()
            check_forward(x.double(), w.double(), b, res, "silu", out)
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        got = []
        for i in range(8):
            got.append(lf.linear(xd, wd, bias=bd, act="silu", residual=rd, stream=streams[i % 2])[0])
        torch.cuda.synchronize()
        assert all(torch.equal(g, out) for g in got)
    lf.check_device_error()
