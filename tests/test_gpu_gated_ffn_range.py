"""gated_ffn's e4m3 form with scales whose product is a subnormal fp32 number, and its
activations far from zero.  Bounds as in test_gpu_gated_ffn.py, with the parts that are
particular to a test derived there."""
import pytest
import torch

import ffn_reference as ref
import layout_folding_gb300 as lf

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
HALF = ref.half_step(BF16)
FAST = 2.0 ** -18
ACC = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _device():
    lf.lib()
    torch.cuda.set_device(0)
    lf.check_device_error()
    yield
    torch.cuda.synchronize()
    lf.check_device_error()


@pytest.mark.parametrize("M,F,K", [(1, 8, 16), (3, 136, 80), (48, 520, 2048), (129, 392, 144), (1030, 136, 192),
                                   (130, 264, 2064)])
def test_scales_whose_product_is_subnormal(M, F, K):
    """x_scale about 2^-100 and the gate's w_scale about 2^-46: their product keeps four
    bits in fp32, but with sums of some 2^20 the gate is an ordinary bf16 number, and the up
    projection (w_scale 2^120) brings the output to about 2^-80, far from bf16's ends.  Every
    factor is at least one half of its exponent's range away from fp32's, so K ACC + 4 F32 of
    the sum of magnitudes bounds the projections as for any other scales."""
    g = torch.Generator().manual_seed(M + F + K)

    def codes(*shape):
        return (200 + 248 * torch.rand(*shape, generator=g)).to(E4M3)

    def scales(n, exponent):
        return ((1 + torch.rand(n, generator=g, dtype=torch.float64)) * 2.0 ** exponent).float()
    x, xs = codes(M, K), scales(M, -100)
    w, ws = codes(2 * F, K), torch.cat([scales(F, -46), scales(F, 120)])
    out, _ = lf.gated_ffn(x.to(DEV), w.to(DEV), x_scale=xs.to(DEV), w_scale=ws.to(DEV))
    x64, w64 = x.double() * xs.double()[:, None], w.double() * ws.double()[:, None]
    want, p = ref.gated(x64, w64, "silu")
    d = (K * ACC + 4 * ref.F32) * (x64.abs() @ w64.abs().t())
    gate, up, dg, du = p[:, :F], p[:, F:], d[:, :F], d[:, F:]
    bound = 1.13 * up.abs() * dg + ref.act(gate, "silu").abs() * du + 1.13 * dg * du + (HALF + FAST) * want.abs()
    bad = ~((out.cpu().double() - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float(out.cpu().double()[bad][0] / want[bad][0]))
