"""The slopes of the activations where a kept projection is far from zero, up to bf16's
largest number: 1 or 0 there.  |v| >= 1e4, so 1 - phi(v) and v phi'(v) are below exp(-9000)
in 64 bits, and every result is exact: dout or 0, and for the other projection's gradient
dout act(v), which is dout v or 0."""
import pytest
import torch

import layout_folding_gb300 as lf

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
FAR = [1e4, 1e9, 1e13, 1e18, 1.2e18, 1e19, 4e19, 5.2e19, 7e19, 1e20, 1e25, 1e30, 2e38, float(torch.finfo(BF16).max)]


def far():
    v = torch.tensor(FAR, dtype=BF16)
    return torch.cat([v, -v, v[:4]]).view(4, 8).to(DEV)


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_slope_of_a_projection(name):
    pre = far()
    M, N, K = 4, 8, 16
    dout = torch.linspace(-2, 2, M * N).to(BF16).view(M, N).to(DEV)
    x, w = torch.ones(M, K, dtype=BF16, device=DEV), torch.zeros(N, K, dtype=BF16, device=DEV)
    w[:, 0] = 1.0
    dz = torch.empty_like(dout)
    want = torch.where(pre > 0, dout, torch.zeros_like(dout))
    dx, dw, db = lf.linear_backward(dout, x, w, pre=pre, act=name, bias=torch.zeros(N, device=DEV), dz=dz)
    lf.check_device_error()
    assert torch.equal(dz, want)
    # sums of at most eight bf16 numbers of like size, in fp32
    torch.testing.assert_close(dx[:, 0], want.double().sum(1).to(BF16), rtol=2.0 ** -7, atol=2.0 ** -20)
    torch.testing.assert_close(dw[:, 3], want.double().sum(0).to(BF16), rtol=2.0 ** -7, atol=2.0 ** -20)
    torch.testing.assert_close(db, want.double().sum(0).float(), rtol=2.0 ** -20, atol=2.0 ** -20)


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_slope_of_gated_projections(name):
    g = far()
    M, F = g.shape
    gu = torch.cat([g, torch.full_like(g, 0.5)], 1)
    dout = torch.ones(M, F, dtype=BF16, device=DEV)
    x, w = torch.zeros(M, 8, dtype=BF16, device=DEV), torch.zeros(2 * F, 8, dtype=BF16, device=DEV)
    dgu = torch.empty_like(gu)
    lf.gated_ffn_backward(dout, x, w, gu, act=name, dgu=dgu)
    lf.check_device_error()
    assert torch.equal(dgu[:, :F], torch.where(g > 0, 0.5 * dout, torch.zeros_like(dout)))
    assert torch.equal(dgu[:, F:], torch.where(g > 0, g, torch.zeros_like(g)))
