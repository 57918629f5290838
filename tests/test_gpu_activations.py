"""The activations of the gated projections and their slopes, value by value over every
bf16 number of magnitude 2^-10 to 128, with one product and exact operands: what is left
is the kernels' own fp32 evaluation and one rounding to bf16.

phi(v) = act(v) / v is off by E(v) phi(v).  An exponential of x is off by the rounding of
its exponent, |x| 2^-23 (the factor log2 e and its product), which phi feels by the share
1 - phi, and ex2.approx, the reciprocal, a polynomial and the last products by at most
2^-20 together:
  silu        x = v                     E = 2^-20 + (1 - phi) |v| 2^-23
  gelu        x = v^2 / 2 (v^2 rounded) E = 2^-20 + (1 - phi) v^2 2^-23
  gelu_tanh   x = 1.6 (v + 0.045 v^3)   E = 2^-20 + (1 - phi) |x| 2^-22  (its four operations)
The slope is phi + v phi'.  phi' = phi (1 - phi) x' of silu and gelu_tanh is off by E + 2^-20,
and by 2^-21 phi x' for the difference 1 - phi near phi = 1; gelu's is the normal density,
off by 2^-20 + v^2 2^-23.  All flush to zero below 2^-126 or where 1 + exp(-x)
passes 2^126: products with |v| and |x'| of up to 2^9 stay below 2^-115.
The rounding to bf16 is half the spacing at the value.
"""
import math

import pytest
import torch

import ffn_reference as ref
import layout_folding_gb300 as lf

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
FLUSH = 2.0 ** -115
C2, A3 = 2 * math.sqrt(2 / math.pi), 0.044715


def values():
    bits = torch.arange(0x3a80, 0x4301, dtype=torch.int32)      # 2^-10 .. 128
    v = torch.cat([bits, bits + 0x8000 - 0x10000]).to(torch.int16).view(BF16)
    return torch.cat([v, torch.zeros(-v.numel() % 8, dtype=BF16)])


def exact(v, name):
    """phi, phi' and what they may be off by, in 64 bits."""
    if name == "gelu":
        p, q = (0.5 * torch.erfc(s * v * math.sqrt(0.5)) for s in (-1, 1))
        dp = torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        return p, dp, (2.0 ** -20 + q * v * v * 2.0 ** -23) * p, (2.0 ** -20 + v * v * 2.0 ** -23) * dp
    x, dx, ex = ((v, torch.ones_like(v), v.abs() * 2.0 ** -23) if name == "silu" else
                 (C2 * (v + A3 * v ** 3), C2 * (1 + 3 * A3 * v * v), C2 * (v + A3 * v ** 3).abs() * 2.0 ** -22))
    p, q = torch.sigmoid(x), torch.sigmoid(-x)
    e = 2.0 ** -20 + q * ex
    return p, p * q * dx, e * p, (e + 2.0 ** -20) * p * q * dx + 2.0 ** -21 * p * dx


def half_spacing(want):
    e = torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -126)))
    return 2.0 ** (e - 8)


def close(got, want, off, what):
    # the rounding is of a value that may lie `off` further out, in the next binade
    bound = off + half_spacing(want.abs() + off) + FLUSH
    bad = ~((got.double().cpu() - want).abs() <= bound)
    assert not bad.any(), "%s: %d off, first %s" % (what, int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_activation_of_every_value(name):
    v = values()
    M, K, F = v.numel(), 8, 8
    x = torch.zeros(M, K, dtype=BF16)
    x[:, 0], x[:, 1] = v, 1.0
    w = torch.zeros(2 * F, K, dtype=BF16)
    w[:F, 0], w[F:, 1] = 1.0, 1.0
    xd, wd = x.to(DEV), w.to(DEV)
    p, _, off, _ = exact(v.double(), name)
    want = v.double() * p
    out, _ = lf.gated_ffn(xd, wd, act=name)                        # the pair kernel
    close(out, want[:, None].expand(M, F), (off * v.double().abs())[:, None], name)
    for i in range(0, M, 16 * 128):                                # the few-token kernel
        few = lf.gated_ffn(xd[i:i + 16 * 128:128].contiguous(), wd, act=name)[0]
        assert torch.equal(few, out[i:i + 16 * 128:128])
    lf.check_device_error()


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_slope_of_every_value(name):
    v = values()
    M, K, F = v.numel() // 8, 8, 8
    g = v.view(M, F)
    gu = torch.cat([g, torch.ones_like(g)], 1).to(DEV)
    one = torch.ones(M, F, dtype=BF16, device=DEV)
    x, w = torch.zeros(M, K, dtype=BF16, device=DEV), torch.zeros(2 * F, K, dtype=BF16, device=DEV)
    dgu = torch.empty_like(gu)
    lf.gated_ffn_backward(one, x, w, gu, act=name, dgu=dgu)
    lf.check_device_error()
    v64 = g.double()
    p, dp, off, off_dp = exact(v64, name)
    close(dgu[:, :F], p + v64 * dp, off + off_dp * v64.abs(), name + " slope")
    close(dgu[:, F:], v64 * p, off * v64.abs(), name)
