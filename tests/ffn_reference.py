"""Plain 64-bit CPU implementations of the feed-forward operators, written from
their formulas, and the elementwise error bounds that the tests hold the
kernels to.  Gradients come from torch's autograd on the 64-bit forward."""
import math

import torch

E4M3_MAX = 448.0
F32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half the spacing of the subnormal numbers: the absolute part of a rounding."""
    fi = torch.finfo(dtype)
    return fi.tiny * fi.eps / 2


def norm_factor(h, eps):
    return 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)


def rms_norm(h, weight, eps):
    return h * norm_factor(h, eps) * weight


def row_scale(f):
    amax = f.abs().amax(-1)
    return torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)


def act(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * torch.erfc(-v * math.sqrt(0.5))
    return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))


def gated(x, w, name):
    gu = x @ w.t()
    f = w.shape[0] // 2
    return act(gu[..., :f], name) * gu[..., f:], gu


def gated_from_gu(gu, name):
    f = gu.shape[-1] // 2
    return act(gu[..., :f], name) * gu[..., f:]


def grads(out, inputs, dout):
    return torch.autograd.grad(out, inputs, dout)
