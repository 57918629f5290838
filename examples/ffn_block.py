"""A feed-forward block on this library's operators, trained and then used for
generation.

    h = x + residual;  y = rms_norm(h);  a = act(y Wg^T) * (y Wu^T);  out = h + a Wd^T

Training runs in bf16 and hands gradients on explicitly (no autograd graph):
add_rms_norm -> gated_ffn -> gemm_nt forward, and back through two folded
products of the down projection, gated_ffn_backward and add_rms_norm_backward,
the stream's own gradient entering the latter as `dh`.  Generation quantises the
gated projections once to e4m3 with a scale for each output channel; every
token's norm then writes e4m3 with a scale for the token.

    python examples/ffn_block.py [--tokens 512] [--hidden 1024] [--ffn 2816] [--steps 20]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import layout_folding_gb300 as lf  # noqa: E402

E4M3_MAX = 448.0


class Block:
    def __init__(self, hidden, ffn, act="silu", eps=1e-6, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return torch.empty(*shape, device="cuda").normal_(0.0, std, generator=g).bfloat16()
        self.act, self.eps = act, eps
        self.norm = torch.ones(hidden, device="cuda").bfloat16()
        self.w_in = normal(2 * ffn, hidden, std=1 / math.sqrt(hidden))  # gate rows, then up rows
        self.w_out = normal(hidden, ffn, std=1 / math.sqrt(ffn))

    def forward(self, x, residual):
        """Returns the block's output (to be added to the stream h) and what backward needs."""
        y, h, _ = lf.add_rms_norm(x, self.norm, residual=residual, eps=self.eps)
        a, gu = lf.gated_ffn(y, self.w_in, act=self.act, want_gu=True)
        return lf.gemm_nt(a, self.w_out), h, (y, h, gu, a)

    def backward(self, dout, dh, kept):
        """dout, dh: the gradients of forward's output and of h.  Returns the gradient of
        x (and of residual: they are the same) and of norm, w_in, w_out."""
        y, h, gu, a = kept
        da = lf.gemm_layout(dout, self.w_out, w_mn=True)                # dout . Wd, Wd read as stored
        dw_out = lf.gemm_layout(dout, a, x_mn=True, w_mn=True)          # dout^T . a
        dy, dw_in = lf.gated_ffn_backward(da, y, self.w_in, gu, act=self.act, dgu=gu)
        dx, dnorm = lf.add_rms_norm_backward(dy, h, self.norm, dh=dh, eps=self.eps)
        return dx, dnorm, dw_in, dw_out

    def quantise(self):
        """w_in in e4m3 with a scale for each row, for generation."""
        w = self.w_in.float()
        scale = w.abs().amax(1) / E4M3_MAX
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        self.w_in8, self.w_in_scale = (w / scale[:, None]).to(torch.float8_e4m3fn), scale

    def generate(self, x, residual):
        """One step for a few tokens: the stream is updated in place."""
        y8, h, scale = lf.add_rms_norm(x, self.norm, residual=residual, eps=self.eps, fp8=True, h=residual)
        a, _ = lf.gated_ffn(y8, self.w_in8, act=self.act, x_scale=scale, w_scale=self.w_in_scale)
        return lf.gemm_nt(a, self.w_out), h


def train(block, x, residual, target, steps, lr):
    """Plain gradient descent on the mean squared error of h + out; returns the losses."""
    losses = []
    n = x.numel()
    for _ in range(steps):
        out, h, kept = block.forward(x, residual)
        diff = (h.float() + out.float()) - target
        losses.append(float((diff * diff).sum()) / n)
        grad = (2.0 * diff).bfloat16()
        _, dnorm, dw_in, dw_out = block.backward(grad, grad, kept)
        for w, dw in ((block.norm, dnorm), (block.w_in, dw_in), (block.w_out, dw_out)):
            w.copy_((w.float() - lr / n * dw.float()).bfloat16())
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--ffn", type=int, default=2816)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, residual = (torch.empty(a.tokens, a.hidden, device="cuda").normal_(0.0, s, generator=g).bfloat16()
                   for s in (0.5, 1.0))
    teacher, block = Block(a.hidden, a.ffn, seed=2), Block(a.hidden, a.ffn, seed=3)
    out, h, _ = teacher.forward(x, residual)
    target = h.float() + out.float()
    losses = train(block, x, residual, target, a.steps, lr=0.1 * a.hidden)
    block.quantise()
    out16, _, _ = block.forward(x[:4], residual[:4])
    out8, _ = block.generate(x[:4], residual[:4].clone())
    off = float((out8.float() - out16.float()).norm() / out16.float().norm())
    lf.check_device_error()
    print("loss %.4f -> %.4f in %d steps; e4m3 generation is %.3f off bf16" % (losses[0], losses[-1], a.steps, off))
    return losses, off


if __name__ == "__main__":
    main()
