"""The feed-forward operators' outputs are the same however they are allocated: directly,
under a dispatch mode, and with torch.empty alone."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import layout_folding_gb300 as lf
from layout_folding_gb300 import ffn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Count(TorchDispatchMode):
    made = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.made += func.overloadpacket.__name__ == "empty"
        return func(*args, **(kwargs or {}))


def outputs():
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.empty(*shape, device="cuda").normal_(generator=g).to(BF16)
    x, w, wi, do = normal(9, 64), normal(64), normal(144, 64), normal(9, 72)
    y, h, _ = lf.add_rms_norm(x, w, residual=x)
    q, _, s = lf.add_rms_norm(x, w, fp8=True)
    out, gu = lf.gated_ffn(y, wi, want_gu=True)
    dy, dwi = lf.gated_ffn_backward(do, y, wi, gu)
    dx, dw = lf.add_rms_norm_backward(dy, h, w)
    return [t.float() for t in (y, h, q, s, out, gu, dy, dwi, dx, dw)]


def test_outputs_do_not_depend_on_their_allocation(monkeypatch):
    first = outputs()
    with Count() as count:
        seen = outputs()
    assert count.made >= 4 + 12  # the inputs made above, and at least the calls' outputs, dgu and one scratch
    monkeypatch.setattr(ffn, "_strided", None)
    plain = outputs()
    lf.check_device_error()
    for a, b, c in zip(first, seen, plain):
        assert torch.equal(a, b) and torch.equal(a, c)
