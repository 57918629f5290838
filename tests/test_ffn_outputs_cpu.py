"""How the feed-forward binding allocates: past the dispatcher where that is cheaper, but
never where a dispatch mode is to see the tensor, and with torch.empty where the cheaper
call does not exist."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from layout_folding_gb300 import ffn

REF = torch.zeros(1)


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.ops = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.ops.append((func.overloadpacket.__name__, tuple(args[0]) if args and not torch.is_tensor(args[0]) else None))
        return func(*args, **(kwargs or {}))


@pytest.fixture
def strided(monkeypatch):
    """Records the cheap allocations."""
    calls = []

    def call(shape, stride, dtype):
        calls.append(shape)
        return torch.empty_strided(shape, stride, dtype=dtype)
    monkeypatch.setattr(ffn, "_strided", call)
    return calls


@pytest.mark.parametrize("shape", [(3, 5), (7,), (0, 4), (4, 0)])
def test_a_dispatch_mode_sees_new_outputs(strided, shape):
    with Seen() as seen:
        t = ffn._new(shape, torch.bfloat16, REF)
    assert seen.ops == [("empty", shape)] and not strided
    assert t.shape == shape and t.dtype == torch.bfloat16 and t.is_contiguous()


@pytest.mark.parametrize("shape", [(3, 5), (7,), (), (0, 4), (4, 0)])
def test_without_one_they_are_allocated_directly(strided, shape):
    t = ffn._new(shape, torch.float32, REF)
    assert strided == [shape] and t.shape == shape and t.is_contiguous()


@pytest.mark.parametrize("shape", [(3, 5), (7,), (), (0, 4), (2, 3, 4)])
def test_where_torch_has_no_such_call(monkeypatch, shape):
    monkeypatch.setattr(ffn, "_strided", None)
    monkeypatch.setattr(ffn, "_dispatch_modes", None)
    t = ffn._new(shape, torch.float16, REF)
    assert t.shape == shape and t.dtype == torch.float16 and t.is_contiguous() and t.device == REF.device
