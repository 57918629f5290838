"""The compiled part of the binding without a GPU: it is built, and leaves every call whose
tensors are not on one to the Python functions."""
import pytest
import torch

from layout_folding_gb300 import build as lfbuild
from layout_folding_gb300 import compiled
from test_current_device_cpu import on


@pytest.fixture(scope="module")
def module():
    lfbuild.build()
    module = compiled.load()
    if module is None:
        pytest.skip("no headers of PyTorch or Python here")
    return module


@pytest.mark.parametrize("args", [(), (1, 2), tuple(range(9)), (None,) * 9, (torch.zeros(4, 8),) * 9, (on(0, (4, 8)),) * 9])
def test_calls_that_are_not_taken(module, args):
    for name in compiled._NAMES:
        call = getattr(module, name)
        for n in (len(args), 8, 9, 11):
            assert call(*(args * 2)[:n]) is None


def test_bind_wants_addresses(module):
    with pytest.raises(TypeError):
        module.bind(1, 2)
    with pytest.raises(TypeError):
        module.bind(*"abcdefg")


def test_without_the_module_python_does_the_call(monkeypatch):
    monkeypatch.setattr(compiled, "PATH", compiled.PATH + ".none")
    assert compiled.load() is None
    for name in compiled._NAMES:
        monkeypatch.setattr(compiled, name, compiled._first(name))
    assert compiled.linear(1, 2) is None and compiled.block_norm(1) is None
