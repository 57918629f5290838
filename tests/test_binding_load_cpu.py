"""What the compiled part of the binding does where it cannot be loaded, without a GPU."""
import os
import sysconfig
import warnings

import pytest
import torch

import layout_folding_gb300 as lf
from layout_folding_gb300 import build as lfbuild
from layout_folding_gb300 import compiled


@pytest.fixture
def fresh(monkeypatch, tmp_path):
    """The functions as they stand before their first call, a library, and no compiled module yet."""
    lfbuild.build()
    monkeypatch.setattr(compiled, "PATH", str(tmp_path / "_binding.so"))
    for name in compiled._NAMES:
        monkeypatch.setattr(compiled, name, compiled._first(name))
    return tmp_path


def test_the_name_says_what_it_is_built_for():
    assert lfbuild.BINDING_PATH == compiled.PATH
    name = os.path.basename(compiled.PATH)
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name


@pytest.mark.parametrize("content", [b"", b"\x7fELF\x02\x01\x01", b"not a library"])
def test_a_module_that_does_not_load_is_said_once_and_python_does_the_calls(fresh, content):
    (fresh / "_binding.so").write_bytes(content)
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.warns(RuntimeWarning, match="does not load") as said:
        with pytest.raises(TypeError, match="CUDA tensor"):
            lf.linear(x, x)
    assert len(said) == 1
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        for call in (lambda: lf.linear(x, x), lambda: lf.linear_backward(x, x, x), lambda: lf.block_norm(x, x),
                     lambda: lf.block_norm_backward(x, x, x)):
            with pytest.raises(TypeError, match="CUDA tensor"):
                call()


def test_a_library_that_is_built_after_the_first_call_is_taken(fresh, monkeypatch):
    if not os.path.exists(lfbuild.BINDING_PATH):
        pytest.skip("the compiled part of the binding is not built here")
    there = lf.LIB_PATH
    monkeypatch.setattr(lf, "LIB_PATH", str(fresh / "none.so"))
    assert compiled.linear(*range(8)) is None and compiled.block_norm(*range(9)) is None
    monkeypatch.setattr(lf, "LIB_PATH", there)
    monkeypatch.setattr(compiled, "PATH", lfbuild.BINDING_PATH)
    assert compiled.linear(*range(8)) is None
    assert all("built-in" in repr(getattr(compiled, name)) for name in compiled._NAMES)
