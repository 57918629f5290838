"""The compiled part of the binding (csrc/binding.cpp): block_norm, block_norm_backward,
linear and linear_backward of the plain kind, which answer None for any other.  It is
loaded with the first call, and calls the same library; where it is not built (the
machine has no headers of PyTorch or Python), every call takes the Python functions."""
from __future__ import annotations

import ctypes
import importlib.util
import os

import layout_folding_gb300 as _lf

PATH = os.path.join(_lf.PKG, "_lib", "_binding.so")
_NAMES = ("block_norm", "block_norm_backward", "linear", "linear_backward")
_LIBRARY = ("block_norm", "block_norm_backward", "block_norm_backward_scratch", "linear", "linear_e4m3",
            "linear_backward", "linear_backward_scratch")


def _nothing(*args):
    return None


def load():
    """The compiled module, or None where it or the library is not built."""
    if not (os.path.exists(PATH) and os.path.exists(_lf.LIB_PATH)):
        return None
    import torch  # noqa: F401  (whose libraries the module uses)
    spec = importlib.util.spec_from_file_location("layout_folding_gb300._binding", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    library = ctypes.CDLL(_lf.LIB_PATH)
    module.bind(*[ctypes.cast(getattr(library, n), ctypes.c_void_p).value for n in _LIBRARY])
    return module


def _first(name):
    """Stands for a function until its first call, which loads the module."""
    def call(*args):
        module = load()
        for n in _NAMES:
            globals()[n] = _nothing if module is None else getattr(module, n)
        return globals()[name](*args)
    return call


block_norm, block_norm_backward, linear, linear_backward = map(_first, _NAMES)
