"""The compiled part of the binding (csrc/binding.cpp): block_norm, block_norm_backward,
linear and linear_backward of the plain kind, which answer None for any other.  It is
loaded with the first call, and calls the same library; where it is not built (the
machine has no compiler, or no headers of PyTorch or Python) or does not load, every
call takes the Python functions."""
from __future__ import annotations

import ctypes
import importlib.util
import os
import sysconfig
import warnings

import torch

import layout_folding_gb300 as _lf

# of one Python and one PyTorch, whose headers it is built from: another one's is not taken
PATH = os.path.join(_lf.PKG, "_lib", "_binding.%s.torch-%s.so" % (sysconfig.get_config_var("SOABI"), torch.__version__))
_NAMES = ("block_norm", "block_norm_backward", "linear", "linear_backward")
_LIBRARY = ("block_norm", "block_norm_backward", "block_norm_backward_scratch", "linear", "linear_e4m3",
            "linear_backward", "linear_backward_scratch")


def _nothing(*args):
    return None


def load():
    """The compiled module, or None where it or the library is not built, or it does not load."""
    if not (os.path.exists(PATH) and os.path.exists(_lf.LIB_PATH)):
        return None
    spec = importlib.util.spec_from_file_location("layout_folding_gb300._binding", PATH)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        warnings.warn("the compiled part of the binding does not load, its calls are done in Python: %s" % e, RuntimeWarning,
                      stacklevel=2)
        return None
    library = ctypes.CDLL(_lf.LIB_PATH)
    module.bind(*[ctypes.cast(getattr(library, n), ctypes.c_void_p).value for n in _LIBRARY])
    return module


def _first(name):
    """Stands for a function until its first call with a library, which loads the module."""
    def call(*args):
        if not os.path.exists(_lf.LIB_PATH):
            return None  # (the Python function says so; the library may be built yet)
        module = load()
        for n in _NAMES:
            globals()[n] = _nothing if module is None else getattr(module, n)
        return globals()[name](*args)
    return call


block_norm, block_norm_backward, linear, linear_backward = map(_first, _NAMES)
