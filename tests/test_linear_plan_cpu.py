"""How linear says which way its last call took, without a GPU."""
import ctypes
import subprocess
import sys

import pytest

import layout_folding_gb300 as lf
from layout_folding_gb300 import build as lfbuild


@pytest.fixture(scope="module")
def L():
    lfbuild.build()
    return lf.lib()


def test_every_output_is_optional(L):
    L.lf_last_linear_plan(None, None, None, None)
    v = ctypes.c_int(-1)
    for i in range(4):
        args = [None] * 4
        args[i] = ctypes.byref(v)
        v.value = -1
        L.lf_last_linear_plan(*args)
        assert v.value >= 0


def test_empty_before_any_call_and_after_a_refused_one(L):
    code = ("import layout_folding_gb300 as lf; L = lf.lib(); A = 1 << 20; nothing = lf.last_linear_plan(); "
            "assert L.linear(A, A, None, 0, 3, None, A, None, 4, 12, 64, None) == 3; "
            "assert nothing == lf.last_linear_plan() == {'few_tokens': False, 'tile_n': 0, 'split': 0, 'stages': 0}")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=lfbuild.ROOT)
    assert r.returncode == 0, r.stderr[-1000:]
