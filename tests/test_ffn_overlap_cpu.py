"""add_rms_norm with an output in an input's memory: allowed where rows coincide,
refused before any CUDA call where a row's output would lie over other rows' input."""
import pytest
import torch

import layout_folding_gb300 as lf
from layout_folding_gb300 import build as lfbuild

A, B, C, D_, E = (i << 24 for i in (1, 2, 3, 4, 5))  # distinct, aligned, never used
SHAPE = 2


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("fake addresses, which a call that is not refused would use")
    lfbuild.build()
    return lf.lib()


def status(L, **kw):
    a = dict(x=A, ldx=64, res=B, ldr=64, w=C, h=D_, y=E, scale=None, dtype=0, wdtype=0, ydtype=0, eps=1e-6, M=4, D=64)
    a.update(kw)
    return L.add_rms_norm(*[a[k] for k in ("x", "ldx", "res", "ldr", "w", "h", "y", "scale", "dtype", "wdtype", "ydtype",
                                           "eps", "M", "D")], None)


@pytest.mark.parametrize("kw", [
    dict(y=A, ydtype=3, scale=C),                     # codes over the rows they come from
    dict(y=A, ydtype=3, scale=C, M=1),
    dict(y=A, ydtype=3, scale=C, res=None, h=None),
    dict(y=A, ldx=72),                                # packed rows over pitched ones
    dict(y=A, ldx=72, res=None, h=None),
    dict(h=A, ldx=72),
    dict(h=B, ldr=72),
])
def test_rows_that_do_not_coincide_are_refused(L, kw):
    assert status(L, **kw) == SHAPE


@pytest.mark.parametrize("kw", [
    dict(), dict(y=A), dict(h=A), dict(h=B), dict(y=A, h=B), dict(y=A, res=None, h=None),
    dict(y=A, ldx=72, M=1), dict(h=B, ldr=72, M=1),   # one row has no pitch
    dict(ydtype=3, scale=C, h=A), dict(ydtype=3, scale=C, h=B), dict(h=A, ldr=72), dict(h=B, ldx=72),
])
def test_rows_that_coincide_are_not(L, kw):
    """These go on to the device: any status but a refused argument's."""
    assert status(L, **kw) not in (0, 1, 2, 3)
