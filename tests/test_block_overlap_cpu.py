"""linear, block_norm and their gradients with outputs that lie in one another or in memory that
is read beside or after them: refused before any CUDA call.  What the header allows, and
what cannot disturb the result, goes on to the device."""
import pytest
import torch

import layout_folding_gb300 as lf
from layout_folding_gb300 import build as lfbuild

AT = [i << 24 for i in range(1, 17)]  # distinct, aligned, never used, 16 MiB apart
SHAPE = 2


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("fake addresses, which a call that is not refused would use")
    lfbuild.build()
    return lf.lib()


def call(f, names, defaults, kw):
    """f's status with the buffers named in kw at another's address (plus an offset in bytes)."""
    a = dict(zip(defaults, AT))
    a.update({k: v for k, v in defaults.items() if v is not None})
    for k, v in kw.items():
        name, off = v if isinstance(v, tuple) else (v, 0)
        a[k] = a[name] + off if isinstance(name, str) else name
    return f(*[a[k] for k in names], None)


def linear(L, kw):
    names = "x w bias bias_dtype act residual out pre M N K".split()
    return call(L.linear, names, dict(x=None, w=None, bias=None, residual=None, out=None, pre=None, bias_dtype=0, act=0, M=64,
                                      N=64, K=64), kw)


def linear_e4m3(L, kw):
    names = "x xs w ws bias bias_dtype act residual out M N K".split()
    return call(L.linear_e4m3, names, dict(x=None, xs=None, w=None, ws=None, bias=None, residual=None, out=None, bias_dtype=2,
                                           act=3, M=64, N=64, K=64), kw)


def linear_backward(L, kw):
    names = "dout x w pre act dz dx dw db bias_dtype scratch M N K".split()
    return call(L.linear_backward, names, dict(dout=None, x=None, w=None, pre=None, dz=None, dx=None, dw=None, db=None,
                                               scratch=None, act=1, bias_dtype=2, M=64, N=64, K=64), kw)


def block_norm(L, kw):
    names = "x ldx res ldr post pre gate rows gdtype h y scale dtype wdtype ydtype eps beta alpha M D".split()
    return call(L.block_norm, names, dict(x=None, res=None, post=None, pre=None, gate=None, h=None, y=None, scale=0, ldx=64,
                                          ldr=64, rows=2, gdtype=0, dtype=0, wdtype=0, ydtype=0, eps=1e-6, beta=1.0, alpha=1.0,
                                          M=64, D=64), kw)


def block_norm_backward(L, kw):
    names = ("dy x h post pre gate rows gdtype dh dx dres dpost dpre dgate scratch dtype wdtype eps beta alpha M D").split()
    return call(L.block_norm_backward, names, dict(dy=None, x=None, h=None, post=None, pre=None, gate=None, dh=None, dx=None,
                                                   dres=None, dpost=None, dpre=None, dgate=None, scratch=None, rows=2,
                                                   gdtype=0, dtype=0, wdtype=0, eps=1e-6, beta=1.0, alpha=1.0, M=64, D=64), kw)


REFUSED = [
    (linear, [dict(out="x"), dict(out="w"), dict(out="bias"), dict(out=("x", 64)), dict(out=("residual", 128)),
              dict(out=("residual", -128)), dict(pre="x"), dict(pre="w"), dict(pre="bias"), dict(pre="out"),
              dict(pre="residual"), dict(pre=("out", 64 * 64 * 2 - 16)), dict(pre=("out", 16 - 64 * 64 * 2))]),
    (linear_e4m3, [dict(out="x"), dict(out="w"), dict(out="xs"), dict(out="ws"), dict(out="bias"),
                   dict(out=("residual", 16)), dict(xs=("out", 64 * 64 * 2 - 4))]),
    (linear_backward, [dict(dx="x"), dict(dx="w"), dict(dx="dz"), dict(dx="dw"), dict(dw="x"), dict(dw="w"), dict(dw="dz"),
                       dict(dz="x"), dict(dz="w"), dict(dz=("pre", 16)), dict(dz=("dout", -16)), dict(db="dz"), dict(db="x"),
                       dict(db="w"), dict(db="dx"), dict(db="dw"), dict(db="dout"), dict(db="pre"),
                       dict(act=3, dx="dout"), dict(act=3, dw="dout"), dict(act=3, db="dout")]),
    (block_norm, [dict(h="post"), dict(h="pre"), dict(h="gate"), dict(y="post"), dict(y="pre"), dict(y="gate"), dict(h="y"),
                  dict(h=("y", 128)), dict(h=("x", 128)), dict(h=("res", -128)), dict(y=("x", 16)), dict(y=("res", 16)),
                  dict(ydtype=3, scale="h"), dict(ydtype=3, scale="y"), dict(ydtype=3, scale="x"), dict(ydtype=3, scale="post"),
                  dict(ydtype=3, scale="res"), dict(rows=64, h="gate"),
                  dict(dtype=2, wdtype=2, gdtype=2, ydtype=2, h=("y", 64 * 64 * 4 - 16))]),
    (block_norm_backward, [dict(dx="dres"), dict(dx=("dres", 16)), dict(dx="post"), dict(dx="pre"), dict(dx="gate"),
                           dict(dres="post"), dict(dres="pre"), dict(dres="gate"), dict(dx=("x", 16)), dict(dres=("dy", -16)),
                           dict(dpost="dpre"), dict(dpost="dgate"), dict(dpre="dgate"), dict(dpost="post"), dict(dpost="gate"),
                           dict(dgate="gate"), dict(dgate="post"), dict(dpre="post"), dict(dpost="dx"), dict(dgate="dres"),
                           dict(dpre=("dx", 64 * 64 * 2 - 16)), dict(dpost=("dgate", 128))]),
]
ALLOWED = [
    (linear, [{}, dict(out="residual"), dict(out=("residual", 64 * 64 * 2)), dict(pre=("out", 64 * 64 * 2)), dict(x="w"),
              dict(residual="x"), dict(pre=0, out="residual"), dict(bias="w")]),
    (linear_e4m3, [{}, dict(out="residual"), dict(x="w"), dict(xs="ws"), dict(xs=("out", 64 * 64 * 2))]),
    (linear_backward, [{}, dict(dz="pre"), dict(dz="dout"), dict(dx=0, dw="w"), dict(dw=0, dx="x"), dict(dx="dout"),
                       dict(dw="pre"), dict(act=3, dz=0, pre=0), dict(act=3, dz="x", pre="w"), dict(dout="x"), dict(db=0)]),
    (block_norm, [{}, dict(h="x"), dict(h="res"), dict(h="res", y="x"), dict(h="x", y="res"), dict(res="x", h="x"),
                  dict(x="post"), dict(post="pre"), dict(ldx=1 << 13, h=("x", 256)), dict(gate=0, rows=-1),
                  dict(pre=0, y="h"), dict(ydtype=3, scale=("h", 64 * 64 * 2))]),
    (block_norm_backward, [{}, dict(dx="dy", dres="dh"), dict(dx="x", dres="h"), dict(dx="h", dres="x"), dict(dpre="pre"),
                           dict(dpost="dy"), dict(dx=("dres", 64 * 64 * 2)), dict(dh="dy"), dict(gate=0, dgate=0, rows=-1),
                           dict(pre=0, dpre=0, dx="dy"), dict(dpost=0, dpre=0, dgate=0, scratch=0)]),
]


@pytest.mark.parametrize("f,kw", [(f, kw) for f, kws in REFUSED for kw in kws], ids=lambda v: getattr(v, "__name__", str(v)))
def test_refused(L, f, kw):
    assert f(L, {}) not in (0, 1, 2, 3)
    assert f(L, kw) == SHAPE


@pytest.mark.parametrize("f,kw", [(f, kw) for f, kws in ALLOWED for kw in kws], ids=lambda v: getattr(v, "__name__", str(v)))
def test_goes_on_to_the_device(L, f, kw):
    """Any status but a refused argument's."""
    assert f(L, kw) not in (0, 1, 2, 3)


def test_sizes_whose_bytes_pass_63_bits(L):
    most = (1 << 31) - 1
    kw = dict(dtype=2, wdtype=2, gdtype=2, ydtype=2, M=most, D=most, ldx=most, ldr=most, gate=0)
    assert block_norm(L, kw) == SHAPE                             # every buffer reaches over all others
