"""linear and its gradient: a projection with bias, activation and residual in its
epilogue (include/layoutfold.h is the contract).  Streams, new tensors, the current
device and the missing autograd graph are as in the other operators (see ffn.py)."""
from __future__ import annotations

import functools

import torch

import layout_folding_gb300 as _lf

from . import compiled as _compiled
from . import ffn as _f
from .ffn import ACTIVATIONS, LF_BF16, LF_FP32

LF_ACT_NONE = 3

_BF16, _F32, _FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _act_code(act):
    code = LF_ACT_NONE if act is None else ACTIVATIONS.get(act)
    if code is None:
        raise ValueError("act must be None or one of %s, got %r" % (", ".join(sorted(ACTIVATIONS)), act))
    return code


def _dims(x, w, dtype, stream):
    _f._cuda(x, "x")
    dev = x.get_device()
    _f._on_current(dev, stream)
    _f._require(x, dtype, dev, "x")
    _f._require(w, dtype, dev, "w")
    if w.dim() != 2 or x.dim() == 0 or w.shape[1] != x.shape[-1]:
        raise ValueError("w must be [N, K] with K = x.shape[-1]")
    N, K = w.shape
    return x.numel() // K if K else 0, N, K, dev


def _bias_code(bias, N, dev, name):
    """(lf_dtype, address) of a bias or of its gradient; bf16 or fp32 [N]."""
    if bias is None:
        return LF_BF16, None
    _f._cuda(bias, name)
    if bias.dtype != _BF16 and bias.dtype != _F32:
        raise TypeError("%s must be bf16 or fp32, got %s" % (name, bias.dtype))
    _f._require(bias, bias.dtype, dev, name)
    if bias.numel() != N:
        raise ValueError("%s must hold N = %d elements" % (name, N))
    return (LF_FP32 if bias.dtype == _F32 else LF_BF16), bias.data_ptr()


@functools.lru_cache(maxsize=1024)
def _scratch_bytes(M, N, K):
    return _f._lib().linear_backward_scratch(M, N, K)


def linear(x, w, bias=None, act=None, residual=None, x_scale=None, w_scale=None, want_pre=False, out=None, pre=None,
           stream=None):
    """out = act(x @ w.T + bias) + residual in one kernel, rounded once; act None,
    "silu", "gelu" or "gelu_tanh".

    x [..., K] and w [N, K] in bf16, or both float8_e4m3fn with fp32 scales for each
    token (x_scale, x's leading shape) and each row of w (w_scale [N]); bias [N] in
    bf16 or fp32; residual bf16 [..., N].  Returns (out bf16 [..., N], pre): pre is
    x @ w.T + bias in bf16, which linear_backward takes where there is an activation,
    when want_pre (bf16 operands only), else None.  out may be the residual itself."""
    code = _act_code(act)
    if stream is None and out is None and pre is None:
        made = _compiled.linear(x, w, bias, code, residual, x_scale, w_scale, want_pre)
        if made.__class__ is tuple:
            return made
        if made is not None:
            _lf._check(made, "linear" if x_scale is None else "linear_e4m3")
    scaled = x_scale is not None or w_scale is not None
    M, N, K, dev = _dims(x, w, _FP8 if scaled else _BF16, stream)
    shape = (*x.shape[:-1], N)
    bcode, b_ptr = _bias_code(bias, N, dev, "bias")
    r_ptr = p_ptr = None
    if residual is not None:
        r_ptr = _f._output(residual, _BF16, shape, dev, "residual").data_ptr()
    if scaled:
        if x_scale is None or w_scale is None or want_pre or pre is not None:
            raise ValueError("e4m3 operands take both x_scale and w_scale, and keep no pre")
        _f._require(x_scale, _F32, dev, "x_scale")
        _f._require(w_scale, _F32, dev, "w_scale")
        if x_scale.numel() != M or w_scale.numel() != N:
            raise ValueError("x_scale must hold one scale per row of x and w_scale one per row of w")
    out = _f._new(shape, _BF16, x, stream) if out is None else _f._output(out, _BF16, shape, dev, "out")
    if want_pre or pre is not None:
        pre = _f._new(shape, _BF16, x, stream) if pre is None else _f._output(pre, _BF16, shape, dev, "pre")
        p_ptr = pre.data_ptr()
    if M == 0 and N > 0 and K > 0:
        return out, pre
    L = _f._lib()
    if scaled:
        st = L.linear_e4m3(x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), b_ptr, bcode, code, r_ptr,
                           out.data_ptr(), M, N, K, _f._handle(stream, dev))
    else:
        st = L.linear(x.data_ptr(), w.data_ptr(), b_ptr, bcode, code, r_ptr, out.data_ptr(), p_ptr, M, N, K,
                      _f._handle(stream, dev))
    if st:
        _lf._check(st, "linear_e4m3" if scaled else "linear")
    return out, pre


def linear_backward(dout, x, w, pre=None, act=None, bias=None, want_dx=True, want_dw=True, dx=None, dw=None, dbias=None,
                    dz=None, stream=None):
    """Gradient of linear (bf16): dout [..., N], pre as linear returned it (needed with
    an activation).  Returns (dx [..., K], dw [N, K], dbias [N]); dx and dw are None
    where not wanted, dbias has bias's type and is None without a bias (or a dbias to
    write).  The residual's gradient is dout itself.  With an activation dz [..., N]
    receives the gradient of x @ w.T + bias (pass pre or dout to reuse its memory; a
    new tensor by default)."""
    code = _act_code(act)
    if stream is None and dx is None and dw is None and dbias is None and dz is None:
        made = _compiled.linear_backward(dout, x, w, pre, code, bias, want_dx, want_dw)
        if made.__class__ is tuple:
            return made
        if made is not None:
            _lf._check(made, "linear_backward")
    M, N, K, dev = _dims(x, w, _BF16, stream)
    shape = (*x.shape[:-1], N)
    _f._output(dout, _BF16, shape, dev, "dout")
    pre_ptr = dz_ptr = None
    if act is not None:
        if pre is None:
            raise ValueError("an activation's gradient takes the pre that linear kept")
        pre_ptr = _f._output(pre, _BF16, shape, dev, "pre").data_ptr()
        dz = _f._new(shape, _BF16, x, stream) if dz is None else _f._output(dz, _BF16, shape, dev, "dz")
        dz_ptr = dz.data_ptr()
    elif dz is not None:
        raise ValueError("without an activation dz is dout and is not written")
    if bias is not None:
        _bias_code(bias, N, dev, "bias")
        if dbias is None:
            dbias = _f._new(bias.shape, bias.dtype, x, stream)
        elif dbias.dtype != bias.dtype:
            raise TypeError("dbias must have bias's type")
    bcode, db_ptr = _bias_code(dbias, N, dev, "dbias")
    if want_dx or dx is not None:
        dx = _f._new(x.shape, _BF16, x, stream) if dx is None else _f._output(dx, _BF16, x.shape, dev, "dx")
    if want_dw or dw is not None:
        dw = _f._new(w.shape, _BF16, x, stream) if dw is None else _f._output(dw, _BF16, w.shape, dev, "dw")
    if M == 0 and N > 0 and K > 0:
        return dx, _f._zeroed(dw, stream), _f._zeroed(dbias, stream)
    nbytes = _scratch_bytes(M, N, K)
    scratch = _f._new((nbytes,), torch.uint8, x, stream) if nbytes else None
    st = _f._lib().linear_backward(dout.data_ptr(), x.data_ptr(), w.data_ptr(), pre_ptr, code, dz_ptr,
                                   None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr(), db_ptr,
                                   bcode, None if scratch is None else scratch.data_ptr(), M, N, K,
                                   _f._handle(stream, dev))
    if st:
        _lf._check(st, "linear_backward")
    return dx, dw, dbias
