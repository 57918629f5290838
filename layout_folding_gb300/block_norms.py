"""block_norm and its gradient: the norms after and before a block with its gate and
scales (include/layoutfold.h is the contract).  Streams, new tensors, the current device
and the missing autograd graph are as in the other operators (see ffn.py)."""
from __future__ import annotations

import functools

import torch

import layout_folding_gb300 as _lf

from . import compiled as _compiled
from . import ffn as _f
from .ffn import LF_BF16, LF_E4M3, LF_FP32

_F32, _FP8 = torch.float32, torch.float8_e4m3fn
_Tensor = torch.Tensor


def _parameters(post, pre, code, dtype, D, dev):
    """wdtype of the two weights, which are of one type."""
    wcode = code
    if post is not None:
        wcode = _f._weight_type(post, code, dtype, D, dev)
    if pre is not None:
        pcode = _f._weight_type(pre, code, dtype, D, dev)
        if post is not None and pcode != wcode:
            raise TypeError("post and pre must be of one type")
        wcode = pcode
    return wcode


def _gate(gate, shape, M, dtype, dev):
    """(gate_rows, lf_dtype, address) of the gate of rows of `shape`."""
    if gate is None:
        return 0, LF_BF16, None
    code = _f._CODES.get(gate.dtype, -1) if isinstance(gate, _Tensor) else -1
    if code < 0 or (gate.dtype != dtype and code != LF_FP32):
        raise TypeError("gate must be a %s or float32 tensor" % dtype)
    if gate.get_device() != dev or not gate.is_contiguous():
        _f._require(gate, gate.dtype, dev, "gate")
    gs = tuple(gate.shape)
    if not gs or gs[-1] != shape[-1]:
        raise ValueError("gate must hold rows of D = %d elements" % shape[-1])
    rows = 1
    for n in gs[:-1]:
        rows *= n
    if len(gs) > 2:
        # one row for each index of x's first dimensions: [B, 1, D] for x [B, S, D]
        lead = list(gs[:-1])
        while lead and lead[-1] == 1:
            lead.pop()
        if len(gs) != len(shape) or tuple(lead) != tuple(shape[:len(lead)]):
            raise ValueError("gate must be [D], [G, D], or x's shape with 1 in place of its last dimensions but D")
    if M > 0 and (rows == 0 or M % rows):
        raise ValueError("gate must have a number of rows that divides x's %d" % M)
    return rows, code, gate.data_ptr()


@functools.lru_cache(maxsize=1024)
def _scratch_bytes(M, D, code, gate_rows):
    return _f._lib().block_norm_backward_scratch(M, D, code, gate_rows)


def block_norm(x, residual, post=None, pre=None, gate=None, branch_scale=1.0, residual_scale=1.0, eps=1e-6, fp8=False,
               h=None, y=None, scale=None, stream=None):
    """The norm after a block, its gate, the scaled addition to the stream and the norm
    before the next block, over the last dimension:
      p = x / sqrt(mean(x^2) + eps) * post                           (x without post)
      h = residual_scale * residual + branch_scale * (p * gate)      (rounded to x's type)
      f = h / sqrt(mean(h^2) + eps) * pre
    Returns (y, h, scale): y = f in x's type with scale None; with fp8 y =
    float8_e4m3fn(f / scale) and scale fp32 of x's leading shape (add_rms_norm's); without
    pre (None, h, None).
    x, residual: bf16, fp16 or fp32 [..., D], contiguous or 2-D slices of wider rows; post,
    pre [D] of one type, x's or fp32; gate in x's type or fp32: [D], [G, D] (each row for
    the next M / G of x's M rows in order), or x's shape with 1 in place of its last
    dimensions but D.  h may be passed as residual or x, to update a contiguous stream in
    place."""
    if stream is None and h is None and y is None and scale is None:
        made = _compiled.block_norm(x, residual, post, pre, gate, branch_scale, residual_scale, eps, fp8)
        if made.__class__ is tuple:
            return made
        if made is not None:
            _lf._check(made, "block_norm")
    dtype = getattr(x, "dtype", None)
    code = _f._CODES.get(dtype, -1)
    dev = x.get_device() if code >= 0 else -1
    shape = x.shape if dev >= 0 else ()
    if not shape:
        _f._stream_type(x, "x")  # raises
    _f._on_current(dev, stream)
    D = shape[-1]
    M = x.numel() // D if D else 0
    ldx = D if x.is_contiguous() else _f._pitch(x, "x")
    if not isinstance(residual, _Tensor) or residual.dtype != dtype or residual.get_device() != dev:
        _f._cuda(residual, "residual")
        raise TypeError("residual must be %s on cuda:%d" % (dtype, dev))
    if residual.shape != shape:
        raise ValueError("residual must have x's shape")
    ldr = D if residual.is_contiguous() else _f._pitch(residual, "residual")
    wcode = _parameters(post, pre, code, dtype, D, dev)
    rows, gcode, g_ptr = _gate(gate, shape, M, dtype, dev)
    h = _f._new(shape, dtype, x, stream) if h is None else _f._output(h, dtype, shape, dev, "h")
    y_ptr = s_ptr = None
    if scale is not None and not fp8:
        raise ValueError("scale is written only with fp8")
    if pre is None:
        if fp8 or y is not None:
            raise ValueError("without pre there is no y and no fp8")
    else:
        ytype = _FP8 if fp8 else dtype
        y = _f._new(shape, ytype, x, stream) if y is None else _f._output(y, ytype, shape, dev, "y")
        y_ptr = y.data_ptr()
        if fp8:
            scale = (_f._new(shape[:-1], _F32, x, stream) if scale is None
                     else _f._output(scale, _F32, shape[:-1], dev, "scale"))
            s_ptr = scale.data_ptr()
    if M > 0 or D == 0:
        st = _f._lib().block_norm(x.data_ptr(), ldx, residual.data_ptr(), ldr, None if post is None else post.data_ptr(),
                                  None if pre is None else pre.data_ptr(), g_ptr, rows, gcode, h.data_ptr(), y_ptr, s_ptr,
                                  code, wcode, LF_E4M3 if fp8 else code, eps, branch_scale, residual_scale, M, D,
                                  _f._handle(stream, dev))
        if st:
            _lf._check(st, "block_norm")
    return y, h, scale


def block_norm_backward(dy, x, h, post=None, pre=None, gate=None, dh=None, branch_scale=1.0, residual_scale=1.0, eps=1e-6,
                        want_dparams=True, dx=None, dresidual=None, dpost=None, dpre=None, dgate=None, stream=None):
    """Gradient of block_norm: dy and dh (or None) arrive at its y and h; x, h, post, pre,
    gate and the scales are block_norm's.  dy, x, h, dh contiguous [..., D] of one type; dy
    and h are not read (None allowed) without pre, where dh is needed.  Returns (dx,
    dresidual, dpost, dpre, dgate): the first two in x's type, the others in their
    parameter's type and shape, None for a parameter that is None, and with want_dparams
    False for those that are not given a tensor.  dx and dresidual may each be passed as
    dy, x, h or dh, to reuse its memory."""
    if stream is None and dx is None and dresidual is None and dpost is None and dpre is None and dgate is None:
        made = _compiled.block_norm_backward(dy, x, h, post, pre, gate, dh, branch_scale, residual_scale, eps, want_dparams)
        if made.__class__ is tuple:
            return made
        if made is not None:
            _lf._check(made, "block_norm_backward")
    dtype = getattr(x, "dtype", None)
    code = _f._CODES.get(dtype, -1)
    dev = x.get_device() if code >= 0 else -1
    shape = x.shape if dev >= 0 else ()
    if not shape:
        _f._stream_type(x, "x")  # raises
    _f._on_current(dev, stream)
    _f._require(x, dtype, dev, "x")
    D = shape[-1]
    M = x.numel() // D if D else 0
    wcode = _parameters(post, pre, code, dtype, D, dev)
    rows, gcode, g_ptr = _gate(gate, shape, M, dtype, dev)
    ptrs = []
    for t, name, needed in ((dy, "dy", pre is not None), (h, "h", pre is not None), (dh, "dh", pre is None)):
        if t is None:
            if needed:
                raise ValueError("%s is needed %s pre" % (name, "without" if pre is None else "with"))
            ptrs.append(None)
            continue
        _f._require(t, dtype, dev, name)
        if t.shape != shape:
            raise ValueError("%s must have x's shape" % name)
        ptrs.append(t.data_ptr())
    dx = _f._new(shape, dtype, x, stream) if dx is None else _f._output(dx, dtype, shape, dev, "dx")
    dresidual = (_f._new(shape, dtype, x, stream) if dresidual is None
                 else _f._output(dresidual, dtype, shape, dev, "dresidual"))
    grads = []
    for g, param, name in ((dpost, post, "dpost"), (dpre, pre, "dpre"), (dgate, gate, "dgate")):
        if param is None:
            if g is not None:
                raise ValueError("%s is written only with its parameter" % name)
        elif g is not None:
            _f._output(g, param.dtype, param.shape, dev, name)
        elif want_dparams:
            g = _f._new(param.shape, param.dtype, x, stream)
        grads.append(g)
    if M == 0 and D > 0:
        return (dx, dresidual, *[_f._zeroed(g, stream) for g in grads])
    scratch = None
    if any(g is not None for g in grads):
        scratch = _f._new((_scratch_bytes(M, D, code, rows),), torch.uint8, x, stream)
    st = _f._lib().block_norm_backward(ptrs[0], x.data_ptr(), ptrs[1], None if post is None else post.data_ptr(),
                                       None if pre is None else pre.data_ptr(), g_ptr, rows, gcode, ptrs[2], dx.data_ptr(),
                                       dresidual.data_ptr(), *[None if g is None else g.data_ptr() for g in grads],
                                       None if scratch is None else scratch.data_ptr(), code, wcode, eps, branch_scale,
                                       residual_scale, M, D, _f._handle(stream, dev))
    if st:
        _lf._check(st, "block_norm_backward")
    return (dx, dresidual, *grads)
