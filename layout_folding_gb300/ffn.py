"""The feed-forward operators of the binding: add_rms_norm, gated_ffn and their
gradients (include/layoutfold.h is the contract, as for the rest).  Gradients are
calls of their own: no autograd graph is recorded through any operator here.

One token's norm runs for about 3 us on the GPU, so the host's share is kept
small: checks are attribute reads, the stream is read as a raw handle, and
outputs come from _new (between launches an output costs 4 us from
Tensor.new_empty, 2 us from torch.empty, 1 us from the allocation call that
torch's compiled programs use; one buffer cut into views costs more than three
tensors).  With `stream` the call runs there, its new tensors are memory of that
stream, and ordering it against the current stream is the caller's, as for every
other operator.  Tensors and stream are of the current device.
"""
from __future__ import annotations

import functools

import torch

import layout_folding_gb300 as _lf

LF_BF16, LF_FP16, LF_FP32, LF_E4M3 = 0, 1, 2, 3
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}

_BF16, _F32, _FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_CODES = {torch.bfloat16: LF_BF16, torch.float16: LF_FP16, torch.float32: LF_FP32}
# the current stream as an integer, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_L = None
try:
    # contiguous tensors on the current device, without the general argument parser -- and
    # without the dispatcher, so only while no dispatch mode (one that tracks allocations,
    # say) wants to see them
    from torch._C._dynamo.guards import _empty_strided_cuda as _strided
    _dispatch_modes = torch._C._len_torch_dispatch_stack
except (ImportError, AttributeError):  # pragma: no cover
    _strided = _dispatch_modes = None
# the current device as an integer (the calls have a CUDA tensor in hand, so CUDA is initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on_current(device, stream):
    """Kernels are launched on the current device, with its tensor maps, limits and
    error word: tensors or a stream of another one are refused."""
    current = _current_device()
    if device != current:
        raise ValueError("the tensors are on cuda:%d and the current device is cuda:%d" % (device, current))
    if stream is not None and stream.device.index != current:
        raise ValueError("stream is of cuda:%d and the current device is cuda:%d" % (stream.device.index, current))


def _new_on(stream, shape, dtype, device):
    """The same for a call on a stream of its own: memory whose earlier users, if
    any, ran on that stream (work that the current stream still has to do may
    read anything else that it freed), and that is not handed out again before
    the current stream is done with it either."""
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if current != stream:
        t.record_stream(current)
    return t


def _new(shape, dtype, ref, stream=None):
    """A contiguous tensor of `shape` on ref's device, the current one."""
    if stream is not None:
        return _new_on(stream, shape, dtype, ref.device)
    n = len(shape)
    if _strided is None or n > 2 or _dispatch_modes():
        return torch.empty(shape, dtype=dtype, device=ref.device)
    if n == 2:
        return _strided(tuple(shape), (shape[1] or 1, 1), dtype)
    return _strided(tuple(shape), (1,) if n else (), dtype)


def _lib():
    global _L
    if _L is None:
        _L = _lf.lib()
    return _L


@functools.lru_cache(maxsize=1024)
def _norm_scratch(M, D):
    return _lib().add_rms_norm_backward_scratch(M, D)


@functools.lru_cache(maxsize=1024)
def _gated_scratch(M, F, K):
    return _lib().gated_ffn_backward_scratch(M, F, K)


def _handle(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


_Tensor = torch.Tensor


def _cuda(t, name):
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)


def _require(t, dtype, device, name):
    """t: a contiguous CUDA tensor of `dtype` on `device`."""
    if isinstance(t, _Tensor) and t.dtype == dtype and t.get_device() == device and t.is_contiguous():
        return
    _cuda(t, name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("%s must be on cuda:%d" % (name, device))


def _output(t, dtype, shape, device, name):
    _require(t, dtype, device, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be %s" % (name, tuple(shape)))
    return t


def _stream_type(t, name):
    """(lf_dtype, device) of a tensor that holds rows of the stream."""
    _cuda(t, name)
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be bf16, fp16 or fp32, got %s" % (name, t.dtype))
    if t.dim() == 0:
        raise ValueError("%s must have at least one dimension" % name)
    return code, t.get_device()


def _weight_type(weight, code, dtype, D, device):
    wcode = _CODES.get(weight.dtype, -1) if isinstance(weight, _Tensor) else -1
    if wcode != code and wcode != LF_FP32:
        raise TypeError("weight must be a %s or float32 tensor" % dtype)
    if weight.get_device() != device or not weight.is_contiguous():
        _require(weight, weight.dtype, device, "weight")
    if weight.numel() != D:
        raise ValueError("weight must hold D = %d elements" % D)
    return wcode


def _pitch(t, name):
    """Row pitch of [..., D]: contiguous, or 2-D with unit column stride (a slice
    of wider rows)."""
    if t.is_contiguous():
        return t.shape[-1]
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1) or (t.stride(0) < t.shape[1] and t.shape[0] > 1):
        raise ValueError("%s must be contiguous, or 2-D with unit column stride and rows that do not overlap" % name)
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _activation(act):
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError("act must be one of %s, got %r" % (", ".join(sorted(ACTIVATIONS)), act))
    return code


def _zeroed(t, stream):
    """t filled with zeros: the weight gradient of no rows."""
    if t is not None:
        with torch.cuda.stream(stream):
            t.zero_()
    return t


def add_rms_norm(x, weight, residual=None, eps=1e-6, fp8=False, h=None, y=None, scale=None, stream=None):
    """Residual addition and root-mean-square norm over the last dimension.

    h = x + residual (rounded to x's type; x itself when residual is None),
    f = h / sqrt(mean(h^2) + eps) * weight.  Returns (y, h, scale): y = f in x's
    type with scale None, or with fp8 y = float8_e4m3fn(f / scale) and scale fp32
    of x's leading shape (one per row: max|f| / 448, 1 where that is 0).  No
    rows at all give empty outputs (and zero weight gradients) here and below.
    x, residual: bf16, fp16 or fp32 [..., D], contiguous or 2-D slices of wider
    rows; weight [D] in x's type or fp32.  h may be passed as residual (or x)
    itself, to update a contiguous stream in place."""
    dtype = getattr(x, "dtype", None)
    code = _CODES.get(dtype, -1)
    dev = x.get_device() if code >= 0 else -1
    shape = x.shape if dev >= 0 else ()
    if not shape:
        _stream_type(x, "x")  # raises
    _on_current(dev, stream)
    D = shape[-1]
    M = x.numel() // D if D else 0
    ldx = D if x.is_contiguous() else _pitch(x, "x")
    wcode = _weight_type(weight, code, dtype, D, dev)
    ldr = 0
    r_ptr = h_ptr = s_ptr = None
    if residual is not None:
        if not isinstance(residual, _Tensor) or residual.dtype != dtype or residual.get_device() != dev:
            _cuda(residual, "residual")
            raise TypeError("residual must be %s on cuda:%d" % (dtype, dev))
        if residual.shape != shape:
            raise ValueError("residual must have x's shape")
        ldr = D if residual.is_contiguous() else _pitch(residual, "residual")
        r_ptr = residual.data_ptr()
        h = _new(shape, dtype, x, stream) if h is None else _output(h, dtype, shape, dev, "h")
        h_ptr = h.data_ptr()
    elif h is not None:
        raise ValueError("h is written only where a residual is added")
    if fp8:
        y = _new(shape, _FP8, x, stream) if y is None else _output(y, _FP8, shape, dev, "y")
        scale = (_new(shape[:-1], _F32, x, stream) if scale is None
                 else _output(scale, _F32, shape[:-1], dev, "scale"))
        s_ptr = scale.data_ptr()
    else:
        if scale is not None:
            raise ValueError("scale is written only with fp8")
        y = _new(shape, dtype, x, stream) if y is None else _output(y, dtype, shape, dev, "y")
    if M > 0 or D == 0:
        st = _lib().add_rms_norm(x.data_ptr(), ldx, r_ptr, ldr, weight.data_ptr(), h_ptr, y.data_ptr(), s_ptr, code,
                                 wcode, LF_E4M3 if fp8 else code, eps, M, D, _handle(stream, dev))
        if st:
            _lf._check(st, "add_rms_norm")
    return y, (x if residual is None else h), scale


def add_rms_norm_backward(dy, h, weight, dh=None, eps=1e-6, want_dweight=True, dx=None, dweight=None, stream=None):
    """Gradient of add_rms_norm.  dy, h (add_rms_norm's) and dh (the gradient
    arriving at h by other ways, or None) contiguous [..., D] of one type.
    Returns (dx, dweight): dx in h's type is the gradient of x and of residual,
    dweight has weight's type (None when not wanted)."""
    dtype = getattr(h, "dtype", None)
    code = _CODES.get(dtype, -1)
    dev = h.get_device() if code >= 0 else -1
    shape = h.shape if dev >= 0 else ()
    if not shape:
        _stream_type(h, "h")  # raises
    _on_current(dev, stream)
    _require(h, dtype, dev, "h")
    _require(dy, dtype, dev, "dy")
    if dy.shape != shape:
        raise ValueError("dy must have h's shape")
    D = shape[-1]
    M = h.numel() // D if D else 0
    wcode = _weight_type(weight, code, dtype, D, dev)
    dh_ptr = dw_ptr = scratch = scratch_ptr = None
    if dh is not None:
        _require(dh, dtype, dev, "dh")
        if dh.shape != shape:
            raise ValueError("dh must have h's shape")
        dh_ptr = dh.data_ptr()
    dx = _new(shape, dtype, h, stream) if dx is None else _output(dx, dtype, shape, dev, "dx")
    if want_dweight or dweight is not None:
        dweight = (_new(weight.shape, weight.dtype, h, stream) if dweight is None
                   else _output(dweight, weight.dtype, weight.shape, dev, "dweight"))
        if M > 0:
            scratch = _new((_norm_scratch(M, D),), torch.uint8, h, stream)
            dw_ptr, scratch_ptr = dweight.data_ptr(), scratch.data_ptr()
    if M == 0 and D > 0:
        return dx, _zeroed(dweight, stream)
    st = _lib().add_rms_norm_backward(dy.data_ptr(), h.data_ptr(), weight.data_ptr(), dh_ptr, dx.data_ptr(), dw_ptr,
                                      scratch_ptr, code, wcode, eps, M, D, _handle(stream, dev))
    if st:
        _lf._check(st, "add_rms_norm_backward")
    return dx, dweight


def _gated_dims(x, w, dtype, stream):
    _cuda(x, "x")
    dev = x.get_device()
    _on_current(dev, stream)
    _require(x, dtype, dev, "x")
    _require(w, dtype, dev, "w")
    if w.dim() != 2 or x.dim() == 0 or w.shape[1] != x.shape[-1] or w.shape[0] % 2:
        raise ValueError("w must be [2F, K] with K = x.shape[-1]: the gate's rows, then the up projection's")
    K, F = w.shape[1], w.shape[0] // 2
    return x.numel() // K if K else 0, F, K, dev


def gated_ffn(x, w, act="silu", x_scale=None, w_scale=None, want_gu=False, out=None, gu=None, stream=None):
    """The gated projections: out = act(x @ Wg.T) * (x @ Wu.T), w [2F, K] holding
    Wg's rows and then Wu's; act "silu", "gelu" or "gelu_tanh".

    x [..., K] and w in bf16, or both float8_e4m3fn with fp32 scales for each
    token (x_scale, x's leading shape) and each row of w (w_scale [2F]).
    Returns (out bf16 [..., F], gu): gu is bf16 [..., 2F], the two projections
    that gated_ffn_backward takes, when want_gu (bf16 operands only), else None."""
    code = _activation(act)
    scaled = x_scale is not None or w_scale is not None
    M, F, K, dev = _gated_dims(x, w, _FP8 if scaled else _BF16, stream)
    lead = x.shape[:-1]
    out = (_new((*lead, F), _BF16, x, stream) if out is None
           else _output(out, _BF16, (*lead, F), dev, "out"))
    if scaled:
        if x_scale is None or w_scale is None or want_gu or gu is not None:
            raise ValueError("e4m3 operands take both x_scale and w_scale, and keep no gu")
        _require(x_scale, _F32, dev, "x_scale")
        _require(w_scale, _F32, dev, "w_scale")
        if x_scale.numel() != M or w_scale.numel() != 2 * F:
            raise ValueError("x_scale must hold one scale per row of x and w_scale one per row of w")
    elif want_gu or gu is not None:
        gu = (_new((*lead, 2 * F), _BF16, x, stream) if gu is None
              else _output(gu, _BF16, (*lead, 2 * F), dev, "gu"))
    if M == 0 and F > 0 and K > 0:
        return out, gu
    if scaled:
        _lf._check(_lib().gated_ffn_e4m3(x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), code,
                                            out.data_ptr(), M, F, K, _handle(stream, dev)), "gated_ffn_e4m3")
    else:
        _lf._check(_lib().gated_ffn(x.data_ptr(), w.data_ptr(), code, out.data_ptr(),
                                       None if gu is None else gu.data_ptr(), M, F, K, _handle(stream, dev)),
                   "gated_ffn")
    return out, gu


def gated_ffn_backward(dout, x, w, gu, act="silu", want_dx=True, want_dw=True, dx=None, dw=None, dgu=None,
                       stream=None):
    """Gradient of gated_ffn (bf16): dout [..., F], gu [..., 2F] as gated_ffn
    returned it.  Returns (dx [..., K], dw [2F, K]), None where not wanted.
    dgu [..., 2F] receives the gradient of the two projections (pass gu itself
    to reuse its memory; a new tensor by default)."""
    code = _activation(act)
    M, F, K, dev = _gated_dims(x, w, _BF16, stream)
    lead = x.shape[:-1]
    _require(dout, _BF16, dev, "dout")
    _require(gu, _BF16, dev, "gu")
    if tuple(dout.shape) != (*lead, F) or tuple(gu.shape) != (*lead, 2 * F):
        raise ValueError("dout must be [..., F] and gu [..., 2F] for x's rows")
    if dgu is None:
        dgu = _new(gu.shape, _BF16, x, stream)
    else:
        _output(dgu, _BF16, gu.shape, dev, "dgu")
    if want_dx or dx is not None:
        dx = _new(x.shape, _BF16, x, stream) if dx is None else _output(dx, _BF16, x.shape, dev, "dx")
    if want_dw or dw is not None:
        dw = _new(w.shape, _BF16, x, stream) if dw is None else _output(dw, _BF16, w.shape, dev, "dw")
    if M == 0 and F > 0 and K > 0:
        return dx, _zeroed(dw, stream)
    L = _lib()
    nbytes = _gated_scratch(M, F, K)
    scratch = _new((nbytes,), torch.uint8, x, stream) if nbytes else None
    _lf._check(L.gated_ffn_backward(dout.data_ptr(), x.data_ptr(), w.data_ptr(), gu.data_ptr(), code, dgu.data_ptr(),
                                    None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr(),
                                    None if scratch is None else scratch.data_ptr(), M, F, K, _handle(stream, dev)),
               "gated_ffn_backward")
    return dx, dw
