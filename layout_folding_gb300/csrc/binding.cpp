// binding.cpp -- the common calls of the projections and of the norms around a block
// without the interpreter's share: checks, new outputs and the call itself.  The functions
// of the Python modules (projections.py, block_norms.py) ask here first.  A call that is
// not of the plain kind -- given outputs, a stream, sliced rows, no rows, anything that
// has to be refused -- is not taken (None), and the Python function does it or says what
// is wrong with it.  A call that is taken returns its outputs, or the library's status;
// other Python threads run while it allocates and launches.
//
// One call's share of the host with two outputs (Grace): block_norm 12.3 us in
// Python, 4.6 to 4.9 here; its gradient 22 and 11; linear 10 and 4.0.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "layoutfold.h"

namespace {

struct Library {
    decltype(&block_norm) norm = nullptr;
    decltype(&block_norm_backward) norm_backward = nullptr;
    decltype(&block_norm_backward_scratch) norm_scratch = nullptr;
    decltype(&linear) lin = nullptr;
    decltype(&linear_e4m3) lin_e4m3 = nullptr;
    decltype(&linear_backward) lin_backward = nullptr;
    decltype(&linear_backward_scratch) lin_scratch = nullptr;
} lib;

using at::Tensor;

// A plain tensor of the current device, contiguous; null for None.  False: not one.
bool plain(PyObject *o, int device, const Tensor **t)
{
    *t = nullptr;
    if (o == Py_None)
        return true;
    if (!THPVariable_CheckExact(o))
        return false;
    const Tensor &v = THPVariable_Unpack(o);
    if (!v.defined() || v.layout() != at::kStrided || !v.is_cuda() || v.get_device() != device || !v.is_contiguous())
        return false;
    *t = &v;
    return true;
}
// The current device where the call's first tensor is on a GPU, else -1.
int device_for(PyObject *x)
{
    return THPVariable_CheckExact(x) && THPVariable_Unpack(x).is_cuda() ? c10::cuda::current_device() : -1;
}
bool required(PyObject *o, int device, const Tensor **t) { return plain(o, device, t) && *t; }

int code_of(at::ScalarType t)
{
    return t == at::kBFloat16 ? LF_BF16 : t == at::kHalf ? LF_FP16 : t == at::kFloat ? LF_FP32 : -1;
}
bool is_rows(const Tensor *t, const Tensor &x)
{
    return t->scalar_type() == x.scalar_type() && t->sizes() == x.sizes();
}
const void *at_of(const Tensor *t) { return t ? t->const_data_ptr() : nullptr; }
void *out_of(const Tensor &t) { return t.defined() ? t.mutable_data_ptr() : nullptr; }

Tensor new_like(const Tensor &x, at::IntArrayRef sizes, at::ScalarType type)
{
    return at::empty(sizes, x.options().dtype(type));
}
Tensor scratch_of(const Tensor &x, int64_t bytes)
{
    return bytes > 0 ? at::empty({bytes}, x.options().dtype(at::kByte)) : Tensor();
}
PyObject *wrap(const Tensor &t)
{
    if (!t.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
template <class... T>
PyObject *outputs(const T &...t)
{
    PyObject *o[] = {wrap(t)...};
    constexpr Py_ssize_t n = sizeof...(t);
    PyObject *tuple = PyTuple_New(n);
    bool ok = tuple != nullptr;
    for (Py_ssize_t i = 0; i < n; ++i) {
        ok = ok && o[i];
        if (ok)
            PyTuple_SET_ITEM(tuple, i, o[i]);
        else
            Py_XDECREF(o[i]);
    }
    if (!ok)
        Py_CLEAR(tuple);
    return tuple;
}
// The interpreter is left to other threads in its scope: an allocation may wait for the
// device, a launch for room in its queue, and what runs before it there may be a host
// function that needs the interpreter.
struct WithoutInterpreter {
    PyThreadState *state = PyEval_SaveThread();
    WithoutInterpreter() = default;
    WithoutInterpreter(const WithoutInterpreter &) = delete;
    ~WithoutInterpreter() { PyEval_RestoreThread(state); }
};
PyObject *status(lf_status s) { return PyLong_FromLong(s); }

bool number(PyObject *o, float *v)
{
    if (!PyFloat_CheckExact(o) && !PyLong_CheckExact(o))
        return false;
    const double d = PyFloat_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    *v = static_cast<float>(d);
    return true;
}
bool boolean(PyObject *o, bool *v)
{
    *v = o == Py_True;
    return o == Py_True || o == Py_False;
}

// What block_norm and its gradient share.
struct Block {
    const Tensor *x, *post, *pre, *gate;
    int device, code, wcode, gate_code = LF_BF16;
    int64_t M, D, gate_rows = 0;
    float branch, residual, eps;
    bool read(PyObject *px, PyObject *ppost, PyObject *ppre, PyObject *pgate, PyObject *b, PyObject *r, PyObject *e)
    {
        device = device_for(px);
        if (device < 0 || !required(px, device, &x) || x->dim() == 0 || (code = code_of(x->scalar_type())) < 0)
            return false;
        D = x->size(-1);
        M = D > 0 ? x->numel() / D : 0;
        if (M <= 0 || !plain(ppost, device, &post) || !plain(ppre, device, &pre) || !plain(pgate, device, &gate) ||
            !number(b, &branch) || !number(r, &residual) || !number(e, &eps))
            return false;
        wcode = code;
        for (const Tensor *w : {post, pre})
            if (w) {
                wcode = code_of(w->scalar_type());
                if ((wcode != code && wcode != LF_FP32) || w->numel() != D)
                    return false;
            }
        if (post && pre && post->scalar_type() != pre->scalar_type())
            return false;
        if (!gate)
            return true;
        gate_code = code_of(gate->scalar_type());
        if ((gate_code != code && gate_code != LF_FP32) || gate->dim() < 1 || gate->dim() > 2 || gate->size(-1) != D)
            return false;
        gate_rows = gate->dim() == 1 ? 1 : gate->size(0);
        return gate_rows > 0 && M % gate_rows == 0;
    }
    cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
};

// (x, residual, post, pre, gate, branch_scale, residual_scale, eps, fp8) -> (y, h, scale)
PyObject *py_block_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Block c;
    const Tensor *residual;
    bool fp8;
    if (n != 9 || !lib.norm || !c.read(a[0], a[2], a[3], a[4], a[5], a[6], a[7]) || !boolean(a[8], &fp8) ||
        !required(a[1], c.device, &residual) || !is_rows(residual, *c.x) || (fp8 && !c.pre))
        Py_RETURN_NONE;
    Tensor h, y, scale;
    const auto call = [&] {
        const WithoutInterpreter others_run;
        h = new_like(*c.x, c.x->sizes(), c.x->scalar_type());
        if (c.pre) {
            y = new_like(*c.x, c.x->sizes(), fp8 ? at::kFloat8_e4m3fn : c.x->scalar_type());
            if (fp8)
                scale = new_like(*c.x, c.x->sizes().slice(0, c.x->dim() - 1), at::kFloat);
        }
        return lib.norm(at_of(c.x), c.D, at_of(residual), c.D, at_of(c.post), at_of(c.pre), at_of(c.gate), c.gate_rows,
                        c.gate_code, out_of(h), out_of(y), static_cast<float *>(out_of(scale)), c.code, c.wcode,
                        fp8 ? LF_E4M3 : c.code, c.eps, c.branch, c.residual, c.M, c.D, c.stream());
    };
    const lf_status s = call();
    return s == LF_OK ? outputs(y, h, scale) : status(s);
    END_HANDLE_TH_ERRORS
}

// (dy, x, h, post, pre, gate, dh, branch_scale, residual_scale, eps, want_dparams) ->
// (dx, dresidual, dpost, dpre, dgate)
PyObject *py_block_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Block c;
    const Tensor *dy, *h, *dh;
    bool params;
    if (n != 11 || !lib.norm_backward || !c.read(a[1], a[3], a[4], a[5], a[7], a[8], a[9]) || !boolean(a[10], &params) ||
        !plain(a[0], c.device, &dy) || !plain(a[2], c.device, &h) || !plain(a[6], c.device, &dh) ||
        (c.pre ? !dy || !h : !dh) || (dy && !is_rows(dy, *c.x)) || (h && !is_rows(h, *c.x)) || (dh && !is_rows(dh, *c.x)))
        Py_RETURN_NONE;
    Tensor dx, dres, dpost, dpre, dgate;
    const auto call = [&] {
        const WithoutInterpreter others_run;
        const auto gradient = [&](const Tensor *p) { return p && params ? new_like(*p, p->sizes(), p->scalar_type()) : Tensor(); };
        dx = new_like(*c.x, c.x->sizes(), c.x->scalar_type());
        dres = new_like(*c.x, c.x->sizes(), c.x->scalar_type());
        dpost = gradient(c.post);
        dpre = gradient(c.pre);
        dgate = gradient(c.gate);
        Tensor scratch;
        if (dpost.defined() || dpre.defined() || dgate.defined())
            scratch = scratch_of(*c.x, lib.norm_scratch(c.M, c.D, c.code, c.gate_rows));
        return lib.norm_backward(at_of(dy), at_of(c.x), at_of(h), at_of(c.post), at_of(c.pre), at_of(c.gate), c.gate_rows,
                                 c.gate_code, at_of(dh), out_of(dx), out_of(dres), out_of(dpost), out_of(dpre),
                                 out_of(dgate), out_of(scratch), c.code, c.wcode, c.eps, c.branch, c.residual, c.M, c.D,
                                 c.stream());
    };
    const lf_status s = call();
    return s == LF_OK ? outputs(dx, dres, dpost, dpre, dgate) : status(s);
    END_HANDLE_TH_ERRORS
}

// What linear and its gradient share: x [..., K], w [N, K], bias [N].
struct Projection {
    const Tensor *x, *w, *bias;
    int device, bias_code = LF_BF16;
    long act;
    int64_t M, N, K;
    at::DimVector out;  // the output's shape
    bool read(PyObject *px, PyObject *pw, PyObject *pbias, PyObject *pact, at::ScalarType type)
    {
        device = device_for(px);
        if (device < 0 || !required(px, device, &x) || !required(pw, device, &w) || !plain(pbias, device, &bias) || !PyLong_CheckExact(pact))
            return false;
        act = PyLong_AsLong(pact);
        if (x->scalar_type() != type || w->scalar_type() != type || x->dim() == 0 || w->dim() != 2 || w->size(1) != x->size(-1))
            return false;
        N = w->size(0);
        K = w->size(1);
        M = K > 0 ? x->numel() / K : 0;
        if (M <= 0 || N <= 0)
            return false;
        if (bias) {
            bias_code = code_of(bias->scalar_type());
            if ((bias_code != LF_BF16 && bias_code != LF_FP32) || bias->numel() != N)
                return false;
        }
        out.assign(x->sizes().begin(), x->sizes().end());
        out.back() = N;
        return true;
    }
    bool is_output(const Tensor *t) const { return t->scalar_type() == at::kBFloat16 && t->sizes() == at::IntArrayRef(out); }
    cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
};

// (x, w, bias, act code, residual, x_scale, w_scale, want_pre) -> (out, pre)
PyObject *py_linear(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 8 || !lib.lin)
        Py_RETURN_NONE;
    const bool e4m3 = a[5] != Py_None;
    Projection c;
    const Tensor *residual, *xs, *ws;
    bool want_pre;
    if (!c.read(a[0], a[1], a[2], a[3], e4m3 ? at::kFloat8_e4m3fn : at::kBFloat16) || !plain(a[4], c.device, &residual) ||
        !plain(a[5], c.device, &xs) || !plain(a[6], c.device, &ws) || !boolean(a[7], &want_pre) || !xs != !ws ||
        (residual && !c.is_output(residual)))
        Py_RETURN_NONE;
    if (e4m3 && (want_pre || xs->scalar_type() != at::kFloat || ws->scalar_type() != at::kFloat || xs->numel() != c.M ||
                 ws->numel() != c.N))
        Py_RETURN_NONE;
    Tensor out, pre;
    const auto call = [&] {
        const WithoutInterpreter others_run;
        out = new_like(*c.x, c.out, at::kBFloat16);
        if (want_pre)
            pre = new_like(*c.x, c.out, at::kBFloat16);
        return e4m3 ? lib.lin_e4m3(at_of(c.x), static_cast<const float *>(at_of(xs)), at_of(c.w),
                                   static_cast<const float *>(at_of(ws)), at_of(c.bias), c.bias_code,
                                   static_cast<int>(c.act), at_of(residual), out_of(out), c.M, c.N, c.K, c.stream())
                    : lib.lin(at_of(c.x), at_of(c.w), at_of(c.bias), c.bias_code, static_cast<int>(c.act), at_of(residual),
                              out_of(out), out_of(pre), c.M, c.N, c.K, c.stream());
    };
    const lf_status s = call();
    return s == LF_OK ? outputs(out, pre) : status(s);
    END_HANDLE_TH_ERRORS
}

// (dout, x, w, pre, act code, bias, want_dx, want_dw) -> (dx, dw, dbias)
PyObject *py_linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Projection c;
    const Tensor *dout, *pre;
    bool want_dx, want_dw;
    if (n != 8 || !lib.lin_backward || !c.read(a[1], a[2], a[5], a[4], at::kBFloat16) || !required(a[0], c.device, &dout) ||
        !plain(a[3], c.device, &pre) || !boolean(a[6], &want_dx) || !boolean(a[7], &want_dw) || !c.is_output(dout))
        Py_RETURN_NONE;
    const bool activated = c.act != LF_ACT_NONE;
    if (activated && (!pre || !c.is_output(pre)))
        Py_RETURN_NONE;
    Tensor dx, dw, db;
    const auto call = [&] {
        const WithoutInterpreter others_run;
        Tensor dz;
        if (activated)
            dz = new_like(*c.x, c.out, at::kBFloat16);
        if (want_dx)
            dx = new_like(*c.x, c.x->sizes(), at::kBFloat16);
        if (want_dw)
            dw = new_like(*c.w, c.w->sizes(), at::kBFloat16);
        if (c.bias)
            db = new_like(*c.bias, c.bias->sizes(), c.bias->scalar_type());
        const Tensor scratch = scratch_of(*c.x, lib.lin_scratch(c.M, c.N, c.K));
        return lib.lin_backward(at_of(dout), at_of(c.x), at_of(c.w), activated ? at_of(pre) : nullptr,
                                static_cast<int>(c.act), out_of(dz), out_of(dx), out_of(dw), out_of(db), c.bias_code,
                                out_of(scratch), c.M, c.N, c.K, c.stream());
    };
    const lf_status s = call();
    return s == LF_OK ? outputs(dx, dw, db) : status(s);
    END_HANDLE_TH_ERRORS
}

// The library's functions: their addresses, in Library's order.
PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    void *p[7];
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
        return nullptr;
    }
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred())
            return nullptr;
    }
    lib.norm = reinterpret_cast<decltype(lib.norm)>(p[0]);
    lib.norm_backward = reinterpret_cast<decltype(lib.norm_backward)>(p[1]);
    lib.norm_scratch = reinterpret_cast<decltype(lib.norm_scratch)>(p[2]);
    lib.lin = reinterpret_cast<decltype(lib.lin)>(p[3]);
    lib.lin_e4m3 = reinterpret_cast<decltype(lib.lin_e4m3)>(p[4]);
    lib.lin_backward = reinterpret_cast<decltype(lib.lin_backward)>(p[5]);
    lib.lin_scratch = reinterpret_cast<decltype(lib.lin_scratch)>(p[6]);
    Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"bind", fast(py_bind), METH_FASTCALL, nullptr},
                         {"block_norm", fast(py_block_norm), METH_FASTCALL, nullptr},
                         {"block_norm_backward", fast(py_block_norm_backward), METH_FASTCALL, nullptr},
                         {"linear", fast(py_linear), METH_FASTCALL, nullptr},
                         {"linear_backward", fast(py_linear_backward), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
