// binding.cpp -- the Python side of the 8-bit checkpoints and the losses as a
// CPython extension (module _step): checks of types, shapes, strides and
// devices, allocation of the outputs, and one call of the C entry point of
// include/qlora_nf4.h.  It does no arithmetic.  These calls come once per
// layer or step on tensors whose kernels may take a few microseconds;
// through ctypes the checks and allocations alone took 5 to 14 us a call.
// _ops.py holds the functions that users call.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/qlora_nf4.h"

namespace {

PyObject* g_error = nullptr;     // QLoRAError(function, code)
PyObject* g_need = nullptr;      // _ops._need: raises the ValueError for a tensor that is not as wanted
PyObject* g_rows = nullptr;      // _ops._rows: the same for logits

[[noreturn]] void raise(PyObject* type, const char* text) {
    PyErr_SetString(type, text);
    throw python_error();
}

void check(const char* fn, int rc) {
    if (rc == QLORA_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "si", fn, rc);
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

// The current device; -1 without one, which no tensor is on.
int current_device() {
    c10::DeviceIndex d = -1;
    return c10::cuda::GetDevice(&d) == cudaSuccess ? d : -1;
}

int64_t to_int(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

uint64_t to_u64(PyObject* o) {
    const unsigned long long v = PyLong_AsUnsignedLongLongMask(o);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) throw python_error();
    return v;
}

float to_float(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
}

bool to_bool(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

// The raw handle of the stream: the argument, or the current stream.
qlora_stream_t to_stream(PyObject* o, int dev) {
    if (o != Py_None) return reinterpret_cast<qlora_stream_t>(to_u64(o));
    return c10::cuda::getCurrentCUDAStream(dev).stream();
}

// The address of a dense tensor of this type and shape on the current device.
void* need(PyObject* o, const char* name, at::ScalarType dt, at::IntArrayRef shape, int dev) {
    if (THPVariable_Check(o)) {
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.scalar_type() == dt && t.sizes() == shape && t.is_contiguous() && t.is_cuda() && t.get_device() == dev)
            return t.data_ptr();
    }
    PyObject* s = PyTuple_New((Py_ssize_t)shape.size());
    if (s == nullptr) throw python_error();
    for (size_t i = 0; i < shape.size(); ++i) PyTuple_SET_ITEM(s, (Py_ssize_t)i, PyLong_FromLongLong(shape[i]));
    PyObject* r = PyObject_CallFunction(g_need, "OsOO", o, name, (PyObject*)torch::getTHPDtype(dt), s);
    Py_DECREF(s);
    if (r == nullptr) throw python_error();
    Py_DECREF(r);
    raise(PyExc_RuntimeError, name);
}

void* opt(PyObject* o, const char* name, at::ScalarType dt, at::IntArrayRef shape, int dev) {
    return o == Py_None ? nullptr : need(o, name, dt, shape, dev);
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType dt, int dev) {
    return at::detail::empty_cuda(shape, dt, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
}

// The caller's workspace, or one of n bytes.
struct Workspace {
    at::Tensor own;
    void* p;
    size_t n;
    Workspace(PyObject* o, const char* fn, size_t bytes, int dev) {
        if (bytes == 0) check(fn, QLORA_ERR_SHAPE);
        if (o == Py_None) own = empty({(int64_t)bytes}, at::kByte, dev);
        else if (!THPVariable_Check(o)) raise(PyExc_ValueError, "ws: a tensor wanted");
        const at::Tensor& t = o == Py_None ? own : THPVariable_Unpack(o);
        if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
            raise(PyExc_ValueError, "ws: a dense tensor on the current CUDA device wanted");
        p = t.data_ptr();
        n = (size_t)t.nbytes();
    }
};

// [M, V] logits or their gradient with dense rows.
struct Rows {
    void* p;
    int dtype;
    at::ScalarType dt;
    int64_t M, V, ld;
    Rows(PyObject* o, const char* name, int dev) {
        if (THPVariable_Check(o)) {
            const at::Tensor& t = THPVariable_Unpack(o);
            dt = t.scalar_type();
            if (t.dim() == 2 && (dt == at::kBFloat16 || dt == at::kFloat) && t.is_cuda() && t.get_device() == dev &&
                (t.stride(1) == 1 || t.size(1) <= 1)) {
                M = t.size(0);
                V = t.size(1);
                ld = M > 1 ? t.stride(0) : std::max(V, t.stride(0));
                dtype = dt == at::kFloat ? QLORA_LOGITS_FP32 : QLORA_LOGITS_BF16;
                p = t.data_ptr();
                return;
            }
        }
        PyObject* r = PyObject_CallFunction(g_rows, "Os", o, name);
        if (r == nullptr) throw python_error();
        Py_DECREF(r);
        raise(PyExc_RuntimeError, name);
    }
};

// The gradient: the caller's tensor, a new one, or none.
struct Grad {
    PyObject* obj;               // a new reference
    void* p = nullptr;
    int64_t ld;
    Grad(PyObject* o, bool want, const Rows& l, int dev) : ld(l.V) {
        if (o != Py_None) {
            const Rows g(o, "dlogits", dev);
            if (g.M != l.M || g.V != l.V || g.dt != l.dt) need(o, "dlogits", l.dt, {l.M, l.V}, dev);
            p = g.p;
            ld = g.ld;
            Py_INCREF(o);
            obj = o;
        } else if (want) {
            const at::Tensor t = empty({l.M, l.V}, l.dt, dev);
            p = t.data_ptr();
            obj = THPVariable_Wrap(t);
        } else {
            Py_INCREF(Py_None);
            obj = Py_None;
        }
    }
    ~Grad() { Py_XDECREF(obj); }
    PyObject* take() {
        PyObject* o = obj;
        obj = nullptr;
        return o;
    }
};

void args(const char* fn, Py_ssize_t n, Py_ssize_t want) {
    if (n != want) raise(PyExc_TypeError, fn);
}

// (X, fmt, codes | None, scales | None, stream) -> (codes, scales)
PyObject* py_act8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    args("act8_quantize", n, 5);
    if (!THPVariable_Check(a[0]) || THPVariable_Unpack(a[0]).dim() != 2)
        raise(PyExc_ValueError, "X: a bf16 [M, K] tensor wanted");
    const int dev = current_device();
    const int64_t M = THPVariable_Unpack(a[0]).size(0), K = THPVariable_Unpack(a[0]).size(1);
    const void* X = need(a[0], "X", at::kBFloat16, {M, K}, dev);
    const bool own = a[2] == Py_None;
    const at::Tensor c = own ? empty({M, K}, at::kByte, dev) : at::Tensor();
    const at::Tensor s = own ? empty({M, K / QLORA_ACT8_BLOCK}, at::kByte, dev) : at::Tensor();
    void* pc = own ? c.data_ptr() : need(a[2], "codes", at::kByte, {M, K}, dev);
    void* ps = own ? s.data_ptr() : need(a[3], "scales", at::kByte, {M, K / QLORA_ACT8_BLOCK}, dev);
    check("act8_quantize", act8_quantize((const qlora_bf16*)X, M, K, (int)to_int(a[1]), (uint8_t*)pc, (uint8_t*)ps,
                                         to_stream(a[4], dev)));
    if (!own) return PyTuple_Pack(2, a[2], a[3]);
    return Py_BuildValue("NN", THPVariable_Wrap(c), THPVariable_Wrap(s));
    END_HANDLE_TH_ERRORS
}

act8_tensor checkpoint(PyObject* const* a, int dev) {     // codes, scales, M, K, fmt
    const int64_t M = to_int(a[2]), K = to_int(a[3]);
    act8_tensor x;
    x.codes = (const uint8_t*)need(a[0], "codes", at::kByte, {M, K}, dev);
    x.scales = (const uint8_t*)need(a[1], "scales", at::kByte, {M, K / QLORA_ACT8_BLOCK}, dev);
    x.M = M;
    x.K = K;
    x.fmt = (int32_t)to_int(a[4]);
    return x;
}

// (codes, scales, M, K, fmt, out | None, stream) -> X
PyObject* py_act8_dequant(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    args("act8_dequant", n, 7);
    const int dev = current_device();
    const act8_tensor x = checkpoint(a, dev);
    const at::Tensor t = a[5] == Py_None ? empty({x.M, x.K}, at::kBFloat16, dev) : at::Tensor();
    void* p = a[5] == Py_None ? t.data_ptr() : need(a[5], "out", at::kBFloat16, {x.M, x.K}, dev);
    check("act8_dequant", act8_dequant(&x, (qlora_bf16*)p, to_stream(a[6], dev)));
    if (a[5] == Py_None) return THPVariable_Wrap(t);
    Py_INCREF(a[5]);
    return a[5];
    END_HANDLE_TH_ERRORS
}

// (codes, scales, M, K, fmt, packed, wcodes, wscale, wmean, N, K, quant_type, dY, A, B, scaling, dropout_p, seed,
//  offset, T | None, dX | None, dA | None, dB | None, ws | None, stream) -> (dX, dA, dB)
PyObject* py_bwd_act8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    args("qlora_linear_bwd_act8", n, 25);
    const int dev = current_device();
    const act8_tensor x = checkpoint(a, dev);
    nf4dq_weight w;
    w.N = to_int(a[9]);
    w.K = to_int(a[10]);
    w.quant_type = (int32_t)to_int(a[11]);
    int64_t pb = 0, nb = 0, ng = 0;
    check("qlora_linear_bwd_act8", nf4dq_sizes(w.N, w.K, &pb, &nb, &ng));
    w.packed = (const uint8_t*)need(a[5], "packed", at::kByte, {w.N, w.K / 2}, dev);
    w.codes = (const int8_t*)need(a[6], "w.codes", at::kChar, {nb}, dev);
    w.scale = (const float*)need(a[7], "w.scale", at::kFloat, {ng}, dev);
    w.mean = (const float*)need(a[8], "w.mean", at::kFloat, {ng}, dev);
    if (!THPVariable_Check(a[13]) || THPVariable_Unpack(a[13]).dim() != 2)
        raise(PyExc_ValueError, "A: a bf16 [r, K] tensor wanted");
    const at::ScalarType bf = at::kBFloat16;
    const int64_t M = x.M, N = w.N, K = w.K, r = THPVariable_Unpack(a[13]).size(0);
    const void* dY = need(a[12], "dY", bf, {M, N}, dev);
    const void* A = need(a[13], "A", bf, {r, K}, dev);
    const void* B = need(a[14], "B", bf, {N, r}, dev);
    const void* T = opt(a[19], "T", bf, {M, r}, dev);
    const float p = to_float(a[16]);
    const int64_t shape[3][2] = {{M, K}, {r, K}, {N, r}};
    static const char* const name[3] = {"dX", "dA", "dB"};
    at::Tensor own[3];
    void* out[3];
    for (int i = 0; i < 3; ++i) {
        if (a[20 + i] == Py_None) {
            own[i] = empty(shape[i], bf, dev);
            out[i] = own[i].data_ptr();
        } else {
            out[i] = need(a[20 + i], name[i], bf, shape[i], dev);
        }
    }
    const Workspace ws(a[23], "qlora_act8_workspace_bytes",
                       qlora_act8_workspace_bytes(M, N, K, r > QLORA_MAX_RANK ? 0 : (int)r, p > 0.f), dev);
    check("qlora_linear_bwd_act8",
          qlora_linear_bwd_act8(&x, (const qlora_bf16*)dY, &w, (const qlora_bf16*)A, (const qlora_bf16*)B, (int)r,
                                to_float(a[15]), p, to_u64(a[17]), to_u64(a[18]), (const qlora_bf16*)T,
                                (qlora_bf16*)out[0], (qlora_bf16*)out[1], (qlora_bf16*)out[2], ws.p, ws.n,
                                to_stream(a[24], dev)));
    PyObject* t = PyTuple_New(3);
    if (t == nullptr) return nullptr;
    for (int i = 0; i < 3; ++i) {
        PyObject* o = a[20 + i];
        if (o == Py_None) o = THPVariable_Wrap(own[i]);
        else Py_INCREF(o);
        PyTuple_SET_ITEM(t, i, o);
    }
    return t;
    END_HANDLE_TH_ERRORS
}

// (logits, targets, logit_scale, out | None, stream) -> logp
PyObject* py_token_logprob(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    args("token_logprob", n, 5);
    const int dev = current_device();
    const Rows l(a[0], "logits", dev);
    const void* y = need(a[1], "targets", at::kLong, {l.M}, dev);
    const at::Tensor t = a[3] == Py_None ? empty({l.M}, at::kFloat, dev) : at::Tensor();
    void* p = a[3] == Py_None ? t.data_ptr() : need(a[3], "out", at::kFloat, {l.M}, dev);
    check("token_logprob", token_logprob(l.p, l.dtype, l.M, l.V, l.ld, to_float(a[2]), (const int64_t*)y, (float*)p,
                                         to_stream(a[4], dev)));
    if (a[3] == Py_None) return THPVariable_Wrap(t);
    Py_INCREF(a[3]);
    return a[3];
    END_HANDLE_TH_ERRORS
}

// (logits, targets, cu_seqlens, ref_logp | None, beta, kind, label_smoothing, margin, average, logit_scale,
//  grad_scale, dlogits | None, want_grad, ws | None, stream) -> (loss, rewards, logp, dlogits | None)
PyObject* py_preference_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    args("preference_loss", n, 15);
    const int dev = current_device();
    const Rows l(a[0], "logits", dev);
    const int64_t nc = THPVariable_Check(a[2]) ? THPVariable_Unpack(a[2]).numel() : 0;
    if (nc < 3 || nc % 2 != 1) raise(PyExc_ValueError, "cu_seqlens: an int32 [2 P + 1] tensor wanted");
    const void* y = need(a[1], "targets", at::kLong, {l.M}, dev);
    const void* cu = need(a[2], "cu_seqlens", at::kInt, {nc}, dev);
    const void* ref = opt(a[3], "ref_logp", at::kFloat, {l.M}, dev);
    Grad g(a[11], to_bool(a[12]), l, dev);
    const at::Tensor loss = empty({}, at::kFloat, dev), rewards = empty({nc - 1}, at::kFloat, dev);
    const at::Tensor logp = empty({l.M}, at::kFloat, dev);
    const Workspace ws(a[13], "loss_workspace_bytes", loss_workspace_bytes(l.M), dev);
    check("preference_loss",
          preference_loss(l.p, l.dtype, l.M, l.V, l.ld, to_float(a[9]), (const int64_t*)y, (const int32_t*)cu, nc / 2,
                          (const float*)ref, (int)to_int(a[5]), to_float(a[4]), to_float(a[6]), to_float(a[7]),
                          to_bool(a[8]), to_float(a[10]), (float*)loss.data_ptr(), (float*)rewards.data_ptr(),
                          (float*)logp.data_ptr(), g.p, g.ld, ws.p, ws.n, to_stream(a[14], dev)));
    return Py_BuildValue("NNNN", THPVariable_Wrap(loss), THPVariable_Wrap(rewards), THPVariable_Wrap(logp), g.take());
    END_HANDLE_TH_ERRORS
}

// (logits, targets, advantages, weights, old_logp | None, ref_logp | None, clip_low, clip_high, kl_coef, logit_scale,
//  grad_scale, dlogits | None, want_grad, ws | None, stream) -> (stats, logp, dlogits | None)
PyObject* py_policy_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    args("policy_loss", n, 15);
    const int dev = current_device();
    const Rows l(a[0], "logits", dev);
    const void* y = need(a[1], "targets", at::kLong, {l.M}, dev);
    const void* adv = need(a[2], "advantages", at::kFloat, {l.M}, dev);
    const void* w = need(a[3], "weights", at::kFloat, {l.M}, dev);
    const void* old = opt(a[4], "old_logp", at::kFloat, {l.M}, dev);
    const void* ref = opt(a[5], "ref_logp", at::kFloat, {l.M}, dev);
    Grad g(a[11], to_bool(a[12]), l, dev);
    const at::Tensor stats = empty({4}, at::kFloat, dev), logp = empty({l.M}, at::kFloat, dev);
    const Workspace ws(a[13], "loss_workspace_bytes", loss_workspace_bytes(l.M), dev);
    check("policy_loss",
          policy_loss(l.p, l.dtype, l.M, l.V, l.ld, to_float(a[9]), (const int64_t*)y, (const float*)adv,
                      (const float*)w, (const float*)old, (const float*)ref, to_float(a[6]), to_float(a[7]),
                      to_float(a[8]), to_float(a[10]), (float*)stats.data_ptr(), (float*)logp.data_ptr(), g.p, g.ld,
                      ws.p, ws.n, to_stream(a[14], dev)));
    return Py_BuildValue("NNN", THPVariable_Wrap(stats), THPVariable_Wrap(logp), g.take());
    END_HANDLE_TH_ERRORS
}

// (QLoRAError, _need, _rows)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    args("bind", n, 3);
    PyObject** slot[3] = {&g_error, &g_need, &g_rows};
    for (int i = 0; i < 3; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*slot[i], a[i]);
    }
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define FAST(name, fn) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST("bind", py_bind),
                          FAST("act8_quantize", py_act8_quantize),
                          FAST("act8_dequant", py_act8_dequant),
                          FAST("qlora_linear_bwd_act8", py_bwd_act8),
                          FAST("token_logprob", py_token_logprob),
                          FAST("preference_loss", py_preference_loss),
                          FAST("policy_loss", py_policy_loss),
                          {nullptr, nullptr, 0, nullptr}};
// the module's docstring; build.py looks for it in the built file
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_step", QLORA_TORCH_STAMP, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step() { return PyModule_Create(&kModule); }
