// target_binding.cpp -- Python entry of the target's operators (include/lookup_target.h).
//
// These calls take a dozen tensors each and their kernels run for microseconds: checked
// and marshalled in Python they take 25 to 35 us to enqueue, here 5 to 12.  Everything a
// call does is one function: check the tensors, allocate what the caller did not give,
// enter the library through the C ABI (its entry points are handed over as addresses,
// so nothing links against it) with the interpreter's lock released.  A function
// returns its outputs, or the library's error code as an int.

#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "lookup_target.h"

namespace {

decltype(&lookup_kv_append) g_kv_append = nullptr;
decltype(&lookup_paged_attention) g_attention = nullptr;
decltype(&lookup_paged_attention_workspace_bytes) g_attention_bytes = nullptr;
decltype(&lookup_verify_logits) g_verify = nullptr;
decltype(&lookup_verify_logits_workspace_bytes) g_verify_bytes = nullptr;

// A refusal: raised as ValueError or TypeError.
struct Refused {
    PyObject *type;
    std::string what;
};
[[noreturn]] void refuse(std::string what) { throw Refused{PyExc_ValueError, std::move(what)}; }
[[noreturn]] void refuse_type(std::string what) { throw Refused{PyExc_TypeError, std::move(what)}; }

std::string words(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t k = 0; k < shape.size(); ++k) s += (k ? ", " : "") + std::to_string(shape[k]);
    return s + (shape.size() == 1 ? ",)" : ")");
}
const char *words(at::ScalarType t) {
    switch (t) {
    case at::kInt: return "torch.int32";
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    default: return c10::toString(t);
    }
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a torch tensor");
    return THPVariable_Unpack(o);
}

// A tensor that results depend on.  The operators have no backward pass, so where a
// gradient is being recorded it would be lost without a word.
const at::Tensor &operand(PyObject *o, const char *name) {
    const at::Tensor &t = tensor(o, name);
    if (t.requires_grad() && c10::GradMode::is_enabled())
        refuse(std::string(name) + " requires a gradient, which this call does not give: call it under torch.no_grad()");
    return t;
}

// The pointer of a contiguous tensor of this type, shape and device.
template <typename P = void>
P *dense(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, const c10::Device &dev) {
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous() || t.device() != dev)
        refuse(std::string(name) + " must be a contiguous " + words(type) + " tensor of shape " + words(shape) + " on " +
               dev.str());
    return static_cast<P *>(t.data_ptr());
}
template <typename P = void>
P *maybe(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, const c10::Device &dev) {
    return o == Py_None ? nullptr : dense<P>(o, name, type, shape, dev);
}

// The pointer of a tensor whose last axis is dense; its other strides follow.
const void *strided(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape,
                    const c10::Device &dev, int64_t *strides) {
    if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev)
        refuse(std::string(name) + " must be a " + words(type) + " tensor of shape " + words(shape) + " on " + dev.str());
    const size_t n = shape.size();
    if (t.stride(int64_t(n) - 1) != 1 && shape[n - 1] > 1) refuse(std::string(name) + ": the last axis must be dense");
    for (size_t k = 0; k + 1 < n; ++k) strides[k] = t.stride(int64_t(k));
    return t.data_ptr();
}

int32_t size32(int64_t x, const char *name) {
    if (x > INT32_MAX) refuse(std::string(name) + " has 2^31 elements or more along an axis");
    return int32_t(x);
}

int type_code(const at::Tensor &t, const char *name, bool with_f32) {
    if (t.scalar_type() == at::kHalf) return LOOKUP_TYPE_F16;
    if (t.scalar_type() == at::kBFloat16) return LOOKUP_TYPE_BF16;
    if (with_f32 && t.scalar_type() == at::kFloat) return LOOKUP_TYPE_F32;
    refuse_type(std::string(name) + ": unsupported dtype " + words(t.scalar_type()));
}

const c10::Device cuda_device(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    return t.device();
}

long whole(PyObject *o, const char *name) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    if (x > INT32_MAX || x < INT32_MIN) refuse(std::string(name) + " is out of range");
    return x;
}

// The stream of a call: the given torch.cuda.Stream, made current, or the device's current
// one.  PyTorch's allocator keeps memory per stream, so what a call allocates comes from
// its own stream's: other streams' may still be in use by work that they have queued.
class On {
    c10::cuda::CUDAGuard device_;
    c10::cuda::OptionalCUDAStreamGuard current_;

public:
    const c10::Device dev;
    const c10::cuda::CUDAStream caller;                  // current when the call was made
    const c10::cuda::CUDAStream stream;

    On(PyObject *o, const c10::Device &d)
        : device_(d), dev(d), caller(c10::cuda::getCurrentCUDAStream(d.index())), stream(given(o, caller)) {
        if (stream.device() != dev) refuse("stream must be of the tensors' device, " + dev.str());
        if (stream != caller) current_.reset_stream(stream);
    }

private:
    static c10::cuda::CUDAStream given(PyObject *o, const c10::cuda::CUDAStream &caller) {
        if (o == Py_None) return caller;
        int64_t v[3];
        const char *names[3] = {"stream_id", "device_index", "device_type"};
        for (int k = 0; k < 3; ++k) {
            PyObject *a = PyObject_GetAttrString(o, names[k]);
            if (!a) throw python_error();
            v[k] = PyLong_AsLongLong(a);
            Py_DECREF(a);
            if (v[k] == -1 && PyErr_Occurred()) throw python_error();
        }
        return c10::cuda::CUDAStream::unpack3(v[0], c10::DeviceIndex(v[1]), c10::DeviceType(v[2]));
    }
};

// The caller's output, checked, or a new one: of the call's stream, and not used again
// before the caller's stream is past what it does with it.
at::Tensor output(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, const On &on) {
    if (o != Py_None) {
        dense(o, name, type, shape, on.dev);
        return THPVariable_Unpack(o);
    }
    at::Tensor t = at::empty(shape, at::TensorOptions().dtype(type).device(on.dev));
    if (on.stream != on.caller && t.numel()) t.record_stream(on.caller.unwrap());
    return t;
}

// The call's workspace: the caller's, or one of the call's stream, where whatever takes its
// memory next runs after the call.
struct Workspace {
    at::Tensor t;
    size_t bytes;
};
Workspace workspace(PyObject *o, size_t bytes, const On &on) {
    if (o != Py_None) {
        const at::Tensor &t = tensor(o, "workspace");
        if (t.device() != on.dev || !t.is_contiguous()) refuse("workspace must be a contiguous tensor on " + on.dev.str());
        return {t, size_t(t.numel()) * t.element_size()};
    }
    return {at::empty({int64_t(bytes)}, at::TensorOptions().dtype(at::kByte).device(on.dev)), bytes};
}

// The interpreter's lock released while the library enqueues.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

PyObject *result(int rc, const at::Tensor *outs, int n) {
    if (rc) return PyLong_FromLong(rc);
    PyObject *tuple = PyTuple_New(n);
    if (!tuple) return nullptr;
    for (int k = 0; k < n; ++k) {
        PyObject *o = THPVariable_Wrap(outs[k]);
        if (!o) {
            Py_DECREF(tuple);
            return nullptr;
        }
        PyTuple_SET_ITEM(tuple, k, o);
    }
    return tuple;
}

void expect(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) refuse_type("wrong number of arguments");
}

// The paged cache of a call for B requests and head size D.
struct Paged {
    int32_t pages, hkv, page, max_pages;
    void *k, *v;
    const int32_t *table, *kv_len, *q_len;
};
Paged paged(PyObject *k_cache, PyObject *v_cache, PyObject *table, PyObject *kv_len, PyObject *q_len, int64_t B,
            int64_t D, at::ScalarType type, const c10::Device &dev) {
    const at::Tensor &kc = operand(k_cache, "k_cache"), &bt = tensor(table, "block_table");
    operand(v_cache, "v_cache");
    if (kc.dim() != 4 || bt.dim() != 2)
        refuse("k_cache must be [pages, Hkv, page_size, D] and block_table [B, max_pages]");
    const int64_t shape[4] = {kc.size(0), kc.size(1), kc.size(2), D};
    Paged p;
    p.k = dense(k_cache, "k_cache", type, shape, dev);
    p.v = dense(v_cache, "v_cache", type, shape, dev);
    p.table = dense<int32_t>(table, "block_table", at::kInt, {B, bt.size(1)}, dev);
    p.kv_len = dense<int32_t>(kv_len, "kv_len", at::kInt, {B}, dev);
    p.q_len = maybe<int32_t>(q_len, "q_len", at::kInt, {B}, dev);
    p.pages = size32(shape[0], "k_cache");
    p.hkv = size32(shape[1], "k_cache");
    p.page = size32(shape[2], "k_cache");
    p.max_pages = size32(bt.size(1), "block_table");
    return p;
}

PyObject *kv_append(PyObject *const *a, Py_ssize_t n) {
    expect(n, 13);
    const at::Tensor &q = operand(a[0], "q");
    const c10::Device dev = cuda_device(q, "q");
    if (q.dim() != 4) refuse("q must be [B, N, Hq, D]");
    const int64_t B = q.size(0), N = q.size(1), hq = q.size(2), D = q.size(3);
    const at::ScalarType type = q.scalar_type();
    const int code = type_code(q, "q", false);
    const Paged c = paged(a[5], a[6], a[4], a[3], a[8], B, D, type, dev);
    int64_t qs[3], ks[3], vs[3];
    const void *qp = strided(q, "q", type, {B, N, hq, D}, dev, qs);
    const void *kp = strided(operand(a[1], "k"), "k", type, {B, N, int64_t(c.hkv), D}, dev, ks);
    const void *vp = strided(operand(a[2], "v"), "v", type, {B, N, int64_t(c.hkv), D}, dev, vs);
    const float *rotary = nullptr;
    int32_t max_pos = 0, rot = 0;
    if (a[7] != Py_None) {
        const at::Tensor &r = tensor(a[7], "rotary");
        if (r.dim() != 2) refuse("rotary must be [max_pos, rot]");
        max_pos = size32(r.size(0), "rotary");
        rot = size32(r.size(1), "rotary");
        rotary = dense<float>(a[7], "rotary", at::kFloat, {r.size(0), r.size(1)}, dev);
    }
    const int interleaved = PyObject_IsTrue(a[9]);
    if (interleaved < 0) throw python_error();
    const On on(a[12], dev);
    at::Tensor outs[2] = {output(a[10], "out_q", type, {B, N, hq, D}, on), output(a[11], "status", at::kInt, {B}, on)};
    if (N == 0) outs[1].zero_();
    int rc;
    {
        Unlocked unlocked;
        rc = g_kv_append(qp, qs, kp, ks, vp, vs, c.kv_len, c.q_len, c.table, size32(B, "q"), size32(N, "q"),
                         size32(hq, "q"), c.hkv, size32(D, "q"), c.max_pages, c.pages, c.page, rotary, rot, max_pos,
                         interleaved, code, c.k, c.v, outs[0].data_ptr(), static_cast<int32_t *>(outs[1].data_ptr()),
                         on.stream.stream());
    }
    return result(rc, outs, 2);
}

PyObject *attention(PyObject *const *a, Py_ssize_t n) {
    expect(n, 12);
    const at::Tensor &q = operand(a[0], "q");
    const c10::Device dev = cuda_device(q, "q");
    if (q.dim() != 4) refuse("q must be [B, N, Hq, D]");
    const int64_t B = q.size(0), N = q.size(1), hq = q.size(2), D = q.size(3);
    const at::ScalarType type = q.scalar_type();
    const int code = type_code(q, "q", false);
    const Paged c = paged(a[1], a[2], a[3], a[4], a[5], B, D, type, dev);
    int64_t qs[3];
    const void *qp = strided(q, "q", type, {B, N, hq, D}, dev, qs);
    const double scale = a[6] == Py_None ? 1.0 / std::sqrt(double(D)) : PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    const int32_t window = int32_t(whole(a[7], "window"));
    const int32_t b = size32(B, "q"), t = size32(N, "q"), h = size32(hq, "q"), d = size32(D, "q");
    const On on(a[11], dev);
    at::Tensor outs[2] = {output(a[8], "out", type, {B, N, hq, D}, on), output(a[9], "lse", at::kFloat, {B, N, hq}, on)};
    const Workspace ws = workspace(a[10], g_attention_bytes(b, t, h, c.hkv, d), on);
    int rc;
    {
        Unlocked unlocked;
        rc = g_attention(qp, qs, c.k, c.v, c.table, c.kv_len, c.q_len, b, t, h, c.hkv, d, c.max_pages, c.pages, c.page,
                         float(scale), window, code, outs[0].data_ptr(), static_cast<float *>(outs[1].data_ptr()),
                         ws.t.data_ptr(), ws.bytes, on.stream.stream());
    }
    return result(rc, outs, 2);
}

PyObject *verify(PyObject *const *a, Py_ssize_t n) {
    expect(n, 14);
    const at::Tensor &logits = operand(a[2], "logits"), &block = tensor(a[0], "block");
    const c10::Device dev = cuda_device(logits, "logits");
    if (block.dim() != 2 || logits.dim() != 3) refuse("block must be [B, P] and logits [B, P + 1, V]");
    const int64_t B = block.size(0), P = block.size(1), V = logits.size(2);
    const int code = type_code(logits, "logits", true);
    int64_t ls[2], qs[2] = {0, 0};
    const void *lp = strided(logits, "logits", logits.scalar_type(), {B, P + 1, V}, dev, ls);
    const float *noise = maybe<float>(a[3], "noise", at::kFloat, {B, V}, dev);
    const float *u = a[4] == Py_None && (!noise || P == 0) ? nullptr : dense<float>(a[4], "u", at::kFloat, {B, P}, dev);
    const float *temperature = maybe<float>(a[5], "temperature", at::kFloat, {B}, dev);
    const void *qprobs =
        a[6] == Py_None ? nullptr : strided(operand(a[6], "qprobs"), "qprobs", at::kFloat, {B, P, V}, dev, qs);
    const int32_t *point = maybe<int32_t>(a[7], "point_mass", at::kInt, {B, P}, dev);
    const int32_t *blk = dense<int32_t>(a[0], "block", at::kInt, {B, P}, dev);
    const int32_t *len = dense<int32_t>(a[1], "len", at::kInt, {B}, dev);
    const int32_t b = size32(B, "block"), p = size32(P, "block"), v = size32(V, "logits");
    const On on(a[13], dev);
    at::Tensor outs[4] = {output(a[8], "accepted", at::kInt, {B}, on), output(a[9], "commit", at::kInt, {B, P + 1}, on),
                          output(a[10], "ncommit", at::kInt, {B}, on),
                          output(a[11], "logprobs", at::kFloat, {B, P + 1}, on)};
    const Workspace ws = workspace(a[12], g_verify_bytes(b, p, v), on);
    int rc;
    {
        Unlocked unlocked;
        rc = g_verify(blk, len, lp, ls, code, v, noise, temperature, u, static_cast<const float *>(qprobs), qs, point, b,
                      p, static_cast<int32_t *>(outs[0].data_ptr()), static_cast<int32_t *>(outs[1].data_ptr()),
                      static_cast<int32_t *>(outs[2].data_ptr()), static_cast<float *>(outs[3].data_ptr()),
                      ws.t.data_ptr(), ws.bytes, on.stream.stream());
    }
    return result(rc, outs, 4);
}

PyObject *entry_points(PyObject *const *a, Py_ssize_t n) {
    expect(n, 5);
    void *f[5];
    for (int k = 0; k < 5; ++k) {
        f[k] = PyLong_AsVoidPtr(a[k]);
        if (!f[k]) {
            if (!PyErr_Occurred()) refuse("an entry point has no address");
            throw python_error();
        }
    }
    g_kv_append = reinterpret_cast<decltype(g_kv_append)>(f[0]);
    g_attention = reinterpret_cast<decltype(g_attention)>(f[1]);
    g_attention_bytes = reinterpret_cast<decltype(g_attention_bytes)>(f[2]);
    g_verify = reinterpret_cast<decltype(g_verify)>(f[3]);
    g_verify_bytes = reinterpret_cast<decltype(g_verify_bytes)>(f[4]);
    Py_RETURN_NONE;
}

// No C++ exception leaves the module: refusals, Python's and PyTorch's own all become
// Python's.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(a, n);
    } catch (const Refused &r) {
        PyErr_SetString(r.type, r.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyCFunction method() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>));
}

PyMethodDef methods[] = {
    {"entry_points", method<entry_points>(), METH_FASTCALL, "the library's entry points, as addresses"},
    {"kv_append", method<kv_append>(), METH_FASTCALL, "lookup_kv_append"},
    {"attention", method<attention>(), METH_FASTCALL, "lookup_paged_attention"},
    {"verify", method<verify>(), METH_FASTCALL, "lookup_verify_logits"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_target", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__target() { return PyModule_Create(&module); }
