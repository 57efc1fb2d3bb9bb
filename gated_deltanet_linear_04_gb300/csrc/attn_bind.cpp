// Python binding of the full-attention operators (second half of
// include/gdn.h): checks of types, shapes, strides and devices, allocation of
// the outputs that are not given, and the call.  No arithmetic.
//
// The rest of the library is bound with ctypes; these calls are made once per
// layer and token, where the checks and the allocations of one call in
// Python cost more host time than its kernel takes (a read-back of a few
// tokens: 15.5 us of Python, 4.1 us here, 2.7 of them the launch).
#include <Python.h>

#include <initializer_list>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gdn.h"

namespace {

PyObject *g_error = nullptr;   // gdn.GdnError

// attn.KVCache's record: the ABI's struct, the heads and channels its pages were made for, and the device that they
// are on (-1: no pages).
struct Cache {
    gdn_kv_cache c;
    int32_t Hkv, D, device;
};

// A Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject *type, const std::string &text) {
    PyErr_SetString(type, text.c_str());
    throw Raised();
}

std::string show(c10::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const char *type_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

using Shape = std::initializer_list<int64_t>;

// One call: its stream, and the device that all of its tensors are on.
struct Call {
    const char *where;
    int device = -1;
    PyObject *stream_arg;

    Call(const char *w, PyObject *s) : where(w), stream_arg(s) {}

    const at::Tensor &tensor(PyObject *o, at::ScalarType type, const char *name) {
        if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.scalar_type() != type)
            raise(PyExc_TypeError, std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
        return t;
    }

    void shaped(const at::Tensor &t, Shape want, const char *name) {
        if (t.sizes() != c10::IntArrayRef(want.begin(), want.size()))
            raise(PyExc_ValueError, std::string(name) + " must have shape " +
                                        show(c10::IntArrayRef(want.begin(), want.size())) + ", got " + show(t.sizes()));
    }

    void placed(const at::Tensor &t, const char *name) {
        if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
        placed(t.device().index(), name);
    }

    void placed(int d, const char *name) {
        if (device < 0) device = d;
        if (d != device) raise(PyExc_ValueError, std::string(name) + " is on another device than the tensors before it");
    }

    // a dense tensor's address; None gives null if it may
    void *dense(PyObject *o, at::ScalarType type, Shape want, const char *name, bool optional = false) {
        if (optional && o == Py_None) return nullptr;
        const at::Tensor &t = tensor(o, type, name);
        shaped(t, want, name);
        return address(t, name);
    }

    void *address(const at::Tensor &t, const char *name) {
        if (t.numel() == 0) return nullptr;
        placed(t, name);
        if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
        return t.data_ptr();
    }

    struct Heads {
        const uint16_t *p;
        int64_t ts, hs;
    };

    // a [B, T, heads, D] view: dense channels, one token stride over all rows, one head stride
    Heads heads(PyObject *o, const gdn_attn_dims &d, int64_t H, const char *name) {
        const at::Tensor &t = tensor(o, at::kBFloat16, name);
        shaped(t, {d.B, d.T, H, d.D}, name);
        if (t.numel() == 0) return {nullptr, 0, 0};
        int64_t ts = t.stride(1), hs = t.stride(2);
        if (d.T == 1)
            ts = d.B > 1 ? t.stride(0) : 0;
        else if (d.B > 1 && t.stride(0) != d.T * ts)
            raise(PyExc_ValueError, std::string(name) + ": its rows must follow each other at one token stride, got strides " +
                                        show(t.strides()));
        if (H == 1) hs = 0;
        if (t.stride(3) != 1 || ts % 8 != 0 || hs % 8 != 0)
            raise(PyExc_ValueError, std::string(name) + " must have dense channels and token and head strides that are "
                                                        "multiples of 8, got strides " + show(t.strides()));
        placed(t, name);
        return {static_cast<const uint16_t *>(t.data_ptr()), ts, hs};
    }

    // the stream of the call: the given handle, else torch's current one
    cudaStream_t stream() {
        if (device < 0) device = c10::cuda::current_device();
        if (device != c10::cuda::current_device())
            raise(PyExc_ValueError, std::string(where) + ": the tensors are not on the current device");
        if (stream_arg == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
        const unsigned long long v = PyLong_AsUnsignedLongLongMask(stream_arg);
        if (PyErr_Occurred()) throw Raised();
        return reinterpret_cast<cudaStream_t>(v);
    }

    // a block of the caching allocator for work on the call's stream.  It comes from that stream's own pool: one of the
    // current stream's may still be in use by work queued there, which a given stream does not wait for.  The current
    // stream, on which the caller will use it, is recorded: the block is not given out again before it is done with it.
    c10::DataPtr block(size_t bytes) {
        auto *from = c10::cuda::CUDACachingAllocator::get();
        if (stream_arg == Py_None) return from->allocate(bytes);
        const auto d = (c10::DeviceIndex)device;
        const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(d),
                                    on = c10::cuda::getStreamFromExternal(stream(), d);
        if (on.stream() == current.stream()) return from->allocate(bytes);
        c10::cuda::CUDAStreamGuard guard(on);
        c10::DataPtr p = from->allocate(bytes);
        c10::cuda::CUDACachingAllocator::recordStream(p, current);
        return p;
    }

    // a new tensor on the call's device.  Made from the allocator's block directly: through the dispatcher each output of
    // a call took 2.3 us of host time, so 0.7.
    at::Tensor fresh(Shape shape, at::ScalarType type) {
        int64_t n = 1;
        for (int64_t s : shape) n *= s;
        const c10::IntArrayRef sizes(shape.begin(), shape.size());
        if (n == 0 || device < 0 || device != c10::cuda::current_device())
            return at::empty(sizes, at::TensorOptions().dtype(type).device(c10::Device(
                                        c10::kCUDA, (c10::DeviceIndex)(device < 0 ? c10::cuda::current_device() : device))));
        auto *from = c10::cuda::CUDACachingAllocator::get();
        const size_t bytes = (size_t)n * c10::elementSize(type);
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
            c10::Storage(c10::Storage::use_byte_size_t(), bytes, block(bytes), from, /*resizable=*/true),
            c10::DispatchKeySet(c10::DispatchKey::CUDA), c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
        return t;
    }

    // an output: the given tensor, or a new one
    at::Tensor output(PyObject *o, at::ScalarType type, Shape want, const char *name) {
        if (o == Py_None) return fresh(want, type);
        const at::Tensor &t = tensor(o, type, name);
        shaped(t, want, name);
        address(t, name);
        return t;
    }

    void done(gdn_status s) {
        if (s == GDN_OK) return;
        PyObject *e = PyObject_CallFunction(g_error, "is", (int)s, where);
        if (e != nullptr) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
        throw Raised();
    }
};

// A call's scratch: the caller's tensor, or a block that goes back to the allocator, for later work of this stream,
// when the call has been queued.
struct Scratch {
    void *p = nullptr;
    size_t bytes = 0;
    bool own = false;

    void given(Call &c, PyObject *o) {
        const at::Tensor &t = c.tensor(o, at::kByte, "workspace");
        p = c.address(t, "workspace");
        bytes = (size_t)t.numel();
    }
    void make(Call &c, size_t n) {
        const cudaStream_t st = c.stream();
        if (n == 0) return;
        p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(n, st);
        bytes = n;
        own = true;
    }
    Scratch() = default;
    Scratch(const Scratch &) = delete;
    ~Scratch() {
        if (own) c10::cuda::CUDACachingAllocator::raw_delete(p);
    }
};

template <typename T>
T *at_address(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (p == nullptr) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null record");
        throw Raised();
    }
    return static_cast<T *>(p);
}

void *data(const at::Tensor &t) { return t.numel() == 0 ? nullptr : t.data_ptr(); }
uint16_t *bf16(const at::Tensor &t) { return static_cast<uint16_t *>(data(t)); }
float *f32(const at::Tensor &t) { return static_cast<float *>(data(t)); }

struct Norm {
    const float *wq, *wk;
    const uint64_t *freqs;
};

Norm norm_args(Call &c, const gdn_attn_dims &d, PyObject *wq, PyObject *wk, PyObject *freqs) {
    return {static_cast<float *>(c.dense(wq, at::kFloat, {d.D}, "wq", true)),
            static_cast<float *>(c.dense(wk, at::kFloat, {d.D}, "wk", true)),
            static_cast<uint64_t *>(c.dense(freqs, at::kLong, {d.Drot / 2}, "freqs", true))};
}

struct Pages {
    const gdn_kv_cache *c;
    const int32_t *table;
    int32_t width;
};

Pages page_args(Call &c, const gdn_attn_dims &d, PyObject *cache, PyObject *table) {
    const Cache *k = at_address<Cache>(cache);
    if (k->Hkv != d.Hkv || k->D != d.D)
        raise(PyExc_ValueError, std::string(c.where) + ": the cache holds " + std::to_string(k->Hkv) + " heads of " +
                                    std::to_string(k->D) + " channels, the dims say " + std::to_string(d.Hkv) + " of " +
                                    std::to_string(d.D));
    if (k->device >= 0) c.placed(k->device, "the cache");
    const at::Tensor &t = c.tensor(table, at::kInt, "page_table");
    if (t.dim() != 2 || t.size(0) != d.B || t.size(1) > 0x7fffffff)
        raise(PyExc_ValueError, std::string(c.where) + ": page_table must have shape (" + std::to_string(d.B) +
                                    ", width), got " + show(t.sizes()));
    return {&k->c, static_cast<const int32_t *>(c.address(t, "page_table")), (int32_t)t.size(1)};
}

int32_t *index_arg(Call &c, PyObject *o, int64_t n, const char *name, bool optional = false) {
    return static_cast<int32_t *>(c.dense(o, at::kInt, {n}, name, optional));
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b) {
    PyObject *t = PyTuple_New(2);
    if (t == nullptr) throw Raised();
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
    return t;
}

// (dims, q, k, wq, wk, freqs, pos, mask, q_out, k_out, stream) -> (q_out, k_out)
PyObject *qk_norm_rope(PyObject *const *a) {
    const gdn_attn_dims &d = *at_address<gdn_attn_dims>(a[0]);
    Call c("gdn_qk_norm_rope", a[10]);
    const auto q = c.heads(a[1], d, d.Hq, "q"), k = c.heads(a[2], d, d.Hkv, "k");
    const Norm n = norm_args(c, d, a[3], a[4], a[5]);
    const auto *pos = static_cast<int32_t *>(c.dense(a[6], at::kInt, {d.B, d.T}, "pos"));
    const auto *mask = static_cast<uint8_t *>(c.dense(a[7], at::kByte, {d.B, d.T}, "mask", true));
    const at::Tensor qo = c.output(a[8], at::kBFloat16, {d.B, d.T, d.Hq, d.D}, "q_out");
    const at::Tensor ko = c.output(a[9], at::kBFloat16, {d.B, d.T, d.Hkv, d.D}, "k_out");
    c.done(gdn_qk_norm_rope(&d, q.p, q.ts, q.hs, k.p, k.ts, k.hs, n.wq, n.wk, n.freqs, pos, mask, bf16(qo), bf16(ko),
                            (gdn_stream)c.stream()));
    return pair(qo, ko);
}

// (dims, q, k, wq, wk, freqs, pos, mask, dq_out, dk_out, dq, dk, dwq, dwk, workspace, stream) -> (dq, dk, dwq, dwk)
PyObject *qk_norm_rope_backward(PyObject *const *a) {
    const gdn_attn_dims &d = *at_address<gdn_attn_dims>(a[0]);
    Call c("gdn_qk_norm_rope_backward", a[15]);
    const auto q = c.heads(a[1], d, d.Hq, "q"), k = c.heads(a[2], d, d.Hkv, "k");
    const Norm n = norm_args(c, d, a[3], a[4], a[5]);
    const auto *pos = static_cast<int32_t *>(c.dense(a[6], at::kInt, {d.B, d.T}, "pos"));
    const auto *mask = static_cast<uint8_t *>(c.dense(a[7], at::kByte, {d.B, d.T}, "mask", true));
    const auto *dqo = static_cast<uint16_t *>(c.dense(a[8], at::kBFloat16, {d.B, d.T, d.Hq, d.D}, "dq_out"));
    const auto *dko = static_cast<uint16_t *>(c.dense(a[9], at::kBFloat16, {d.B, d.T, d.Hkv, d.D}, "dk_out"));
    const at::Tensor dq = c.output(a[10], at::kBFloat16, {d.B, d.T, d.Hq, d.D}, "dq");
    const at::Tensor dk = c.output(a[11], at::kBFloat16, {d.B, d.T, d.Hkv, d.D}, "dk");
    at::Tensor dwq, dwk;
    Scratch ws;
    if (n.wq != nullptr || a[12] != Py_None) dwq = c.output(a[12], at::kFloat, {d.D}, "dwq");
    if (n.wk != nullptr || a[13] != Py_None) dwk = c.output(a[13], at::kFloat, {d.D}, "dwk");
    if (a[14] != Py_None)
        ws.given(c, a[14]);
    else if (n.wq != nullptr)
        ws.make(c, gdn_qk_norm_rope_backward_workspace_size(&d));
    c.done(gdn_qk_norm_rope_backward(&d, q.p, q.ts, q.hs, k.p, k.ts, k.hs, n.wq, n.wk, n.freqs, pos, mask, dqo, dko,
                                     bf16(dq), bf16(dk), dwq.defined() ? f32(dwq) : nullptr,
                                     dwk.defined() ? f32(dwk) : nullptr, ws.p, ws.bytes,
                                     (gdn_stream)c.stream()));
    PyObject *t = PyTuple_New(4);
    if (t == nullptr) throw Raised();
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(dq));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(dk));
    PyTuple_SET_ITEM(t, 2, dwq.defined() ? THPVariable_Wrap(dwq) : Py_NewRef(Py_None));
    PyTuple_SET_ITEM(t, 3, dwk.defined() ? THPVariable_Wrap(dwk) : Py_NewRef(Py_None));
    return t;
}

// (dims, q, k, v, wq, wk, freqs, cache, page_table, pos, n_new, q_out, stream) -> q_out
PyObject *kv_append(PyObject *const *a) {
    const gdn_attn_dims &d = *at_address<gdn_attn_dims>(a[0]);
    Call c("gdn_kv_append", a[12]);
    const auto q = c.heads(a[1], d, d.Hq, "q"), k = c.heads(a[2], d, d.Hkv, "k"), v = c.heads(a[3], d, d.Hkv, "v");
    const Norm n = norm_args(c, d, a[4], a[5], a[6]);
    const Pages pg = page_args(c, d, a[7], a[8]);
    const int32_t *pos = index_arg(c, a[9], d.B, "pos"), *n_new = index_arg(c, a[10], d.B, "n_new", true);
    const at::Tensor qo = c.output(a[11], at::kBFloat16, {d.B, d.T, d.Hq, d.D}, "q_out");
    c.done(gdn_kv_append(&d, q.p, q.ts, q.hs, k.p, k.ts, k.hs, v.p, v.ts, v.hs, n.wq, n.wk, n.freqs, pg.c, pg.table,
                         pg.width, pos, n_new, bf16(qo), (gdn_stream)c.stream()));
    return THPVariable_Wrap(qo);
}

// (dims, cache, page_table, start, n, k_out, v_out, stream) -> (k_out, v_out)
PyObject *kv_read(PyObject *const *a) {
    const gdn_attn_dims &d = *at_address<gdn_attn_dims>(a[0]);
    Call c("gdn_kv_read", a[7]);
    const Pages pg = page_args(c, d, a[1], a[2]);
    const int32_t *start = index_arg(c, a[3], d.B, "start"), *n = index_arg(c, a[4], d.B, "n", true);
    const at::Tensor ko = c.output(a[5], at::kBFloat16, {d.B, d.T, d.Hkv, d.D}, "k_out");
    const at::Tensor vo = c.output(a[6], at::kBFloat16, {d.B, d.T, d.Hkv, d.D}, "v_out");
    c.done(gdn_kv_read(&d, pg.c, pg.table, pg.width, start, n, bf16(ko), bf16(vo), (gdn_stream)c.stream()));
    return pair(ko, vo);
}

// (dims, q, cache, page_table, pos, n_new, gate, scale, out, lse, want_lse, workspace, stream) -> out or (out, lse)
PyObject *attn_decode(PyObject *const *a) {
    const gdn_attn_dims &d = *at_address<gdn_attn_dims>(a[0]);
    Call c("gdn_attn_decode", a[12]);
    const auto *q = static_cast<uint16_t *>(c.dense(a[1], at::kBFloat16, {d.B, d.T, d.Hq, d.D}, "q"));
    const Pages pg = page_args(c, d, a[2], a[3]);
    const int32_t *pos = index_arg(c, a[4], d.B, "pos"), *n_new = index_arg(c, a[5], d.B, "n_new", true);
    const Call::Heads gate = a[6] == Py_None ? Call::Heads{nullptr, 0, 0} : c.heads(a[6], d, d.Hq, "gate");
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised();
    const at::Tensor out = c.output(a[8], at::kBFloat16, {d.B, d.T, d.Hq, d.D}, "out");
    at::Tensor lse;
    Scratch ws;
    if (a[10] == Py_True || a[9] != Py_None) lse = c.output(a[9], at::kFloat, {d.B, d.T, d.Hq}, "lse");
    if (a[11] != Py_None)
        ws.given(c, a[11]);
    else
        ws.make(c, gdn_attn_decode_workspace_size(&d));
    c.done(gdn_attn_decode(&d, q, pg.c, pg.table, pg.width, pos, n_new, gate.p, gate.ts, gate.hs, (float)scale, bf16(out),
                           lse.defined() ? f32(lse) : nullptr, ws.p, ws.bytes, (gdn_stream)c.stream()));
    return lse.defined() && a[10] == Py_True ? pair(out, lse) : THPVariable_Wrap(out);
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_XDECREF(g_error);
    g_error = Py_NewRef(cls);
    Py_RETURN_NONE;
}

#define ENTRY(f, n) {#f, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(qk_norm_rope, 11), ENTRY(qk_norm_rope_backward, 16), ENTRY(kv_append, 13),
                         ENTRY(kv_read, 8), ENTRY(attn_decode, 13),
                         {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_attn_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_bind(void) { return PyModule_Create(&module_def); }
