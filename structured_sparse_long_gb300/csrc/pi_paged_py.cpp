// pi_paged_py.cpp -- Python side of the paged cache's calls: argument checks, output allocation and the call of the C
// ABI (include/pi_attn.h) in one native function each.
//
// A serving step makes these calls for every layer, and its kernels take a few microseconds, so their host time is what a caller
// waits for.  Tensors are reached through torch's C++ interface: a check is a load, and a new tensor is made without parsing
// Python arguments.  Calls one after the other from Python, with new outputs each (the same through the tensors' Python
// methods, from C): one-token append 2.9 us (4.4), one-token attention 6.2 (9.5; its kernel takes 5.0), read of a ragged batch 7.6
// (10.8; its kernel 7.3).
// The interpreter lock is released where a call may wait (an allocation, a full launch queue).
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <cstdint>
#include <utility>

#include "pi_attn.h"

namespace {

// What a PagedCache hands over: its pages, and the device index of its tensors (-1: host).
struct Handle {
    pi_attn_cache_t cache;
    int device;
};

decltype(&pi_attn_cache_append) f_append;
decltype(&pi_attn_cache_read) f_read;
decltype(&pi_attn_extend_workspace_size) f_extend_size;
decltype(&pi_attn_extend) f_extend;
decltype(&pi_attn_decode_paged) f_decode;

struct Refused {};  // a Python exception is set

struct Unlocked {  // the interpreter lock, released
    PyThreadState *s = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(s); }
};

// ValueError: `name` must be `want`, got (what it is).
[[noreturn]] void refuse(PyObject *t, const char *name, const char *want) {
    if (THPVariable_Check(t)) {
        PyObject *dtype = PyObject_GetAttrString(t, "dtype"), *shape = dtype ? PyObject_GetAttrString(t, "shape") : nullptr;
        PyObject *device = shape ? PyObject_GetAttrString(t, "device") : nullptr;
        PyObject *stride = device ? PyObject_CallMethod(t, "stride", nullptr) : nullptr;
        PyErr_Clear();
        if (stride) PyErr_Format(PyExc_ValueError, "%s must be %s, got %S %S with strides %S on %S", name, want, dtype, shape, stride, device);
        else PyErr_Format(PyExc_ValueError, "%s must be %s, got another kind of tensor", name, want);
        for (PyObject *o : {dtype, shape, device, stride}) Py_XDECREF(o);
    } else {
        PyErr_Format(PyExc_ValueError, "%s must be %s, got %s", name, want, Py_TYPE(t)->tp_name);
    }
    throw Refused{};
}
[[noreturn]] void refuse(const char *what) {
    PyErr_SetString(PyExc_ValueError, what);
    throw Refused{};
}

// A strided tensor of `type` and `dims` dimensions on the cache's device, or null.
const at::Tensor *strided(PyObject *o, const Handle &h, at::ScalarType type, int64_t dims) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    return t.defined() && t.layout() == at::kStrided && t.scalar_type() == type && t.dim() == dims && t.get_device() == h.device ? &t : nullptr;
}

void *address(const at::Tensor &t, const Handle &h) {
    void *p = t.data_ptr();
    return p ? p : (void *)&h;  // an empty tensor: some address, for a call that is not made
}

// A contiguous tensor of a given type and shape (a negative size is taken from it) on the cache's device: its address.
template <int N>
void *dense(PyObject *o, const char *name, const Handle &h, at::ScalarType type, int64_t (&shape)[N], const char *want) {
    const at::Tensor *t = strided(o, h, type, N);
    if (!t || !t->is_contiguous()) refuse(o, name, want);
    for (int i = 0; i < N; ++i) {
        if (shape[i] < 0) shape[i] = t->size(i);
        if (shape[i] != t->size(i)) refuse(o, name, want);
    }
    return address(*t, h);
}

// A packed [T, heads, d] bf16 tensor whose tokens are contiguous (heads < 0: taken from it).
struct Packed {
    int64_t T, heads, stride;
    void *p;
};
Packed packed(PyObject *o, const char *name, const Handle &h, int64_t heads) {
    const at::Tensor *t = strided(o, h, at::kBFloat16, 3);
    if (!t || t->size(2) != h.cache.d || (heads >= 0 && t->size(1) != heads))
        refuse(o, name, "bf16 [T, heads, d] with the cache's head count and size, on its device");
    const int64_t T = t->size(0), n = t->size(1), d = t->size(2);
    if (t->stride(2) != 1 || (n > 1 && t->stride(1) != d)) refuse(o, name, "a tensor whose tokens have contiguous elements");
    return Packed{T, n, T > 1 ? t->stride(0) : n * d, address(*t, h)};
}

at::Tensor new_tensor(const Handle &h, at::ScalarType type, at::IntArrayRef shape) {
    const Unlocked u;
    return at::empty(shape, at::TensorOptions().dtype(type).device(h.device < 0 ? at::Device(at::kCPU) : at::Device(at::kCUDA, h.device)));
}

// An output: the caller's buffer, checked, or (None) a new tensor.
struct Output {
    PyObject *given = nullptr;
    at::Tensor made;
    void *p = nullptr;

    template <int N>
    Output(PyObject *o, const char *name, const Handle &h, at::ScalarType type, int64_t (&shape)[N], const char *want) {
        if (o != Py_None) {
            p = dense(o, name, h, type, shape, want);
            given = o;
        } else {
            made = new_tensor(h, type, shape);
            p = address(made, h);
        }
    }
    PyObject *take() { return given ? Py_NewRef(given) : THPVariable_Wrap(std::move(made)); }  // a new reference
};

// (status, x, y)
PyObject *results(int rc, Output &x, Output &y) {
    PyObject *items[3] = {PyLong_FromLong(rc), x.take(), y.take()};
    PyObject *r = items[0] && items[1] && items[2] ? PyTuple_New(3) : nullptr;
    for (int i = 0; i < 3; ++i) {
        if (r) PyTuple_SET_ITEM(r, i, items[i]);
        else Py_XDECREF(items[i]);
    }
    return r;
}

const Handle &handle_of(PyObject *o) {
    const void *p = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Refused{};
    return *static_cast<const Handle *>(p);
}
void *stream_of(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Refused{};
    return p;
}

// The batch's device tensors.
pi_attn_batch_t batch(PyObject *table, PyObject *cu, PyObject *ctx, int64_t T, const Handle &h) {
    int64_t s[2] = {-1, -1};
    pi_attn_batch_t b{};
    b.table = static_cast<const int *>(dense(table, "table", h, at::kInt, s, "a contiguous int32 [B, width] on the cache's device"));
    int64_t offsets[1] = {s[0] + 1}, seqs[1] = {s[0]};
    b.cu = static_cast<const int *>(dense(cu, "cu", h, at::kInt, offsets, "a contiguous int32 [B + 1] on the cache's device"));
    b.ctx = static_cast<const int *>(dense(ctx, "ctx", h, at::kInt, seqs, "a contiguous int32 [B] on the cache's device"));
    if (T > INT32_MAX || s[0] > INT32_MAX || s[1] > INT32_MAX) refuse("more than 2^31 - 1 tokens, sequences or page-table entries");
    b.B = (int)s[0];
    b.width = (int)s[1];
    b.T = (int)T;
    return b;
}

// k_local, period, S and mode.
struct Pattern {
    int v[4];
    explicit Pattern(PyObject *const *args) {
        for (int i = 0; i < 4; ++i) {
            const long long x = PyLong_AsLongLong(args[i]);
            if (x == -1 && PyErr_Occurred()) throw Refused{};
            if (x < INT32_MIN || x > INT32_MAX) refuse("k_local, period, S and mode are 32-bit numbers");
            v[i] = (int)x;
        }
    }
};

const float *alpha_of(PyObject *alpha, const Handle &h, int64_t T, int64_t H, int mode) {
    int64_t s[2] = {T, H};
    if (alpha != Py_None) return static_cast<const float *>(dense(alpha, "alpha", h, at::kFloat, s, "a contiguous fp32 [T, H] on the cache's device"));
    if (mode != PI_MODE_ECP) refuse("alpha is needed in pi mode");
    return nullptr;
}

// append(k, v, handle, table, cu, ctx, stream) -> status
PyObject *append(PyObject *const *a) {
    const Handle &h = handle_of(a[2]);
    void *stream = stream_of(a[6]);
    const Packed k = packed(a[0], "k", h, h.cache.Hkv), v = packed(a[1], "v", h, h.cache.Hkv);
    if (k.T != v.T) refuse(a[1], "v", "as long as k");
    const pi_attn_batch_t b = batch(a[3], a[4], a[5], k.T, h);
    int rc = PI_OK;
    if (k.T) {
        const Unlocked u;
        rc = f_append(k.p, v.p, k.stride, v.stride, &h.cache, &b, stream);
    }
    return PyLong_FromLong(rc);
}

// read(handle, table, cu, start, rows, k, v, stream) -> (status, k, v)
PyObject *read(PyObject *const *a) {
    const Handle &h = handle_of(a[0]);
    void *stream = stream_of(a[7]);
    const long long rows = PyLong_AsLongLong(a[4]);
    if (PyErr_Occurred()) throw Refused{};
    if (rows < 0) refuse("rows must not be negative");
    const pi_attn_batch_t b = batch(a[1], a[2], a[3], rows, h);
    int64_t shape[3] = {rows, h.cache.Hkv, h.cache.d};
    const char *want = "a contiguous bf16 [rows, Hkv, d] on the cache's device";
    Output k(a[5], "k", h, at::kBFloat16, shape, want), v(a[6], "v", h, at::kBFloat16, shape, want);
    int rc = PI_OK;
    if (rows) {
        const Unlocked u;
        rc = f_read(&h.cache, &b, k.p, v.p, stream);
    }
    return results(rc, k, v);
}

// extend(q, handle, table, cu, ctx, alpha, k_local, period, S, mode, out, lse, workspace, stream) -> (status, out, lse)
PyObject *extend(PyObject *const *a) {
    const Handle &h = handle_of(a[1]);
    void *stream = stream_of(a[13]);
    const Pattern p(a + 6);
    const Packed q = packed(a[0], "q", h, -1);
    const pi_attn_batch_t b = batch(a[2], a[3], a[4], q.T, h);
    const float *alpha = alpha_of(a[5], h, q.T, q.heads, p.v[3]);
    int64_t rows[2] = {q.T, q.heads}, shape[3] = {q.T, q.heads, h.cache.d};
    Output out(a[10], "out", h, at::kBFloat16, shape, "a contiguous bf16 [T, H, d] on the cache's device");
    Output lse(a[11], "lse", h, at::kFloat, rows, "a contiguous fp32 [T, H] on the cache's device");
    if (q.T == 0) return results(PI_OK, out, lse);
    const size_t need = f_extend_size(&h.cache, b.B, b.T, b.width, (int)q.heads, p.v[0], p.v[1], p.v[2], p.v[3]);
    int64_t bytes[1] = {a[12] != Py_None ? -1 : (int64_t)need};
    void *ws = nullptr;
    at::Tensor made;  // lives until the call is enqueued: the allocator hands it out again in the stream's order
    if (a[12] != Py_None) {
        ws = dense(a[12], "workspace", h, at::kByte, bytes, "a contiguous uint8 vector on the cache's device");
        if (bytes[0] < (int64_t)need) {
            PyErr_Format(PyExc_ValueError, "workspace must hold %zu bytes, got %lld", need, (long long)bytes[0]);
            throw Refused{};
        }
        if (bytes[0] == 0) ws = nullptr;  // (an empty tensor has no address; the call takes none where it needs none)
    } else if (need) {
        made = new_tensor(h, at::kByte, bytes);
        ws = made.data_ptr();
    }
    int rc;
    {
        const Unlocked u;
        rc = f_extend(q.p, q.stride, &h.cache, &b, alpha, (int)q.heads, p.v[0], p.v[1], p.v[2], p.v[3], out.p, static_cast<float *>(lse.p), ws,
                      (size_t)bytes[0], stream);
    }
    return results(rc, out, lse);
}

// decode(q, handle, table, lens, alpha, k_local, period, S, mode, out, lse, stream) -> (status, out, lse)
PyObject *decode(PyObject *const *a) {
    const Handle &h = handle_of(a[1]);
    void *stream = stream_of(a[11]);
    const Pattern p(a + 5);
    const Packed q = packed(a[0], "q", h, -1);
    int64_t pages[2] = {q.T, -1}, seqs[1] = {q.T};
    const int *table = static_cast<const int *>(dense(a[2], "table", h, at::kInt, pages, "a contiguous int32 [B, width] on the cache's device"));
    const int *lens = static_cast<const int *>(dense(a[3], "lens", h, at::kInt, seqs, "a contiguous int32 [B] on the cache's device"));
    if (q.T > INT32_MAX || pages[1] > INT32_MAX) refuse("more than 2^31 - 1 sequences or page-table entries");
    const float *alpha = alpha_of(a[4], h, q.T, q.heads, p.v[3]);
    int64_t rows[2] = {q.T, q.heads}, shape[3] = {q.T, q.heads, h.cache.d};
    Output out(a[9], "out", h, at::kBFloat16, shape, "a contiguous bf16 [T, H, d] on the cache's device");
    Output lse(a[10], "lse", h, at::kFloat, rows, "a contiguous fp32 [T, H] on the cache's device");
    int rc = PI_OK;
    if (q.T) {
        const Unlocked u;
        rc = f_decode(q.p, q.stride, &h.cache, table, lens, (int)q.T, (int)pages[1], alpha, (int)q.heads, p.v[0], p.v[1], p.v[2], p.v[3],
                      out.p, static_cast<float *>(lse.p), stream);
    }
    return results(rc, out, lse);
}

// bind(append, read, extend size, extend, decode): addresses of the library's functions
PyObject *bind(PyObject *const *a) {
    void *f[5];
    for (int i = 0; i < 5; ++i) f[i] = stream_of(a[i]);
    f_append = reinterpret_cast<decltype(f_append)>(f[0]);
    f_read = reinterpret_cast<decltype(f_read)>(f[1]);
    f_extend_size = reinterpret_cast<decltype(f_extend_size)>(f[2]);
    f_extend = reinterpret_cast<decltype(f_extend)>(f[3]);
    f_decode = reinterpret_cast<decltype(f_decode)>(f[4]);
    return Py_NewRef(Py_None);
}

// A function of N arguments for Python; no C++ exception leaves it.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    HANDLE_TH_ERRORS
    try {
        return F(a);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name) {
    return PyMethodDef{name, (PyCFunction)(void (*)(void))entry<F, N>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind, 5>("bind"),       method<append, 7>("append"),  method<read, 8>("read"),
                         method<extend, 14>("extend"),  method<decode, 12>("decode"), PyMethodDef{nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pi_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pi_paged(void) { return PyModule_Create(&module); }
