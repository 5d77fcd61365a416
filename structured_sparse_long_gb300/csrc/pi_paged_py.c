/*
 * pi_paged_py.c -- CPython side of the paged cache's calls: argument checks, output allocation and the call of the C
 * ABI (include/pi_attn.h) in one native function each.
 *
 * A serving step makes these calls for every layer, and its kernels take a few microseconds: checks and marshalling in
 * Python and ctypes took longer than they do.  On the host an append takes 4.4 us (6.9 with both in Python, tuned), a decode
 * step 4.5 us with its outputs given and 9 without, most of the difference being torch's for two new tensors.  Tensors are reached through their
 * Python methods, so nothing here depends on torch's headers or binary interface.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "pi_attn.h"

/* What a PagedCache hands over: its pages, and the device index that its tensors answer get_device() with. */
typedef struct {
    pi_attn_cache_t cache;
    int device;
} handle_t;

typedef int (*append_fn)(const void *, const void *, long long, long long, const pi_attn_cache_t *, const pi_attn_batch_t *, void *);
typedef int (*read_fn)(const pi_attn_cache_t *, const pi_attn_batch_t *, void *, void *, void *);
typedef size_t (*extend_size_fn)(const pi_attn_cache_t *, int, int, int, int, int, int, int, int);
typedef int (*extend_fn)(const void *, long long, const pi_attn_cache_t *, const pi_attn_batch_t *, const float *, int, int, int, int,
                         int, void *, float *, void *, size_t, void *);
typedef int (*decode_fn)(const void *, long long, const pi_attn_cache_t *, const int *, const int *, int, int, const float *, int, int,
                         int, int, int, void *, float *, void *);

static append_fn f_append;
static read_fn f_read;
static extend_size_fn f_extend_size;
static extend_fn f_extend;
static decode_fn f_decode;

static PyObject *g_bf16, *g_fp32, *g_int32, *g_uint8, *g_empty, *g_empty_like;                   /* torch's objects */
static PyObject *s_data_ptr, *s_dtype, *s_shape, *s_stride, *s_get_device, *s_is_contiguous;     /* interned names */
static PyObject *kw_empty;                                                                       /* ("dtype", "device") */

/* ValueError: `name` must be `want`, got (what it is). */
static int refuse(PyObject *t, const char *name, const char *want) {
    PyErr_Clear();
    PyObject *dtype = PyObject_GetAttr(t, s_dtype), *shape = dtype ? PyObject_GetAttr(t, s_shape) : NULL;
    PyObject *stride = shape ? PyObject_CallMethodNoArgs(t, s_stride) : NULL;
    PyObject *device = stride ? PyObject_GetAttrString(t, "device") : NULL;
    if (device) {
        PyErr_Format(PyExc_ValueError, "%s must be %s, got %S %S with strides %S on %S", name, want, dtype, shape, stride, device);
    } else {
        PyErr_Clear();
        PyErr_Format(PyExc_ValueError, "%s must be %s, got %s", name, want, Py_TYPE(t)->tp_name);
    }
    Py_XDECREF(dtype);
    Py_XDECREF(shape);
    Py_XDECREF(stride);
    Py_XDECREF(device);
    return -1;
}

/* obj.name() as a number; *ok is cleared on an error. */
static long long call_int(PyObject *obj, PyObject *name, int *ok) {
    PyObject *r = PyObject_CallMethodNoArgs(obj, name);
    long long v = -1;
    if (r) {
        v = (long long)PyLong_AsUnsignedLongLongMask(r);
        Py_DECREF(r);
    }
    if (!r || PyErr_Occurred()) *ok = 0;
    return v;
}

/* A tuple's `n` numbers (tuple: obj.name, or obj.name() if `call`); whether there are as many. */
static int numbers(PyObject *obj, PyObject *name, int call, int n, long long *out) {
    PyObject *t = call ? PyObject_CallMethodNoArgs(obj, name) : PyObject_GetAttr(obj, name);
    int ok = t && PyTuple_Check(t) && PyTuple_GET_SIZE(t) == n;
    for (int i = 0; ok && i < n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        ok = !(out[i] == -1 && PyErr_Occurred());
    }
    Py_XDECREF(t);
    if (!ok) PyErr_Clear();
    return ok;
}

static int has_dtype(PyObject *t, PyObject *dtype) {
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    const int same = d == dtype;
    if (!d) PyErr_Clear();
    Py_XDECREF(d);
    return same;
}

/* A contiguous tensor of a given type and shape (n <= 3 sizes; a negative one is taken from the tensor) on the cache's device:
 * its address, or NULL with a ValueError. */
static void *dense(PyObject *t, const char *name, const handle_t *h, PyObject *dtype, int n, long long *shape, const char *want) {
    long long got[3];
    int ok = has_dtype(t, dtype) && numbers(t, s_shape, 0, n, got);
    for (int i = 0; ok && i < n; ++i) {
        if (shape[i] < 0) shape[i] = got[i];
        ok = shape[i] == got[i];
    }
    if (ok) ok = call_int(t, s_get_device, &ok) == h->device && ok;
    if (ok) {
        PyObject *c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
        ok = c == Py_True;
        Py_XDECREF(c);
    }
    void *p = ok ? (void *)(uintptr_t)call_int(t, s_data_ptr, &ok) : NULL;
    if (!ok) {
        refuse(t, name, want);
        return NULL;
    }
    return p ? p : (void *)h;  /* an empty tensor: some address, for a call that is not made */
}

/* A packed [T, heads, d] bf16 tensor whose tokens are contiguous (heads < 0: taken from it): its address and the stride
 * between tokens; -1 with a ValueError. */
static int packed(PyObject *t, const char *name, const handle_t *h, long long *T, long long *heads, long long *stride, void **p) {
    long long shape[3], st[3];
    int ok = has_dtype(t, g_bf16) && numbers(t, s_shape, 0, 3, shape) && shape[2] == h->cache.d && (*heads < 0 || shape[1] == *heads);
    if (ok) ok = call_int(t, s_get_device, &ok) == h->device && ok;
    if (!ok) return refuse(t, name, "bf16 [T, heads, d] with the cache's head count and size, on its device");
    if (!numbers(t, s_stride, 1, 3, st) || st[2] != 1 || (shape[1] > 1 && st[1] != shape[2]))
        return refuse(t, name, "a tensor whose tokens have contiguous elements");
    *T = shape[0];
    *heads = shape[1];
    *stride = shape[0] > 1 ? st[0] : shape[1] * shape[2];
    *p = (void *)(uintptr_t)call_int(t, s_data_ptr, &ok);
    return ok ? 0 : -1;
}

/* torch.empty(shape, dtype=dtype, device=the cache's index) */
static PyObject *empty(const handle_t *h, PyObject *dtype, int n, const long long *shape) {
    PyObject *size = PyTuple_New(n), *device = PyLong_FromLong(h->device), *r = NULL;
    int ok = size && device;
    for (int i = 0; ok && i < n; ++i) {
        PyObject *x = PyLong_FromLongLong(shape[i]);
        ok = x != NULL;
        if (ok) PyTuple_SET_ITEM(size, i, x);
    }
    if (ok) {
        PyObject *args[3] = {size, dtype, device};
        r = PyObject_Vectorcall(g_empty, args, 1, kw_empty);
    }
    Py_XDECREF(size);
    Py_XDECREF(device);
    return r;
}

/* The caller's output buffer, checked, or (None) a new one: a new reference in *out.  like: a tensor of its type, shape and
 * device, or NULL (a decode call takes 9.0 us on the host with empty_like and 12.5 with empty).  Its strides fall from size to
 * size, whatever their gaps, so what is like it is contiguous. */
static void *output(PyObject *given, const char *name, const handle_t *h, PyObject *dtype, int n, long long *shape, const char *want,
                    PyObject *like, PyObject **out) {
    if (given == Py_None) {
        int ok = 1;
        if (!(*out = like ? PyObject_CallOneArg(g_empty_like, like) : empty(h, dtype, n, shape))) return NULL;
        void *p = (void *)(uintptr_t)call_int(*out, s_data_ptr, &ok);
        if (ok) return p ? p : (void *)h;
    } else {
        void *p = dense(given, name, h, dtype, n, shape, want);
        if (p) {
            Py_INCREF(given);
            *out = given;
            return p;
        }
    }
    Py_CLEAR(*out);
    return NULL;
}

static handle_t *handle_of(PyObject *o) { return (handle_t *)PyLong_AsVoidPtr(o); }

/* The batch's device tensors. */
static int batch(PyObject *table, PyObject *cu, PyObject *ctx, long long T, const handle_t *h, pi_attn_batch_t *b) {
    long long s[2] = {-1, -1};
    if (!(b->table = dense(table, "table", h, g_int32, 2, s, "a contiguous int32 [B, width] on the cache's device"))) return -1;
    b->B = (int)s[0];
    b->width = (int)s[1];
    long long n = s[0] + 1;
    if (!(b->cu = dense(cu, "cu", h, g_int32, 1, &n, "a contiguous int32 [B + 1] on the cache's device"))) return -1;
    if (!(b->ctx = dense(ctx, "ctx", h, g_int32, 1, s, "a contiguous int32 [B] on the cache's device"))) return -1;
    if (T > INT32_MAX || s[0] > INT32_MAX || s[1] > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "more than 2^31 - 1 tokens, sequences or page-table entries");
        return -1;
    }
    b->T = (int)T;
    return 0;
}

/* Whole numbers of the call (k_local, period, S, mode). */
static int ints(PyObject *const *args, int n, int *out) {
    for (int i = 0; i < n; ++i) {
        const long long v = PyLong_AsLongLong(args[i]);
        if (v == -1 && PyErr_Occurred()) return -1;
        if (v < INT32_MIN || v > INT32_MAX) {
            PyErr_SetString(PyExc_ValueError, "k_local, period, S and mode are 32-bit numbers");
            return -1;
        }
        out[i] = (int)v;
    }
    return 0;
}

/* append(k, v, handle, table, cu, ctx, stream) -> status */
static PyObject *py_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 7) return PyErr_Format(PyExc_TypeError, "append takes 7 arguments");
    const handle_t *h = handle_of(a[2]);
    long long T, Tv, heads, ks, vs;
    void *k, *v, *stream = PyLong_AsVoidPtr(a[6]);
    pi_attn_batch_t b;
    if (PyErr_Occurred()) return NULL;
    heads = h->cache.Hkv;
    if (packed(a[0], "k", h, &T, &heads, &ks, &k) || packed(a[1], "v", h, &Tv, &heads, &vs, &v)) return NULL;
    if (T != Tv) {
        refuse(a[1], "v", "as long as k");
        return NULL;
    }
    if (batch(a[3], a[4], a[5], T, h, &b)) return NULL;
    return PyLong_FromLong(T ? f_append(k, v, ks, vs, &h->cache, &b, stream) : PI_OK);
}

/* read(handle, table, cu, start, rows, k, v, stream) -> (status, k, v) */
static PyObject *py_read(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 8) return PyErr_Format(PyExc_TypeError, "read takes 8 arguments");
    const handle_t *h = handle_of(a[0]);
    const long long rows = PyLong_AsLongLong(a[4]);
    void *stream = PyLong_AsVoidPtr(a[7]), *pk, *pv;
    pi_attn_batch_t b;
    PyObject *k = NULL, *v = NULL, *r = NULL;
    if (PyErr_Occurred()) return NULL;
    if (rows < 0) return PyErr_Format(PyExc_ValueError, "rows must not be negative");
    long long shape[3] = {rows, h->cache.Hkv, h->cache.d};
    const char *want = "a contiguous bf16 [rows, Hkv, d] on the cache's device";
    if ((pk = output(a[5], "k", h, g_bf16, 3, shape, want, NULL, &k)) && (pv = output(a[6], "v", h, g_bf16, 3, shape, want, k, &v)) &&
        !batch(a[1], a[2], a[3], rows, h, &b))
        r = Py_BuildValue("iOO", rows ? f_read(&h->cache, &b, pk, pv, stream) : PI_OK, k, v);
    Py_XDECREF(k);
    Py_XDECREF(v);
    return r;
}

/* alpha's address (NULL for None), out and lse of an attention's T rows: 0, or -1 with an error. */
static int rows_of(PyObject *q, PyObject *alpha, PyObject *out, PyObject *lse, const handle_t *h, long long T, long long H, int mode,
                   float **pa, void **po, float **pl, PyObject **o, PyObject **l) {
    long long s2[2] = {T, H}, s3[3] = {T, H, h->cache.d};
    *pa = NULL;
    if (alpha != Py_None) {
        if (!(*pa = dense(alpha, "alpha", h, g_fp32, 2, s2, "a contiguous fp32 [T, H] on the cache's device"))) return -1;
    } else if (mode != PI_MODE_ECP) {
        PyErr_SetString(PyExc_ValueError, "alpha is needed in pi mode");
        return -1;
    }
    if (!(*po = output(out, "out", h, g_bf16, 3, s3, "a contiguous bf16 [T, H, d] on the cache's device", q, o))) return -1;
    PyObject *like = alpha != Py_None ? alpha : NULL;
    if (!(*pl = output(lse, "lse", h, g_fp32, 2, s2, "a contiguous fp32 [T, H] on the cache's device", like, l))) return -1;
    return 0;
}

/* extend(q, handle, table, cu, ctx, alpha, k_local, period, S, mode, out, lse, workspace, stream) -> (status, out, lse) */
static PyObject *py_extend(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 14) return PyErr_Format(PyExc_TypeError, "extend takes 14 arguments");
    const handle_t *h = handle_of(a[1]);
    long long T, H = -1, qs;
    int p[4];
    void *q, *out, *stream = PyLong_AsVoidPtr(a[13]), *ws = NULL;
    float *alpha, *lse;
    pi_attn_batch_t b;
    PyObject *o = NULL, *l = NULL, *w = NULL, *r = NULL;
    if (PyErr_Occurred() || ints(a + 6, 4, p) || packed(a[0], "q", h, &T, &H, &qs, &q) || batch(a[2], a[3], a[4], T, h, &b)) return NULL;
    if (rows_of(a[0], a[5], a[10], a[11], h, T, H, p[3], &alpha, &out, &lse, &o, &l)) goto done;
    if (T == 0) {
        r = Py_BuildValue("iOO", PI_OK, o, l);
        goto done;
    }
    const size_t need = f_extend_size(&h->cache, b.B, b.T, b.width, (int)H, p[0], p[1], p[2], p[3]);
    long long bytes = (long long)need;
    if (a[12] != Py_None) {
        bytes = -1;
        if (!(ws = dense(a[12], "workspace", h, g_uint8, 1, &bytes, "a contiguous uint8 vector on the cache's device"))) goto done;
        if (bytes < (long long)need) {
            PyErr_Format(PyExc_ValueError, "workspace must hold %zu bytes, got %lld", need, bytes);
            goto done;
        }
    } else if (need && !(ws = output(Py_None, "workspace", h, g_uint8, 1, &bytes, "", NULL, &w))) {
        goto done;
    }
    r = Py_BuildValue("iOO",
                      f_extend(q, qs, &h->cache, &b, alpha, (int)H, p[0], p[1], p[2], p[3], out, lse, ws, (size_t)bytes, stream), o, l);
done:
    Py_XDECREF(o);
    Py_XDECREF(l);
    Py_XDECREF(w);
    return r;
}

/* decode(q, handle, table, lens, alpha, k_local, period, S, mode, out, lse, stream) -> (status, out, lse) */
static PyObject *py_decode(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 12) return PyErr_Format(PyExc_TypeError, "decode takes 12 arguments");
    const handle_t *h = handle_of(a[1]);
    long long B, H = -1, qs, s[2];
    int p[4];
    void *q, *out, *table, *lens, *stream = PyLong_AsVoidPtr(a[11]);
    float *alpha, *lse;
    PyObject *o = NULL, *l = NULL, *r = NULL;
    if (PyErr_Occurred() || ints(a + 5, 4, p) || packed(a[0], "q", h, &B, &H, &qs, &q)) return NULL;
    s[0] = B;
    s[1] = -1;
    if (!(table = dense(a[2], "table", h, g_int32, 2, s, "a contiguous int32 [B, width] on the cache's device")) ||
        !(lens = dense(a[3], "lens", h, g_int32, 1, s, "a contiguous int32 [B] on the cache's device")))
        return NULL;
    if (B > INT32_MAX || s[1] > INT32_MAX) return PyErr_Format(PyExc_ValueError, "more than 2^31 - 1 sequences or page-table entries");
    if (!rows_of(a[0], a[4], a[9], a[10], h, B, H, p[3], &alpha, &out, &lse, &o, &l))
        r = Py_BuildValue("iOO",
                          B ? f_decode(q, qs, &h->cache, table, lens, (int)B, (int)s[1], alpha, (int)H, p[0], p[1], p[2], p[3], out, lse,
                                       stream)
                            : PI_OK,
                          o, l);
    Py_XDECREF(o);
    Py_XDECREF(l);
    return r;
}

/* bind(append, read, extend size, extend, decode: addresses; bfloat16, float32, int32, uint8, empty, empty_like: torch's) */
static PyObject *py_bind(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 11) return PyErr_Format(PyExc_TypeError, "bind takes 11 arguments");
    void *f[5];
    for (int i = 0; i < 5; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return NULL;
    f_append = (append_fn)f[0];
    f_read = (read_fn)f[1];
    f_extend_size = (extend_size_fn)f[2];
    f_extend = (extend_fn)f[3];
    f_decode = (decode_fn)f[4];
    PyObject **slots[6] = {&g_bf16, &g_fp32, &g_int32, &g_uint8, &g_empty, &g_empty_like};
    for (int i = 0; i < 6; ++i) {
        Py_INCREF(a[5 + i]);
        Py_XSETREF(*slots[i], a[5 + i]);
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL, NULL},
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
    {"read", (PyCFunction)(void (*)(void))py_read, METH_FASTCALL, NULL},
    {"extend", (PyCFunction)(void (*)(void))py_extend, METH_FASTCALL, NULL},
    {"decode", (PyCFunction)(void (*)(void))py_decode, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pi_paged", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pi_paged(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    kw_empty = Py_BuildValue("(ss)", "dtype", "device");
    if (!s_data_ptr || !s_dtype || !s_shape || !s_stride || !s_get_device || !s_is_contiguous || !kw_empty) return NULL;
    return PyModule_Create(&module);
}
