/*
 * pd_binding.c -- the quick way from torch tensors to libpd for the calls of a
 * decode step, where the launch takes 3 us and reading, checking and passing on
 * some forty properties in Python took 10.  A CPython module over the C API
 * alone (no torch headers): it reads the tensors' properties by name.
 *
 * Each function does what its namesake in api.py says for arguments that are
 * exactly as it needs them (types, shapes, strides, the current device and
 * stream) and returns NotImplemented for anything else, a failing library call
 * among it; api.py then takes its own path, which checks argument by argument
 * and raises what is wrong.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "pd.h"

/* Set once by setup(): torch.bfloat16, torch.uint8, torch.int32, torch.empty,
 * () -> current device, (device) -> its current stream. */
static PyObject *t_bf16, *t_u8, *t_i32, *t_empty, *t_device, *t_stream;
static PyObject *n_shape, *n_dtype, *n_device, *n_stride, *n_data_ptr, *n_get_device, *n_is_contiguous;
static PyObject *kw_empty; /* ("dtype", "device") */

/* What is read of a tensor. */
typedef struct {
    PyObject *dtype; /* borrowed: one of torch's own, which outlive every call */
    long long shape[4], stride[4];
    long long ptr;
} tensor;

static int read_tuple(PyObject *t, long long *v, int dim) {
    int ok = t && PyTuple_Check(t) && PyTuple_GET_SIZE(t) == dim;
    for (int i = 0; ok && i < dim; ++i) {
        v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        ok = !(v[i] == -1 && PyErr_Occurred());
    }
    Py_XDECREF(t);
    return ok;
}

static long long read_int(PyObject *t, PyObject *method) {
    PyObject *r = PyObject_CallMethodNoArgs(t, method);
    const long long v = r ? PyLong_AsLongLong(r) : -1;
    Py_XDECREF(r);
    return v;
}

/* t: a tensor of `dim` dimensions on device `dev`. */
static int read_tensor(PyObject *t, int dim, long long dev, tensor *o) {
    if (!read_tuple(PyObject_GetAttr(t, n_shape), o->shape, dim)) return 0;
    o->dtype = PyObject_GetAttr(t, n_dtype);
    if (!o->dtype) return 0;
    Py_DECREF(o->dtype);
    if (read_int(t, n_get_device) != dev) return 0;
    o->ptr = read_int(t, n_data_ptr);
    return !PyErr_Occurred();
}

/* A contiguous one of the given dtype. */
static int read_whole(PyObject *t, int dim, long long dev, PyObject *dtype, tensor *o) {
    if (!read_tensor(t, dim, dev, o) || o->dtype != dtype) return 0;
    PyObject *c = PyObject_CallMethodNoArgs(t, n_is_contiguous);
    Py_XDECREF(c);
    return c == Py_True;
}

/* BF16 rows [T, H, D], columns contiguous; side: a token's heads side by side. */
static int read_rows(PyObject *t, long long dev, int side, tensor *o) {
    if (!read_tensor(t, 3, dev, o) || o->dtype != t_bf16) return 0;
    if (!read_tuple(PyObject_CallMethodNoArgs(t, n_stride), o->stride, 3) || o->stride[2] != 1) return 0;
    if (o->shape[1] <= 1) o->stride[1] = o->shape[2];               /* (one head, one token: */
    if (o->shape[0] <= 1) o->stride[0] = o->shape[1] * o->shape[2]; /* any stride will do) */
    return !side || o->stride[1] == o->shape[2];
}

static int fits(long long v) { return v >= 0 && v <= 0x7fffffff; }

static long long current(PyObject *fn, long long arg, int with_arg) {
    PyObject *a = with_arg ? PyLong_FromLongLong(arg) : NULL;
    PyObject *r = with_arg ? PyObject_CallOneArg(fn, a) : PyObject_CallNoArgs(fn);
    const long long v = r ? PyLong_AsLongLong(r) : -1;
    Py_XDECREF(a);
    Py_XDECREF(r);
    return v;
}

/* torch.empty(like's shape or (n,), dtype=..., device=like.device) */
static PyObject *empty(PyObject *like, PyObject *shape, PyObject *dtype) {
    PyObject *s = shape ? Py_NewRef(shape) : PyObject_GetAttr(like, n_shape);
    PyObject *d = PyObject_GetAttr(like, n_device);
    PyObject *r = NULL;
    if (s && d) {
        PyObject *args[3] = {s, dtype, d};
        r = PyObject_Vectorcall(t_empty, args, 1, kw_empty);
    }
    Py_XDECREF(s);
    Py_XDECREF(d);
    return r;
}

/* The answer: `out` (a new reference) where the call went through. */
static PyObject *done(int rc, PyObject *out) {
    if (rc == PD_OK && !PyErr_Occurred()) return out;
    Py_XDECREF(out);
    PyErr_Clear();
    Py_RETURN_NOTIMPLEMENTED;
}
static PyObject *other_way(void) {
    PyErr_Clear();
    Py_RETURN_NOTIMPLEMENTED;
}

/* rope(handle, head_dim, x, positions, out | None, inverse) */
static PyObject *rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 6) return other_way();
    const long long handle = PyLong_AsLongLong(a[0]), head_dim = PyLong_AsLongLong(a[1]), inverse = PyLong_AsLongLong(a[5]);
    const long long dev = current(t_device, 0, 0);
    tensor x, pos, o;
    if (PyErr_Occurred() || !handle || !read_rows(a[2], dev, 0, &x) || x.shape[2] != head_dim ||
        !read_whole(a[3], 1, dev, t_i32, &pos) || pos.shape[0] != x.shape[0] || !fits(x.shape[0]) || !fits(x.shape[1]) ||
        (inverse != 0 && inverse != 1))
        return other_way();
    PyObject *out = a[4] == Py_None ? empty(a[2], NULL, t_bf16) : Py_NewRef(a[4]);
    if (!out || !read_rows(out, dev, 0, &o) || o.shape[0] != x.shape[0] || o.shape[1] != x.shape[1] || o.shape[2] != x.shape[2])
        return done(PD_ERR_INVALID, out);
    return done(pd_rope_apply((const pd_rope *)(intptr_t)handle, (const void *)(intptr_t)x.ptr, x.stride[0], x.stride[1],
                              (const int32_t *)(intptr_t)pos.ptr, (void *)(intptr_t)o.ptr, o.stride[0], o.stride[1],
                              (int)x.shape[0], (int)x.shape[1], (int)inverse, (void *)(intptr_t)current(t_stream, dev, 1)),
                out);
}

/* append_kv(handle | 0, head_dim, q, k, v, k_cache, v_cache, block_table, context_lens, token_starts | None,
 *           q_out | None, k_scale, v_scale) -- with queries */
static PyObject *append_kv(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 13) return other_way();
    const long long handle = PyLong_AsLongLong(a[0]), head_dim = PyLong_AsLongLong(a[1]), dev = current(t_device, 0, 0);
    const double ks = PyFloat_AsDouble(a[11]), vs = PyFloat_AsDouble(a[12]);
    tensor q, k, v, kc, vc, bt, cl, ts = {0}, o;
    if (PyErr_Occurred() || !read_rows(a[2], dev, 1, &q) || !read_rows(a[3], dev, 1, &k) || !read_rows(a[4], dev, 1, &v) ||
        !read_whole(a[7], 2, dev, t_i32, &bt) || !read_whole(a[8], 1, dev, t_i32, &cl))
        return other_way();
    if (!read_whole(a[5], 4, dev, t_bf16, &kc) && (PyErr_Occurred() || !read_whole(a[5], 4, dev, t_u8, &kc))) return other_way();
    if (!read_whole(a[6], 4, dev, kc.dtype, &vc)) return other_way();
    if (a[9] != Py_None && (!read_whole(a[9], 1, dev, t_i32, &ts) || ts.shape[0] != cl.shape[0] + 1)) return other_way();
    const long long T = k.shape[0], H = k.shape[1], D = k.shape[2];
    for (int i = 0; i < 4; ++i)
        if (vc.shape[i] != kc.shape[i] || !fits(kc.shape[i])) return other_way();
    if ((handle && D != head_dim) || v.shape[0] != T || v.shape[1] != H || v.shape[2] != D || q.shape[0] != T || q.shape[2] != D ||
        kc.shape[2] != H || kc.shape[3] != D || bt.shape[0] != cl.shape[0] || !fits(T) || !fits(q.shape[1]) ||
        !fits(bt.shape[0]) || !fits(bt.shape[1]))
        return other_way();
    PyObject *out = a[10] == Py_None ? empty(a[2], NULL, t_bf16) : Py_NewRef(a[10]);
    if (!out || !read_whole(out, 3, dev, t_bf16, &o) || o.shape[0] != T || o.shape[1] != q.shape[1] || o.shape[2] != D)
        return done(PD_ERR_INVALID, out);
    void *stream = (void *)(intptr_t)current(t_stream, dev, 1);
    const pd_rope *r = (const pd_rope *)(intptr_t)handle;
#define P(t) ((void *)(intptr_t)(t).ptr)
    const int rc =
        kc.dtype == t_u8
            ? pd_append_kv_fp8(r, P(q), q.stride[0], P(k), k.stride[0], P(v), v.stride[0], P(o), P(kc), P(vc), (float)ks,
                               (float)vs, P(bt), (int)bt.shape[1], P(cl), P(ts), (int)T, (int)cl.shape[0], (int)q.shape[1],
                               (int)H, (int)D, (int)kc.shape[1], (int)kc.shape[0], stream)
            : pd_append_kv(r, P(q), q.stride[0], P(k), k.stride[0], P(v), v.stride[0], P(o), P(kc), P(vc), P(bt),
                           (int)bt.shape[1], P(cl), P(ts), (int)T, (int)cl.shape[0], (int)q.shape[1], (int)H, (int)D,
                           (int)kc.shape[1], (int)kc.shape[0], stream);
    return done(rc, out);
}

/* decode_attn_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts | None, block_table, context_lens,
 *                    inv_sqrt_d, num_splits, out | None, ws | None, k_scale, v_scale) */
static PyObject *decode_attn_prefix(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 14) return other_way();
    const long long dev = current(t_device, 0, 0), splits = PyLong_AsLongLong(a[9]);
    const double scale = PyFloat_AsDouble(a[8]), ks = PyFloat_AsDouble(a[12]), vs = PyFloat_AsDouble(a[13]);
    tensor q, kc, vc, pt, pl, gs = {0}, bt, cl, o, w;
    if (PyErr_Occurred() || !read_whole(a[0], 3, dev, t_bf16, &q) || !read_whole(a[3], 2, dev, t_i32, &pt) ||
        !read_whole(a[4], 1, dev, t_i32, &pl) || !read_whole(a[6], 2, dev, t_i32, &bt) || !read_whole(a[7], 1, dev, t_i32, &cl))
        return other_way();
    if (!read_whole(a[1], 4, dev, t_bf16, &kc) && (PyErr_Occurred() || !read_whole(a[1], 4, dev, t_u8, &kc))) return other_way();
    if (!read_whole(a[2], 4, dev, kc.dtype, &vc)) return other_way();
    if (a[5] != Py_None && (!read_whole(a[5], 1, dev, t_i32, &gs) || gs.shape[0] != pl.shape[0] + 1)) return other_way();
    for (int i = 0; i < 4; ++i)
        if (vc.shape[i] != kc.shape[i] || !fits(kc.shape[i])) return other_way();
    const long long S = q.shape[0], Hq = q.shape[1], D = q.shape[2], H = kc.shape[2], G = pl.shape[0];
    if (kc.shape[3] != D || pt.shape[0] != G || bt.shape[0] != S || cl.shape[0] != S || !fits(S) || !fits(Hq) || !fits(G) ||
        !fits(pt.shape[1]) || !fits(bt.shape[1]) || !fits(splits))
        return other_way();
    PyObject *out = a[10] == Py_None ? empty(a[0], NULL, t_bf16) : Py_NewRef(a[10]);
    if (!out || !read_whole(out, 3, dev, t_bf16, &o) || o.shape[0] != S || o.shape[1] != Hq || o.shape[2] != D)
        return done(PD_ERR_INVALID, out);
    PyObject *ws;
    size_t bytes = pd_prefix_workspace_bytes((int)S, (int)G, (int)Hq, (int)H, (int)D, (int)splits);
    if (a[11] == Py_None) {
        PyObject *size = PyLong_FromSize_t(bytes);
        ws = size ? empty(a[0], size, t_u8) : NULL;
        Py_XDECREF(size);
    } else {
        ws = Py_NewRef(a[11]);
    }
    int rc = PD_ERR_INVALID;
    if (ws && read_whole(ws, 1, dev, t_u8, &w)) {
        void *stream = (void *)(intptr_t)current(t_stream, dev, 1);
        rc = kc.dtype == t_u8
                 ? pd_decode_attn_prefix_fp8(P(q), P(kc), P(vc), (float)ks, (float)vs, P(pt), (int)pt.shape[1], P(pl), P(gs),
                                             (int)G, P(bt), (int)bt.shape[1], P(cl), P(o), (int)S, (int)Hq, (int)H, (int)D,
                                             (int)kc.shape[1], (int)kc.shape[0], (float)scale, (int)splits, P(w),
                                             (size_t)w.shape[0], stream)
                 : pd_decode_attn_prefix(P(q), P(kc), P(vc), P(pt), (int)pt.shape[1], P(pl), P(gs), (int)G, P(bt),
                                         (int)bt.shape[1], P(cl), P(o), (int)S, (int)Hq, (int)H, (int)D, (int)kc.shape[1],
                                         (int)kc.shape[0], (float)scale, (int)splits, P(w), (size_t)w.shape[0], stream);
    }
    Py_XDECREF(ws); /* (the allocator keeps a block for its own stream's next use, after this launch) */
    return done(rc, out);
}

/* setup(bfloat16, uint8, int32, empty, current_device, current_stream) */
static PyObject *setup(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "setup takes six arguments");
        return NULL;
    }
    PyObject **to[6] = {&t_bf16, &t_u8, &t_i32, &t_empty, &t_device, &t_stream};
    for (int i = 0; i < 6; ++i) {
        Py_XDECREF(*to[i]);
        *to[i] = Py_NewRef(a[i]);
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, NULL},
                                {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, NULL},
                                {"append_kv", (PyCFunction)(void (*)(void))append_kv, METH_FASTCALL, NULL},
                                {"decode_attn_prefix", (PyCFunction)(void (*)(void))decode_attn_prefix, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "pd_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

__attribute__((visibility("default"))) PyMODINIT_FUNC PyInit_pd_binding(void) {
    n_shape = PyUnicode_InternFromString("shape");
    n_dtype = PyUnicode_InternFromString("dtype");
    n_device = PyUnicode_InternFromString("device");
    n_stride = PyUnicode_InternFromString("stride");
    n_data_ptr = PyUnicode_InternFromString("data_ptr");
    n_get_device = PyUnicode_InternFromString("get_device");
    n_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    kw_empty = Py_BuildValue("(ss)", "dtype", "device");
    if (!n_shape || !n_dtype || !n_device || !n_stride || !n_data_ptr || !n_get_device || !n_is_contiguous || !kw_empty) return NULL;
    return PyModule_Create(&module);
}
