// pd_binding.cpp -- the quick way from torch tensors to libpd for the calls of a
// decode step, where the launch takes 3 us and reading, checking and passing on
// some forty properties in Python took 10 (through Python's C API by name: 5).
//
// Each function does what its namesake in api.py says for arguments that are
// exactly as it needs them (types, shapes, strides, the current device and
// stream) and returns NotImplemented for anything else, a failing library call
// or an exception among it; api.py then takes its own path, which checks
// argument by argument and raises what is wrong.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pd.h"

namespace {

// Thrown nowhere but here: an argument is not as the quick way needs it.
struct Decline {};
void need(bool ok) {
    if (!ok) throw Decline();
}

// A tensor of `dim` dimensions and the dtype on device `dev`.
const at::Tensor &tensor(PyObject *o, int dim, at::ScalarType dtype, int dev) {
    need(THPVariable_CheckExact(o));
    const at::Tensor &t = THPVariable_Unpack(o);
    need(t.defined() && t.dim() == dim && t.scalar_type() == dtype && t.layout() == at::kStrided && t.is_cuda() &&
         t.get_device() == dev);
    return t;
}
// The same, contiguous.
const at::Tensor &whole(PyObject *o, int dim, at::ScalarType dtype, int dev) {
    const at::Tensor &t = tensor(o, dim, dtype, dev);
    need(t.is_contiguous());
    return t;
}
const at::Tensor &cache(PyObject *o, int dev) {
    need(THPVariable_CheckExact(o));
    const at::ScalarType kind = THPVariable_Unpack(o).scalar_type();
    need(kind == at::kBFloat16 || kind == at::kByte);
    return whole(o, 4, kind, dev);
}

// BF16 rows [T, H, D], columns contiguous; side: a token's heads side by side.
struct Rows {
    const at::Tensor *t;
    int64_t T, H, D, token, head;  // sizes and the strides of a token and a head
    void *data() const { return t->data_ptr(); }
};
Rows rows(PyObject *o, int dev, bool side) {
    const at::Tensor &t = tensor(o, 3, at::kBFloat16, dev);
    Rows r = {&t, t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1)};
    need(t.stride(2) == 1);
    if (r.H <= 1) r.head = r.D;          // (one head, one token:
    if (r.T <= 1) r.token = r.H * r.D;   // any stride will do)
    need(!side || r.head == r.D);
    return r;
}

int fits(int64_t v) {
    need(v >= 0 && v <= 0x7fffffff);
    return static_cast<int>(v);
}
const int32_t *ints(const at::Tensor &t) { return static_cast<const int32_t *>(t.data_ptr()); }
float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    need(!PyErr_Occurred());
    return static_cast<float>(v);
}
long long integer(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    need(!PyErr_Occurred());
    return v;
}
int device() { return c10::cuda::current_device(); }
void *stream(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType dtype, int dev) {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
}

template <class F>
PyObject *quick(Py_ssize_t n, Py_ssize_t want, F body) {
    try {
        need(n == want);
        return body();
    } catch (...) {  // api.py's own way finds out and says what is wrong
    }
    PyErr_Clear();
    Py_RETURN_NOTIMPLEMENTED;
}

// `given`, or for None the tensor made here.
PyObject *answer(PyObject *given, const at::Tensor &made) { return given == Py_None ? THPVariable_Wrap(made) : Py_NewRef(given); }

// rope(handle, head_dim, x, positions, out | None, inverse)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return quick(n, 6, [&] {
        const int dev = device();
        const auto handle = reinterpret_cast<const pd_rope *>(integer(a[0]));
        const Rows x = rows(a[2], dev, false);
        const at::Tensor &pos = whole(a[3], 1, at::kInt, dev);
        const long long inverse = integer(a[5]);
        need(handle && x.D == integer(a[1]) && pos.size(0) == x.T && (inverse == 0 || inverse == 1));
        at::Tensor made;
        Rows o;
        if (a[4] == Py_None) {
            made = fresh(x.t->sizes(), at::kBFloat16, dev);
            o = {&made, x.T, x.H, x.D, x.H * x.D, x.D};
        } else {
            o = rows(a[4], dev, false);
            need(o.T == x.T && o.H == x.H && o.D == x.D);
        }
        need(pd_rope_apply(handle, x.data(), x.token, x.head, ints(pos), o.data(), o.token, o.head, fits(x.T), fits(x.H),
                           static_cast<int>(inverse), stream(dev)) == PD_OK);
        return answer(a[4], made);
    });
}

// append_kv(handle | 0, head_dim, q, k, v, k_cache, v_cache, block_table, context_lens, token_starts | None,
//           q_out | None, k_scale, v_scale) -- with queries
PyObject *append_kv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return quick(n, 13, [&] {
        const int dev = device();
        const auto handle = reinterpret_cast<const pd_rope *>(integer(a[0]));
        const Rows q = rows(a[2], dev, true), k = rows(a[3], dev, true), v = rows(a[4], dev, true);
        const at::Tensor &kc = cache(a[5], dev), &vc = cache(a[6], dev);
        const at::Tensor &table = whole(a[7], 2, at::kInt, dev), &lens = whole(a[8], 1, at::kInt, dev);
        const float ks = real(a[11]), vs = real(a[12]);
        const int64_t S = lens.size(0);
        need((!handle || k.D == integer(a[1])) && v.T == k.T && v.H == k.H && v.D == k.D && q.T == k.T && q.D == k.D &&
             kc.scalar_type() == vc.scalar_type() && kc.sizes() == vc.sizes() && kc.size(2) == k.H && kc.size(3) == k.D &&
             table.size(0) == S);
        const int32_t *starts = nullptr;
        if (a[9] != Py_None) {
            const at::Tensor &t = whole(a[9], 1, at::kInt, dev);
            need(t.size(0) == S + 1);
            starts = ints(t);
        }
        at::Tensor made;
        if (a[10] == Py_None) made = fresh(q.t->sizes(), at::kBFloat16, dev);
        const at::Tensor &out = a[10] == Py_None ? made : whole(a[10], 3, at::kBFloat16, dev);
        need(out.sizes() == q.t->sizes());
        const int T = fits(k.T), Hq = fits(q.H), H = fits(k.H), D = fits(k.D), bs = fits(kc.size(1)), nb = fits(kc.size(0)),
                  mb = fits(table.size(1)), seqs = fits(S);
        const int rc = kc.scalar_type() == at::kByte
                           ? pd_append_kv_fp8(handle, q.data(), q.token, k.data(), k.token, v.data(), v.token, out.data_ptr(),
                                              kc.data_ptr(), vc.data_ptr(), ks, vs, ints(table), mb, ints(lens), starts, T, seqs, Hq,
                                              H, D, bs, nb, stream(dev))
                           : pd_append_kv(handle, q.data(), q.token, k.data(), k.token, v.data(), v.token, out.data_ptr(),
                                          kc.data_ptr(), vc.data_ptr(), ints(table), mb, ints(lens), starts, T, seqs, Hq, H, D, bs,
                                          nb, stream(dev));
        need(rc == PD_OK);
        return answer(a[10], made);
    });
}

// decode_attn_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts | None, block_table, context_lens,
//                    inv_sqrt_d, num_splits, out | None, ws | None, k_scale, v_scale)
PyObject *decode_attn_prefix(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return quick(n, 14, [&] {
        const int dev = device();
        const at::Tensor &q = whole(a[0], 3, at::kBFloat16, dev);
        const at::Tensor &kc = cache(a[1], dev), &vc = cache(a[2], dev);
        const at::Tensor &ptable = whole(a[3], 2, at::kInt, dev), &plens = whole(a[4], 1, at::kInt, dev);
        const at::Tensor &table = whole(a[6], 2, at::kInt, dev), &lens = whole(a[7], 1, at::kInt, dev);
        const float scale = real(a[8]), ks = real(a[12]), vs = real(a[13]);
        const long long splits = integer(a[9]);
        const int S = fits(q.size(0)), Hq = fits(q.size(1)), D = fits(q.size(2)), nb = fits(kc.size(0)), bs = fits(kc.size(1)),
                  H = fits(kc.size(2)), pmb = fits(ptable.size(1)), mb = fits(table.size(1));
        const int64_t G = plens.size(0);
        need(kc.scalar_type() == vc.scalar_type() && kc.sizes() == vc.sizes() && kc.size(3) == D && ptable.size(0) == G &&
             G <= PD_MAX_PREFIX_GROUPS && table.size(0) == S && lens.size(0) == S && splits >= 1 && splits <= PD_MAX_DECODE_SPLITS);
        const int32_t *starts = nullptr;
        if (a[5] != Py_None) {
            const at::Tensor &t = whole(a[5], 1, at::kInt, dev);
            need(t.size(0) == G + 1);
            starts = ints(t);
        }
        at::Tensor made, room;
        if (a[10] == Py_None) made = fresh(q.sizes(), at::kBFloat16, dev);
        const at::Tensor &out = a[10] == Py_None ? made : whole(a[10], 3, at::kBFloat16, dev);
        need(out.sizes() == q.sizes());
        // (a workspace freed at the end: the allocator keeps it for this stream's next use, behind this launch)
        if (a[11] == Py_None)
            room = fresh({static_cast<int64_t>(pd_prefix_workspace_bytes(S, static_cast<int>(G), Hq, H, D, static_cast<int>(splits)))},
                         at::kByte, dev);
        const at::Tensor &ws = a[11] == Py_None ? room : whole(a[11], 1, at::kByte, dev);
        const int g = static_cast<int>(G), sp = static_cast<int>(splits);
        const size_t bytes = static_cast<size_t>(ws.size(0));
        const int rc = kc.scalar_type() == at::kByte
                           ? pd_decode_attn_prefix_fp8(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ks, vs, ints(ptable), pmb,
                                                       ints(plens), starts, g, ints(table), mb, ints(lens), out.data_ptr(), S, Hq, H,
                                                       D, bs, nb, scale, sp, ws.data_ptr(), bytes, stream(dev))
                           : pd_decode_attn_prefix(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), ints(ptable), pmb, ints(plens), starts,
                                                   g, ints(table), mb, ints(lens), out.data_ptr(), S, Hq, H, D, bs, nb, scale, sp,
                                                   ws.data_ptr(), bytes, stream(dev));
        need(rc == PD_OK);
        return answer(a[10], made);
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<rope>("rope"), method<append_kv>("append_kv"), method<decode_attn_prefix>("decode_attn_prefix"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pd_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// (the torch whose tensors it reads: pd.quick() uses it with no other)
extern "C" __attribute__((visibility("default"))) PyObject *PyInit_pd_binding(void) {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", PD_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
