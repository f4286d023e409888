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
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/saved_variable.h>

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

// A forward-mode tangent, which no call here carries on (api.py refuses it).
bool has_tangent(const at::Tensor &t) { return t._fw_grad(0).defined(); }

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

// A tensor of the caller's has been written: a gradient that has saved it learns so by its version.  (Tensors of the
// inference mode have none.)
void wrote(const at::Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void wrote(PyObject *given) {
    if (given != Py_None) wrote(THPVariable_Unpack(given));
}
// `given`, which has been written, or for None the tensor made here.
PyObject *answer(PyObject *given, const at::Tensor &made) {
    wrote(given);
    return given == Py_None ? THPVariable_Wrap(made) : Py_NewRef(given);
}

// rope(handle, head_dim, x, positions, out | None, inverse)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return quick(n, 6, [&] {
        const int dev = device();
        const auto handle = reinterpret_cast<const pd_rope *>(integer(a[0]));
        const Rows x = rows(a[2], dev, false);
        const at::Tensor &pos = whole(a[3], 1, at::kInt, dev);
        const long long inverse = integer(a[5]);
        need(!has_tangent(*x.t) && handle && x.D == integer(a[1]) && pos.size(0) == x.T && (inverse == 0 || inverse == 1));
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

// A norm's weight, or null for None.
const void *weight(PyObject *o, int64_t head_dim, int dev) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = whole(o, 1, at::kBFloat16, dev);
    need(t.size(0) == head_dim && !has_tangent(t));
    return t.data_ptr();
}

// norm_rope(handle | 0, head_dim, x, weight | None, positions | None, out | None, eps, weight_offset)
PyObject *norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return quick(n, 8, [&] {
        const int dev = device();
        const auto handle = reinterpret_cast<const pd_rope *>(integer(a[0]));
        const Rows x = rows(a[2], dev, false);
        const void *w = weight(a[3], x.D, dev);
        const float eps = real(a[6]), offset = real(a[7]);
        const int32_t *positions = nullptr;
        need(!has_tangent(*x.t) && (handle != nullptr) == (a[4] != Py_None));
        if (handle) {
            const at::Tensor &t = whole(a[4], 1, at::kInt, dev);
            need(x.D == integer(a[1]) && t.size(0) == x.T);
            positions = ints(t);
        }
        at::Tensor made;
        Rows o;
        if (a[5] == Py_None) {
            made = fresh(x.t->sizes(), at::kBFloat16, dev);
            o = {&made, x.T, x.H, x.D, x.H * x.D, x.D};
        } else {
            o = rows(a[5], dev, false);
            need(o.T == x.T && o.H == x.H && o.D == x.D);
        }
        need(pd_norm_rope_apply(handle, x.data(), x.token, x.head, w, eps, offset, positions, o.data(), o.token, o.head, fits(x.T),
                                fits(x.H), fits(x.D), stream(dev)) == PD_OK);
        return answer(a[5], made);
    });
}

// A tensor that was saved, as the caller's hooks on saved tensors gave it back: of the type, sizes and device that it had.
const at::Tensor &unpacked(const char *name, const at::Tensor &t, at::ScalarType dtype, at::IntArrayRef sizes, int dev) {
    TORCH_CHECK_VALUE(t.scalar_type() == dtype && t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev && t.sizes() == sizes,
                      "norm_rope's ", name, ": saved as ", dtype, " ", sizes, " on cuda:", dev, ", given back as ", t.scalar_type(), " ",
                      t.sizes(), " on ", t.device());
    return t;
}
// Rows [T, H, D], laid out anew where they come broadcast, transposed or at an odd place.
at::Tensor laid_out(const at::Tensor &t) {
    bool fits_rows = reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 && t.stride(2) == 1;
    for (int i = 0; i < 2; ++i) fits_rows = fits_rows && (t.size(i) <= 1 || (t.stride(i) > 0 && t.stride(i) % 8 == 0));
    return fits_rows ? t : t.clone(at::MemoryFormat::Contiguous);
}
// The same for what has to be contiguous.
at::Tensor in_order(const at::Tensor &t) {
    return t.is_contiguous() && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 ? t : t.clone(at::MemoryFormat::Contiguous);
}

// The interpreter's lock while it lives.
struct Gil {
    const PyGILState_STATE state = PyGILState_Ensure();
    ~Gil() { PyGILState_Release(state); }
};

// The backward pass of norm_rope, as api.py's _NormRotation has it: a node of its own, which the engine's threads run
// with no more of Python than a look at the rotation (a training step of 64 tokens: 224 us through api.py's, 111 through this).
struct NormRotation : torch::autograd::Node {
    torch::autograd::SavedVariable x, weight, positions;  // weight, positions: undefined where there are none
    PyObject *rotation = nullptr;  // the owner of the handle, or null
    float eps = 0, offset = 0;

    ~NormRotation() override {
        if (!rotation || !Py_IsInitialized()) return;  // (at the interpreter's end it may leak)
        const Gil gil;
        Py_DECREF(rotation);
    }
    // The rotation's handle (null where there is none), asked of its owner again, who may have closed it since the forward
    // pass.  The caller holds the interpreter's lock until its launch is done, so that nobody closes it meanwhile.
    const pd_rope *handle() const {
        if (!rotation) return nullptr;
        PyObject *number = PyObject_GetAttrString(rotation, "handle");
        void *h = number && number != Py_None ? PyLong_AsVoidPtr(number) : nullptr;
        Py_XDECREF(number);
        PyErr_Clear();
        TORCH_CHECK_VALUE(h, "the rotation's handle is closed");
        return static_cast<const pd_rope *>(h);
    }
    std::string name() const override { return "NormRotation"; }
    void release_variables() override {
        x.reset_data();
        weight.reset_data();
        positions.reset_data();
    }

    torch::autograd::variable_list apply(torch::autograd::variable_list &&grads) override {
        if (!grads[0].defined()) return {at::Tensor(), at::Tensor()};
        TORCH_CHECK(!has_tangent(grads[0]), "norm_rope's gradient has no forward-mode derivative");
        const bool again = at::GradMode::is_enabled();
        torch::autograd::variable_list out(2);
        {
            at::AutoGradMode off(false);
            const at::Tensor g = laid_out(grads[0]);
            const int dev = static_cast<int>(g.get_device());
            const int64_t T = g.size(0), H = g.size(1), D = g.size(2);
            const at::Tensor v = laid_out(unpacked("x", x.unpack(), at::kBFloat16, {T, H, D}, dev));
            at::Tensor w = weight.unpack(), pos = positions.unpack();
            if (w.defined()) w = in_order(unpacked("weight", w, at::kBFloat16, {D}, dev));
            if (pos.defined()) pos = in_order(unpacked("positions", pos, at::kInt, {T}, dev));
            auto token = [&](const at::Tensor &t) { return T > 1 ? t.stride(0) : H * D; };
            auto head = [&](const at::Tensor &t) { return H > 1 ? t.stride(1) : D; };
            out[0] = fresh({T, H, D}, at::kBFloat16, dev);
            at::Tensor room;
            if (w.defined() && task_should_compute_output(1)) {
                out[1] = fresh({D}, at::kBFloat16, dev);
                room = fresh({static_cast<int64_t>(pd_norm_rope_workspace_bytes(static_cast<int>(D)))}, at::kByte, dev);
            }
            const Gil gil;
            const int rc = pd_norm_rope_backward(handle(), v.data_ptr(), token(v), head(v), w.defined() ? w.data_ptr() : nullptr, eps, offset,
                                                 pos.defined() ? ints(pos) : nullptr, g.data_ptr(), token(g), head(g), out[0].data_ptr(),
                                                 H * D, D, out[1].defined() ? out[1].data_ptr() : nullptr, static_cast<int>(T),
                                                 static_cast<int>(H), static_cast<int>(D), room.defined() ? room.data_ptr() : nullptr,
                                                 room.defined() ? static_cast<size_t>(room.size(0)) : 0, ::stream(dev));
            TORCH_CHECK(rc == PD_OK, "libpd error ", rc, ": ", pd_last_error());
        }
        // (asked for a gradient that can be differentiated: an error where it is, which only what requires a gradient carries)
        for (at::Tensor &t : out) {
            if (!again || !t.defined()) continue;
            t.set_requires_grad(true);
            t = torch::autograd::DelayedError("norm_rope has no second gradient", 1)({t})[0];
        }
        return out;
    }
};

// norm_rope_grad(handle | 0, head_dim, rotation | None, x, weight | None, positions | None, eps, weight_offset) -- of an x or
// a weight that requires a gradient
PyObject *norm_rope_grad(PyObject *, PyObject *const *a, Py_ssize_t n) {
    const std::shared_ptr<NormRotation> node(new NormRotation, torch::autograd::deleteNode);
    at::Tensor x, weights, positions, made;
    PyObject *declined = quick(n, 8, [&]() -> PyObject * {
        const int dev = device();
        const auto handle = reinterpret_cast<const pd_rope *>(integer(a[0]));
        const Rows r = rows(a[3], dev, false);
        const void *w = weight(a[4], r.D, dev);
        need(!has_tangent(*r.t) && (handle != nullptr) == (a[5] != Py_None) && (handle != nullptr) == (a[2] != Py_None));
        x = *r.t;
        if (w) weights = THPVariable_Unpack(a[4]);
        if (handle) {
            positions = whole(a[5], 1, at::kInt, dev);
            need(r.D == integer(a[1]) && positions.size(0) == r.T);
        }
        node->eps = real(a[6]);
        node->offset = real(a[7]);
        made = fresh(x.sizes(), at::kBFloat16, dev);
        need(pd_norm_rope_apply(handle, r.data(), r.token, r.head, w, node->eps, node->offset, handle ? ints(positions) : nullptr,
                                made.data_ptr(), r.H * r.D, r.D, fits(r.T), fits(r.H), fits(r.D), stream(dev)) == PD_OK);
        return nullptr;
    });
    if (declined) return declined;
    // Saving a tensor runs the caller's hooks.  What they raise is not a refusal to be tried again but the caller's to see:
    // torch's checkpoints end a recomputation so.
    HANDLE_TH_ERRORS
    node->x = torch::autograd::SavedVariable(x, false);
    if (weights.defined()) node->weight = torch::autograd::SavedVariable(weights, false);
    if (positions.defined()) {
        node->positions = torch::autograd::SavedVariable(positions, false);
        node->rotation = Py_NewRef(a[2]);
    }
    node->set_next_edges(torch::autograd::collect_next_edges(x, weights));
    torch::autograd::set_history(made, node);
    return THPVariable_Wrap(made);
    END_HANDLE_TH_ERRORS
}

// What append_kv and append_kv_normed have in common: the tensors from q (a[0]) to v, the caches to q_out, and the scales.
struct Append {
    Rows q, k, v;
    const at::Tensor *kc, *vc, *table;
    const int32_t *lens, *starts = nullptr;
    at::Tensor made;
    const at::Tensor *out;
    float ks, vs;
    int T, S, Hq, H, D, bs, nb, mb;
    // rows: of q, k, v; caches: of k_cache, v_cache, block_table, context_lens, token_starts | None, q_out | None
    Append(PyObject *const *rows_of, PyObject *const *caches, PyObject *k_scale, PyObject *v_scale, int dev)
        : q(rows(rows_of[0], dev, true)), k(rows(rows_of[1], dev, true)), v(rows(rows_of[2], dev, true)), kc(&cache(caches[0], dev)),
          vc(&cache(caches[1], dev)), table(&whole(caches[2], 2, at::kInt, dev)), ks(real(k_scale)), vs(real(v_scale)) {
        const at::Tensor &l = whole(caches[3], 1, at::kInt, dev);
        need(v.T == k.T && v.H == k.H && v.D == k.D && q.T == k.T && q.D == k.D && kc->scalar_type() == vc->scalar_type() &&
             kc->sizes() == vc->sizes() && kc->size(2) == k.H && kc->size(3) == k.D && table->size(0) == l.size(0));
        lens = ints(l);
        if (caches[4] != Py_None) {
            const at::Tensor &t = whole(caches[4], 1, at::kInt, dev);
            need(t.size(0) == l.size(0) + 1);
            starts = ints(t);
        }
        if (caches[5] == Py_None) made = fresh(q.t->sizes(), at::kBFloat16, dev);
        out = caches[5] == Py_None ? &made : &whole(caches[5], 3, at::kBFloat16, dev);
        need(out->sizes() == q.t->sizes());
        T = fits(k.T), S = fits(l.size(0)), Hq = fits(q.H), H = fits(k.H), D = fits(k.D), bs = fits(kc->size(1)), nb = fits(kc->size(0)),
        mb = fits(table->size(1));
    }
    bool fp8() const { return kc->scalar_type() == at::kByte; }
    void wrote_caches() const {
        wrote(*kc);
        wrote(*vc);
    }
};

// append_kv(handle | 0, head_dim, q, k, v, k_cache, v_cache, block_table, context_lens, token_starts | None,
//           q_out | None, k_scale, v_scale) -- with queries
PyObject *append_kv(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return quick(n, 13, [&] {
        const int dev = device();
        const auto handle = reinterpret_cast<const pd_rope *>(integer(a[0]));
        const Append p(a + 2, a + 5, a[11], a[12], dev);
        need(!handle || p.D == integer(a[1]));
        const int rc = p.fp8() ? pd_append_kv_fp8(handle, p.q.data(), p.q.token, p.k.data(), p.k.token, p.v.data(), p.v.token,
                                                  p.out->data_ptr(), p.kc->data_ptr(), p.vc->data_ptr(), p.ks, p.vs, ints(*p.table), p.mb,
                                                  p.lens, p.starts, p.T, p.S, p.Hq, p.H, p.D, p.bs, p.nb, stream(dev))
                               : pd_append_kv(handle, p.q.data(), p.q.token, p.k.data(), p.k.token, p.v.data(), p.v.token,
                                              p.out->data_ptr(), p.kc->data_ptr(), p.vc->data_ptr(), ints(*p.table), p.mb, p.lens, p.starts,
                                              p.T, p.S, p.Hq, p.H, p.D, p.bs, p.nb, stream(dev));
        need(rc == PD_OK);
        p.wrote_caches();
        return answer(a[10], p.made);
    });
}

// append_kv_normed(handle | 0, head_dim, q, k, v, q_weight | None, k_weight | None, k_cache, v_cache, block_table,
//                  context_lens, token_starts | None, q_out | None, eps, weight_offset, k_scale, v_scale) -- with queries
PyObject *append_kv_normed(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return quick(n, 17, [&] {
        const int dev = device();
        const auto handle = reinterpret_cast<const pd_rope *>(integer(a[0]));
        const Append p(a + 2, a + 7, a[15], a[16], dev);
        need(!handle || p.D == integer(a[1]));
        const void *qw = weight(a[5], p.D, dev), *kw = weight(a[6], p.D, dev);
        const float eps = real(a[13]), offset = real(a[14]);
        const int rc =
            p.fp8() ? pd_append_kv_normed_fp8(handle, p.q.data(), p.q.token, p.k.data(), p.k.token, p.v.data(), p.v.token, qw, kw, eps,
                                              offset, p.out->data_ptr(), p.kc->data_ptr(), p.vc->data_ptr(), p.ks, p.vs, ints(*p.table), p.mb,
                                              p.lens, p.starts, p.T, p.S, p.Hq, p.H, p.D, p.bs, p.nb, stream(dev))
                    : pd_append_kv_normed(handle, p.q.data(), p.q.token, p.k.data(), p.k.token, p.v.data(), p.v.token, qw, kw, eps, offset,
                                          p.out->data_ptr(), p.kc->data_ptr(), p.vc->data_ptr(), ints(*p.table), p.mb, p.lens, p.starts, p.T,
                                          p.S, p.Hq, p.H, p.D, p.bs, p.nb, stream(dev));
        need(rc == PD_OK);
        p.wrote_caches();
        return answer(a[12], p.made);
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
        wrote(a[11]);
        return answer(a[10], made);
    });
}

// chunk_attn(q, k_cache, v_cache, block_table, context_lens, token_starts | None, inv_sqrt_d, window, out | None,
//            lse | None, ws | None, k_scale, v_scale)
PyObject *chunk_attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return quick(n, 13, [&] {
        const int dev = device();
        const Rows q = rows(a[0], dev, true);
        const at::Tensor &kc = cache(a[1], dev), &vc = cache(a[2], dev);
        const at::Tensor &table = whole(a[3], 2, at::kInt, dev), &lens = whole(a[4], 1, at::kInt, dev);
        const float scale = real(a[6]), ks = real(a[11]), vs = real(a[12]);
        const long long window = integer(a[7]);
        const int64_t S = lens.size(0);
        need(kc.scalar_type() == vc.scalar_type() && kc.sizes() == vc.sizes() && kc.size(3) == q.D && table.size(0) == S && window >= 0);
        const int32_t *starts = nullptr;
        if (a[5] != Py_None) {
            const at::Tensor &t = whole(a[5], 1, at::kInt, dev);
            need(t.size(0) == S + 1);
            starts = ints(t);
        }
        const int T = fits(q.T), Hq = fits(q.H), D = fits(q.D), nb = fits(kc.size(0)), bs = fits(kc.size(1)), H = fits(kc.size(2)),
                  mb = fits(table.size(1)), seqs = fits(S), win = fits(window);
        at::Tensor made, room;
        if (a[8] == Py_None) made = fresh(q.t->sizes(), at::kBFloat16, dev);
        const at::Tensor &out = a[8] == Py_None ? made : whole(a[8], 3, at::kBFloat16, dev);
        need(out.sizes() == q.t->sizes());
        float *lse = nullptr;
        if (a[9] != Py_None) {
            const at::Tensor &t = whole(a[9], 2, at::kFloat, dev);
            need(t.size(0) == q.T && t.size(1) == q.H);
            lse = static_cast<float *>(t.data_ptr());
        }
        if (a[10] == Py_None) room = fresh({static_cast<int64_t>(pd_chunk_workspace_bytes(T, Hq, H, D))}, at::kByte, dev);
        const at::Tensor &ws = a[10] == Py_None ? room : whole(a[10], 1, at::kByte, dev);
        const size_t bytes = static_cast<size_t>(ws.size(0));
        const int rc = kc.scalar_type() == at::kByte
                           ? pd_chunk_attn_fp8(q.data(), q.token, kc.data_ptr(), vc.data_ptr(), ks, vs, ints(table), mb, ints(lens), starts,
                                               out.data_ptr(), lse, T, seqs, Hq, H, D, bs, nb, scale, win, ws.data_ptr(), bytes, stream(dev))
                           : pd_chunk_attn(q.data(), q.token, kc.data_ptr(), vc.data_ptr(), ints(table), mb, ints(lens), starts,
                                           out.data_ptr(), lse, T, seqs, Hq, H, D, bs, nb, scale, win, ws.data_ptr(), bytes, stream(dev));
        need(rc == PD_OK);
        wrote(a[9]);
        wrote(a[10]);
        return answer(a[8], made);
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<rope>("rope"), method<append_kv>("append_kv"), method<norm_rope>("norm_rope"),
                         method<norm_rope_grad>("norm_rope_grad"),
                         method<append_kv_normed>("append_kv_normed"), method<decode_attn_prefix>("decode_attn_prefix"),
                         method<chunk_attn>("chunk_attn"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pd_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// (the torch whose tensors it reads: pd.quick() uses it with no other)
extern "C" __attribute__((visibility("default"))) PyObject *PyInit_pd_binding(void) {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", PD_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
