// pa_marshal.cpp -- the calls of rope_and_cache, decode_grouped and
// prefill_grouped from Python without the interpreter in between.
//
// A decode step's append and attention take a few microseconds on the GPU;
// checking nine tensors in Python takes eight on the host.  These functions
// make the same checks on the tensors themselves (1 us) and call libpa.  They
// decide nothing: whatever is not the plain case -- a wrong type, shape, stride
// or device, buffers that are too small, an empty call -- returns None, and the
// Python binding, which knows what to say or do about it, takes over.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "pa.h"

namespace {

using at::Tensor;

struct Args {
    PyObject *const *a;
    int device;
    bool ok = true;
    void *pointer(int i) const { return THPVariable_Unpack(a[i]).data_ptr(); }
    const Tensor *tensor(int i) {
        if (!THPVariable_Check(a[i])) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(a[i]);
    }
    // A contiguous tensor of the call's device.
    const Tensor *plain(int i, at::ScalarType type, int dim) {
        const Tensor *t = tensor(i);
        if (!t || !t->is_cuda() || t->get_device() != device || t->scalar_type() != type || t->dim() != dim ||
            !t->is_contiguous())
            ok = false;
        return ok ? t : nullptr;
    }
};

// The caches: [N, H, B, D] twice, of one 16-bit type.
bool caches(Args &g, int i, pa_dims *d, at::ScalarType *type) {
    const Tensor *k = g.tensor(i);
    if (!k) return false;
    *type = k->scalar_type();
    if (*type != at::kHalf && *type != at::kBFloat16) return false;
    k = g.plain(i, *type, 4);
    const Tensor *v = g.ok ? g.plain(i + 1, *type, 4) : nullptr;
    if (!v || k->sizes() != v->sizes()) return false;
    for (int j = 0; j < 4; ++j)
        if (k->size(j) <= 0 || k->size(j) > 0x7fffffff) return false;
    d->num_seqs = 0;
    d->num_blocks = static_cast<int32_t>(k->size(0));
    d->num_heads = static_cast<int32_t>(k->size(1));
    d->block_size = static_cast<int32_t>(k->size(2));
    d->head_dim = static_cast<int32_t>(k->size(3));
    d->dtype = *type == at::kBFloat16 ? PA_DTYPE_BF16 : PA_DTYPE_F16;
    return true;
}

// A [T, heads, D] tensor with adjacent heads; its elements between rows.
const Tensor *rows(Args &g, int i, at::ScalarType type, int64_t tokens, int64_t heads, int64_t dim,
                   int64_t *step) {
    const Tensor *t = g.tensor(i);
    if (!t || !t->is_cuda() || t->get_device() != g.device || t->scalar_type() != type || t->dim() != 3 ||
        t->size(0) != tokens || t->size(1) != heads || t->size(2) != dim || t->stride(2) != 1 ||
        (heads > 1 && t->stride(1) != dim)) {
        g.ok = false;
        return nullptr;
    }
    *step = tokens > 1 ? t->stride(0) : heads * dim;
    if (*step < 0 || *step % 8) g.ok = false;
    return g.ok ? t : nullptr;
}

// Whether two sets of T rows share elements (pointers; steps and rows in
// elements of 2 bytes).
bool overlap(const Tensor *a, int64_t a_step, int64_t a_row, const Tensor *b, int64_t b_step, int64_t b_row,
             int64_t T) {
    const int64_t a0 = reinterpret_cast<int64_t>(a->data_ptr()), b0 = reinterpret_cast<int64_t>(b->data_ptr());
    if (a0 + 2 * ((T - 1) * a_step + a_row) <= b0 || b0 + 2 * ((T - 1) * b_step + b_row) <= a0) return false;
    if (a_step == b_step && T > 1 && a_step > 0) {
        int64_t off = (b0 - a0) % (2 * a_step);
        if (off < 0) off += 2 * a_step;
        if (off >= 2 * a_row && off + 2 * b_row <= 2 * a_step) return false;
    }
    return true;
}

void *pointer(PyObject *o) { return PyLong_AsVoidPtr(o); }

// number or None -> double
double number(PyObject *o) { return o == Py_None ? 0.0 : PyFloat_AsDouble(o); }
long integer(PyObject *o) { return o == Py_None ? 0 : PyLong_AsLong(o); }

PyObject *take_over() {
    PyErr_Clear();
    Py_RETURN_NONE;
}

// rope(q_out, q, k, v, k_cache, v_cache, positions, cos_sin, slot_mapping,
//      interleaved, device, stream, fn) -> status or None
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13) return take_over();
    Args g{a, static_cast<int>(integer(a[10]))};
    pa_dims d;
    at::ScalarType type;
    if (!caches(g, 4, &d, &type)) return take_over();
    const Tensor *q = g.tensor(1);
    if (!q || q->dim() != 3) return take_over();
    const int64_t T = q->size(0), Hq = q->size(1), H = d.num_heads, D = d.head_dim;
    int64_t qs, os, ks, vs;
    q = rows(g, 1, type, T, Hq, D, &qs);
    const Tensor *o = g.ok ? rows(g, 0, type, T, Hq, D, &os) : nullptr;
    const Tensor *k = g.ok ? rows(g, 2, type, T, H, D, &ks) : nullptr;
    const Tensor *v = g.ok ? rows(g, 3, type, T, H, D, &vs) : nullptr;
    const Tensor *pos = g.ok ? g.plain(6, at::kInt, 1) : nullptr;
    const Tensor *cs = g.ok ? g.plain(7, at::kFloat, 2) : nullptr;
    const Tensor *slots = g.ok ? g.plain(8, at::kInt, 1) : nullptr;
    if (!g.ok || T <= 0 || T > 0x7fffffff || Hq <= 0 || Hq > 0x7fffffff || pos->size(0) != T ||
        slots->size(0) != T || cs->size(0) > 0x7fffffff || cs->size(1) > 0x7fffffff ||
        (T > 1 && os < Hq * D))
        return take_over();
    const bool in_place = o->data_ptr() == q->data_ptr() && (os == qs || T == 1);
    if ((!in_place && overlap(o, os, Hq * D, q, qs, Hq * D, T)) || overlap(o, os, Hq * D, k, ks, H * D, T) ||
        overlap(o, os, Hq * D, v, vs, H * D, T))
        return take_over();
    const int turn = PyObject_IsTrue(a[9]);
    void *stream = pointer(a[11]);
    auto fn = reinterpret_cast<decltype(&pa_rope_and_cache)>(pointer(a[12]));
    if (PyErr_Occurred() || turn < 0 || !fn) return take_over();
    // every pointer before the interpreter is let go: asking for one may throw
    void *const kp = g.pointer(4), *const vp = g.pointer(5);
    void *const op = o->data_ptr();
    const void *const qp = q->data_ptr(), *const k_new = k->data_ptr(), *const v_new = v->data_ptr();
    const auto *positions = static_cast<const int32_t *>(pos->data_ptr());
    const auto *table = static_cast<const float *>(cs->data_ptr());
    const auto *slot = static_cast<const int32_t *>(slots->data_ptr());
    const int32_t rotary = static_cast<int32_t>(cs->size(1)), most = static_cast<int32_t>(cs->size(0));
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = fn(op, qp, k_new, v_new, kp, vp, positions, table, slot, static_cast<int32_t>(T), static_cast<int32_t>(Hq), qs,
            ks, vs, os, rotary, most, turn, &d, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// What both attention calls share.
struct Attention {
    pa_dims d;
    at::ScalarType type;
    pa_attn_opts opts;
    const Tensor *out, *q, *tables, *lens, *counters, *workspace;
    int64_t S, Hq, MB;
    float scale;
    void *stream;
    // their pointers: taken before the interpreter is let go, for asking may throw
    void *out_p, *k_p, *v_p, *workspace_p;
    const void *q_p;
    const int32_t *tables_p, *lens_p;
    uint32_t *counters_p;
};
// args: out, q, k_cache, v_cache, tables, lens, scale, softcap, slopes, window,
// prefix, counters, workspace, device, stream
bool attention(Args &g, Attention *x) {
    PyObject *const *a = g.a;
    if (!caches(g, 2, &x->d, &x->type)) return false;
    x->q = g.plain(1, x->type, 3);
    x->out = g.ok ? g.plain(0, x->type, 3) : nullptr;
    x->tables = g.ok ? g.plain(4, at::kInt, 2) : nullptr;
    x->lens = g.ok ? g.plain(5, at::kInt, 1) : nullptr;
    if (!g.ok) return false;
    x->S = x->tables->size(0);
    x->MB = x->tables->size(1);
    x->Hq = x->q->size(1);
    if (x->out->sizes() != x->q->sizes() || x->q->size(2) != x->d.head_dim || x->lens->size(0) != x->S ||
        x->S <= 0 || x->S > 0x7fffffff || x->MB <= 0 || x->MB > 0x7fffffff || x->Hq <= 0 ||
        x->Hq > 0x7fffffff || x->Hq % x->d.num_heads)
        return false;
    x->d.num_seqs = static_cast<int32_t>(x->S);
    x->scale = static_cast<float>(PyFloat_AsDouble(a[6]));
    const double cap = number(a[7]);
    x->opts.softcap = static_cast<float>(cap);
    if (x->opts.softcap == 0.f && cap != 0.0) return false;   // 0 would say "none"
    const long window = integer(a[9]);
    if (PyErr_Occurred() || window < 0 || window > 0x7fffffff) return false;
    x->opts.window = static_cast<int32_t>(window);
    x->opts.alibi_slopes = nullptr;
    x->opts.prefix_lens = nullptr;
    if (a[8] != Py_None) {
        const Tensor *t = g.plain(8, at::kFloat, 1);
        if (!t || t->size(0) != x->Hq) return false;
        x->opts.alibi_slopes = static_cast<const float *>(t->data_ptr());
    }
    if (a[10] != Py_None) {
        const Tensor *t = g.plain(10, at::kInt, 1);
        if (!t || t->size(0) != x->S) return false;
        x->opts.prefix_lens = static_cast<const int32_t *>(t->data_ptr());
    }
    x->counters = g.plain(11, at::kInt, 1);
    x->workspace = g.ok ? g.plain(12, at::kByte, 1) : nullptr;
    x->stream = pointer(a[14]);
    if (!g.ok || PyErr_Occurred()) return false;
    x->out_p = x->out->data_ptr();
    x->q_p = x->q->data_ptr();
    x->k_p = g.pointer(2);
    x->v_p = g.pointer(3);
    x->tables_p = static_cast<const int32_t *>(x->tables->data_ptr());
    x->lens_p = static_cast<const int32_t *>(x->lens->data_ptr());
    x->counters_p = static_cast<uint32_t *>(x->counters->data_ptr());
    x->workspace_p = x->workspace->data_ptr();
    return true;
}

// decode(<attention's 15>, fn, workspace_fn, counters_fn) -> status or None
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 18) return take_over();
    Args g{a, static_cast<int>(integer(a[13]))};
    Attention x;
    if (!attention(g, &x) || x.q->size(0) != x.S) return take_over();
    auto fn = reinterpret_cast<decltype(&pa_decode_grouped)>(pointer(a[15]));
    auto ws = reinterpret_cast<decltype(&pa_decode_grouped_workspace_bytes)>(pointer(a[16]));
    auto ct = reinterpret_cast<decltype(&pa_decode_grouped_counters_bytes)>(pointer(a[17]));
    const int32_t Hq = static_cast<int32_t>(x.Hq);
    const size_t need_ct = ct(&x.d, Hq), have_ct = x.counters->numel() * 4, have_ws = x.workspace->numel();
    if (need_ct == 0 || have_ct < need_ct || have_ws < ws(&x.d, Hq)) return take_over();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = fn(x.out_p, x.q_p, x.k_p, x.v_p, x.tables_p, x.lens_p, x.scale, static_cast<int32_t>(x.MB), &x.d, Hq, &x.opts,
            x.workspace_p, have_ws, x.counters_p, have_ct, x.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// prefill(<attention's 15>, query_start, max_query_len, fn, workspace_fn,
//         counters_fn) -> status or None
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 20) return take_over();
    Args g{a, static_cast<int>(integer(a[13]))};
    Attention x;
    if (!attention(g, &x)) return take_over();
    const Tensor *starts = g.plain(15, at::kInt, 1);
    const long most = PyLong_AsLong(a[16]);
    const int64_t total = x.q->size(0);
    if (!starts || PyErr_Occurred() || most <= 0 || most > 0x7fffffff || starts->size(0) != x.S + 1 || total <= 0 ||
        total > 0x7fffffff)
        return take_over();
    auto fn = reinterpret_cast<decltype(&pa_prefill_grouped)>(pointer(a[17]));
    auto ws = reinterpret_cast<decltype(&pa_prefill_grouped_workspace_bytes)>(pointer(a[18]));
    auto ct = reinterpret_cast<decltype(&pa_prefill_grouped_counters_bytes)>(pointer(a[19]));
    const int32_t Hq = static_cast<int32_t>(x.Hq);
    const size_t need_ct = ct(&x.d, Hq), have_ct = x.counters->numel() * 4, have_ws = x.workspace->numel();
    if (need_ct == 0 || have_ct < need_ct || have_ws < ws(&x.d, Hq, static_cast<int32_t>(most))) return take_over();
    const auto *starts_p = static_cast<const int32_t *>(starts->data_ptr());
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = fn(x.out_p, x.q_p, x.k_p, x.v_p, x.tables_p, x.lens_p, starts_p, static_cast<int32_t>(total),
            static_cast<int32_t>(most), x.scale, static_cast<int32_t>(x.MB), &x.d, Hq, &x.opts, x.workspace_p, have_ws,
            x.counters_p, have_ct, x.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// C++ exceptions (a tensor without storage, say) stay inside.
template <PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    try {
        return f(self, a, n);
    } catch (...) {
        return take_over();
    }
}

template <PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)>
constexpr PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&guarded<f>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rope>("rope"), method<decode>("decode"), method<prefill>("prefill"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pa_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_pa_marshal() { return PyModule_Create(&module); }
