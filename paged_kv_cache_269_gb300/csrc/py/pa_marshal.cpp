// pa_marshal.cpp -- the calls of rope_and_cache, decode_grouped, prefill_grouped
// and their forms over an 8-bit cache from Python without the interpreter in
// between.
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

// The caches: [N, H, B, D] twice, of one 16-bit type, or with `like` of e4m3 beside
// a tensor of a 16-bit type.
bool caches(Args &g, int i, pa_dims *d, at::ScalarType *type, const Tensor *like = nullptr) {
    const Tensor *k = g.tensor(i);
    if (!k) return false;
    *type = like ? like->scalar_type() : k->scalar_type();
    if (*type != at::kHalf && *type != at::kBFloat16) return false;
    const at::ScalarType stored = like ? at::kFloat8_e4m3fn : *type;
    k = g.plain(i, stored, 4);
    const Tensor *v = g.ok ? g.plain(i + 1, stored, 4) : nullptr;
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

// The scales of an 8-bit cache: fp32 [H] twice; null pointers where g.ok is false.
struct Scales {
    const float *k = nullptr, *v = nullptr;
};
Scales scales(Args &g, int i, int64_t H) {
    Scales s;
    const Tensor *k = g.plain(i, at::kFloat, 1);
    const Tensor *v = g.ok ? g.plain(i + 1, at::kFloat, 1) : nullptr;
    if (!v || k->size(0) != H || v->size(0) != H) {
        g.ok = false;
        return s;
    }
    s.k = static_cast<const float *>(k->data_ptr());
    s.v = static_cast<const float *>(v->data_ptr());
    return s;
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

// What both appends share: q_out, q, k, v, k_cache, v_cache, positions, cos_sin,
// slot_mapping, interleaved, device, stream.
struct Append {
    pa_dims d;
    int64_t qs, os, ks, vs;
    int32_t T, Hq, rotary, most;
    int turn;
    // taken before the interpreter is let go: asking for one may throw
    void *out, *k_cache, *v_cache, *stream;
    const void *q, *k, *v;
    const int32_t *positions, *slots;
    const float *table;
};
// q8: the caches are e4m3.  optional: q with q_out may be None (k and v alone), and so
// may cos_sin (no rotation), with positions or without.
bool append(Args &g, bool q8, bool optional, Append *x) {
    at::ScalarType type;
    const bool has_q = !optional || g.a[0] != Py_None || g.a[1] != Py_None;
    const bool turns = !optional || g.a[7] != Py_None, placed = turns || g.a[6] != Py_None;
    const Tensor *k = g.tensor(2);
    if (!k || k->dim() != 3 || !caches(g, 4, &x->d, &type, q8 ? k : nullptr)) return false;
    const int64_t T = k->size(0), H = x->d.num_heads, D = x->d.head_dim;
    k = rows(g, 2, type, T, H, D, &x->ks);
    const Tensor *v = g.ok ? rows(g, 3, type, T, H, D, &x->vs) : nullptr;
    const Tensor *slots = g.ok ? g.plain(8, at::kInt, 1) : nullptr;
    if (!g.ok || T <= 0 || T > 0x7fffffff || slots->size(0) != T) return false;
    x->Hq = 0;
    x->qs = x->os = 0;
    x->out = nullptr;
    x->q = nullptr;
    if (has_q) {
        const Tensor *q = g.tensor(1);
        if (!q || q->dim() != 3) return false;
        const int64_t Hq = q->size(1);
        q = rows(g, 1, type, T, Hq, D, &x->qs);
        const Tensor *o = g.ok ? rows(g, 0, type, T, Hq, D, &x->os) : nullptr;
        if (!o || Hq <= 0 || Hq > 0x7fffffff || (T > 1 && x->os < Hq * D)) return false;
        const bool in_place = o->data_ptr() == q->data_ptr() && (x->os == x->qs || T == 1);
        if ((!in_place && overlap(o, x->os, Hq * D, q, x->qs, Hq * D, T)) ||
            overlap(o, x->os, Hq * D, k, x->ks, H * D, T) || overlap(o, x->os, Hq * D, v, x->vs, H * D, T))
            return false;
        x->Hq = static_cast<int32_t>(Hq);
        x->out = o->data_ptr();
        x->q = q->data_ptr();
    }
    x->rotary = x->most = 0;
    x->table = nullptr;
    if (turns) {
        const Tensor *cs = g.plain(7, at::kFloat, 2);
        if (!cs || cs->size(0) > 0x7fffffff || cs->size(1) > 0x7fffffff || cs->size(1) <= 0) return false;
        x->rotary = static_cast<int32_t>(cs->size(1));
        x->most = static_cast<int32_t>(cs->size(0));
        x->table = static_cast<const float *>(cs->data_ptr());
    }
    x->positions = nullptr;
    if (placed) {
        const Tensor *pos = g.plain(6, at::kInt, 1);
        if (!pos || pos->size(0) != T) return false;
        x->positions = static_cast<const int32_t *>(pos->data_ptr());
    }
    x->turn = PyObject_IsTrue(g.a[9]);
    x->stream = pointer(g.a[11]);
    if (PyErr_Occurred() || x->turn < 0) return false;
    x->T = static_cast<int32_t>(T);
    x->k_cache = g.pointer(4);
    x->v_cache = g.pointer(5);
    x->k = k->data_ptr();
    x->v = v->data_ptr();
    x->slots = static_cast<const int32_t *>(slots->data_ptr());
    return true;
}

// rope(<append's 12>, fn) -> status or None
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 13) return take_over();
    Args g{a, static_cast<int>(integer(a[10]))};
    Append x;
    if (!append(g, false, false, &x)) return take_over();
    auto fn = reinterpret_cast<decltype(&pa_rope_and_cache)>(pointer(a[12]));
    if (PyErr_Occurred() || !fn) return take_over();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = fn(x.out, x.q, x.k, x.v, x.k_cache, x.v_cache, x.positions, x.table, x.slots, x.T, x.Hq, x.qs, x.ks, x.vs, x.os,
            x.rotary, x.most, x.turn, &x.d, x.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// norm_rope(<append's 12>, q_weight, k_weight, eps, k_scales, v_scales, fn) -> status or None
PyObject *norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 18) return take_over();
    Args g{a, static_cast<int>(integer(a[10]))};
    const bool q8 = a[15] != Py_None || a[16] != Py_None;
    Append x;
    if (!append(g, q8, true, &x)) return take_over();
    pa_append_opts o{};
    const float **weights[2] = {&o.q_weight, &o.k_weight};
    for (int i = 0; i < 2; ++i) {
        if (a[12 + i] == Py_None) continue;
        const Tensor *t = g.plain(12 + i, at::kFloat, 1);
        if (!t || t->size(0) != x.d.head_dim) return take_over();
        *weights[i] = static_cast<const float *>(t->data_ptr());
    }
    o.eps = static_cast<float>(PyFloat_AsDouble(a[14]));
    if (q8) {
        const Scales s = scales(g, 15, x.d.num_heads);
        o.k_scales = s.k;
        o.v_scales = s.v;
    }
    auto fn = reinterpret_cast<decltype(&pa_norm_rope_and_cache)>(pointer(a[17]));
    if (!g.ok || PyErr_Occurred() || !fn) return take_over();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = fn(x.out, x.q, x.k, x.v, x.k_cache, x.v_cache, x.positions, x.table, x.slots, x.T, x.Hq, x.qs, x.ks, x.vs, x.os,
            x.rotary, x.most, x.turn, &x.d, &o, x.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// gather_q8(k_out, v_out, k_cache, v_cache, k_scales, v_scales, slots, device, stream, fn) -> status or None
PyObject *gather_q8(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 10) return take_over();
    Args g{a, static_cast<int>(integer(a[7]))};
    pa_dims d;
    at::ScalarType type;
    const Tensor *ko = g.tensor(0);
    if (!ko || !caches(g, 2, &d, &type, ko)) return take_over();
    ko = g.plain(0, type, 3);
    const Tensor *vo = g.ok ? g.plain(1, type, 3) : nullptr;
    const Tensor *slots = g.ok ? g.plain(6, at::kInt, 1) : nullptr;
    if (!slots) return take_over();
    const int64_t T = slots->size(0), bytes = T * d.num_heads * d.head_dim * 2;
    if (T <= 0 || T > 0x7fffffff || ko->sizes() != vo->sizes() || ko->size(0) != T || ko->size(1) != d.num_heads ||
        ko->size(2) != d.head_dim)
        return take_over();
    const Scales s = scales(g, 4, d.num_heads);
    void *const kp = ko->data_ptr(), *const vp = vo->data_ptr();
    const int64_t apart = reinterpret_cast<int64_t>(kp) - reinterpret_cast<int64_t>(vp);
    void *stream = pointer(a[8]);
    auto fn = reinterpret_cast<decltype(&pa_gather_cache_q8)>(pointer(a[9]));
    if (!g.ok || PyErr_Occurred() || !fn || (apart < bytes && -apart < bytes)) return take_over();
    const void *const kc = g.pointer(2), *const vc = g.pointer(3);
    const auto *at = static_cast<const int32_t *>(slots->data_ptr());
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = fn(kp, vp, kc, vc, s.k, s.v, at, static_cast<int32_t>(T), &d, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// What both attention calls share.
struct Attention {
    pa_dims d;
    at::ScalarType type;
    Scales scales;
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
// prefix, counters, workspace, device, stream, and over an 8-bit cache (q8)
// k_scales, v_scales
bool attention(Args &g, Attention *x, bool q8) {
    PyObject *const *a = g.a;
    const Tensor *like = q8 ? g.tensor(1) : nullptr;
    if ((q8 && !like) || !caches(g, 2, &x->d, &x->type, like)) return false;
    if (q8) {
        x->scales = scales(g, 15, x->d.num_heads);
        if (!g.ok) return false;
    }
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

// decode(<attention's 15, or 17>, fn, workspace_fn, counters_fn) -> status or None
template <bool kQ8>
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr int at = kQ8 ? 17 : 15;
    if (n != at + 3) return take_over();
    Args g{a, static_cast<int>(integer(a[13]))};
    Attention x;
    if (!attention(g, &x, kQ8) || x.q->size(0) != x.S) return take_over();
    void *const fn = pointer(a[at]);
    auto ws = reinterpret_cast<decltype(&pa_decode_grouped_workspace_bytes)>(pointer(a[at + 1]));
    auto ct = reinterpret_cast<decltype(&pa_decode_grouped_counters_bytes)>(pointer(a[at + 2]));
    const int32_t Hq = static_cast<int32_t>(x.Hq), MB = static_cast<int32_t>(x.MB);
    const size_t need_ct = ct(&x.d, Hq), have_ct = x.counters->numel() * 4, have_ws = x.workspace->numel();
    if (need_ct == 0 || have_ct < need_ct || have_ws < ws(&x.d, Hq)) return take_over();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    if constexpr (kQ8)
        rc = reinterpret_cast<decltype(&pa_decode_grouped_q8)>(fn)(
            x.out_p, x.q_p, x.k_p, x.v_p, x.scales.k, x.scales.v, x.tables_p, x.lens_p, x.scale, MB, &x.d, Hq, &x.opts,
            x.workspace_p, have_ws, x.counters_p, have_ct, x.stream);
    else
        rc = reinterpret_cast<decltype(&pa_decode_grouped)>(fn)(
            x.out_p, x.q_p, x.k_p, x.v_p, x.tables_p, x.lens_p, x.scale, MB, &x.d, Hq, &x.opts, x.workspace_p, have_ws,
            x.counters_p, have_ct, x.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// prefill(<attention's 15, or 17>, query_start, max_query_len, fn, workspace_fn,
//         counters_fn) -> status or None
template <bool kQ8>
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    constexpr int at = kQ8 ? 17 : 15;
    if (n != at + 5) return take_over();
    Args g{a, static_cast<int>(integer(a[13]))};
    Attention x;
    if (!attention(g, &x, kQ8)) return take_over();
    const Tensor *starts = g.plain(at, at::kInt, 1);
    const long most = PyLong_AsLong(a[at + 1]);
    const int64_t total = x.q->size(0);
    if (!starts || PyErr_Occurred() || most <= 0 || most > 0x7fffffff || starts->size(0) != x.S + 1 || total <= 0 ||
        total > 0x7fffffff)
        return take_over();
    void *const fn = pointer(a[at + 2]);
    auto ws = reinterpret_cast<decltype(&pa_prefill_grouped_workspace_bytes)>(pointer(a[at + 3]));
    auto ct = reinterpret_cast<decltype(&pa_prefill_grouped_counters_bytes)>(pointer(a[at + 4]));
    const int32_t Hq = static_cast<int32_t>(x.Hq), MB = static_cast<int32_t>(x.MB);
    const int32_t rows = static_cast<int32_t>(total), longest = static_cast<int32_t>(most);
    const size_t need_ct = ct(&x.d, Hq), have_ct = x.counters->numel() * 4, have_ws = x.workspace->numel();
    if (need_ct == 0 || have_ct < need_ct || have_ws < ws(&x.d, Hq, longest)) return take_over();
    const auto *starts_p = static_cast<const int32_t *>(starts->data_ptr());
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    if constexpr (kQ8)
        rc = reinterpret_cast<decltype(&pa_prefill_grouped_q8)>(fn)(
            x.out_p, x.q_p, x.k_p, x.v_p, x.scales.k, x.scales.v, x.tables_p, x.lens_p, starts_p, rows, longest, x.scale,
            MB, &x.d, Hq, &x.opts, x.workspace_p, have_ws, x.counters_p, have_ct, x.stream);
    else
        rc = reinterpret_cast<decltype(&pa_prefill_grouped)>(fn)(
            x.out_p, x.q_p, x.k_p, x.v_p, x.tables_p, x.lens_p, starts_p, rows, longest, x.scale, MB, &x.d, Hq, &x.opts,
            x.workspace_p, have_ws, x.counters_p, have_ct, x.stream);
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

PyMethodDef methods[] = {method<rope>("rope"),
                         method<decode<false>>("decode"),
                         method<prefill<false>>("prefill"),
                         method<norm_rope>("norm_rope"),
                         method<gather_q8>("gather_q8"),
                         method<decode<true>>("decode_q8"),
                         method<prefill<true>>("prefill_q8"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pa_marshal", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_pa_marshal() { return PyModule_Create(&module); }
