// calls.cpp -- the Python side of the answering calls (include/spava.h): checks
// of tensors, outputs, the current stream, and the library call, compiled.  A
// decode step makes these calls many thousand times a second on tensors of a few
// KiB; interpreted (ctypes, one attribute at a time) the host's part of a call is
// 6 to 9 us beside a launch's 2.5, here it is about one.
//
// Argument marshalling only, like api.py: the computation is libspava's.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <structmember.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/spava.h"

namespace {

// ------------------------------------------------------------------ checks
struct Refused {  // becomes a ValueError
    std::string what;
};

std::string said(const at::Tensor &t) {
    return c10::str(t.scalar_type(), " ", t.sizes(), " on ", t.device(), " strides ", t.strides());
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw Refused{c10::str(name, ": expected a tensor, got ", Py_TYPE(o)->tp_name)};
    return THPVariable_Unpack(o);
}

bool on(const at::Tensor &t, int index) { return t.is_cuda() && t.get_device() == index; }

void check(const at::Tensor &t, at::IntArrayRef shape, at::ScalarType type, int index, const char *name) {
    if (t.scalar_type() != type || t.sizes() != shape || !on(t, index) || !t.is_contiguous())
        throw Refused{c10::str(name, ": expected contiguous ", type, " ", shape, " on cuda:", index, ", got ", said(t))};
}

// Elements between the tokens of a bf16 [rows, heads, d] tensor or view.
int64_t token_stride(const at::Tensor &t, int64_t rows, int64_t heads, int64_t d, int index, const char *name) {
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.size(0) != rows || t.size(1) != heads ||
        t.size(2) != d || !on(t, index))
        throw Refused{c10::str(name, ": expected BFloat16 [", rows, ", ", heads, ", ", d, "] on cuda:", index, ", got ",
                               said(t))};
    if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))
        throw Refused{c10::str(name, ": the heads of a token must be contiguous, got ", said(t))};
    return rows > 1 ? t.stride(0) : heads * d;
}

int64_t rows_of(const at::Tensor &t, const char *name) {
    if (t.dim() != 3) throw Refused{c10::str(name, ": expected [rows, heads, d], got ", said(t))};
    return t.size(0);
}

int64_t new_rows_of(int64_t rows, int64_t n_seqs, const char *name) {
    if (rows == 0 && n_seqs == 0) return 0;
    if (n_seqs == 0 || rows % n_seqs)
        throw Refused{c10::str(name, ": ", rows, " rows for ", n_seqs, " sequences: expected as many for each")};
    return rows / n_seqs;
}

// The given output, checked, or a new one.
at::Tensor output(PyObject *given, at::IntArrayRef shape, at::ScalarType type, int index, const char *name) {
    if (given != Py_None) {
        const at::Tensor &t = tensor(given, name);
        check(t, shape, type, index, name);
        return t;
    }
    // the caching allocator's memory without a trip through the dispatcher (0.25 us each)
    return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index)), std::nullopt);
}

// Raises for a tensor without memory of its own: a transform's or a fake one, one
// whose storage was given back.
void *ptr(const at::Tensor &t, const char *name) {
    void *p = t.data_ptr();
    if (!t.storage().device().is_cuda() || (t.storage().nbytes() == 0 && t.numel() != 0))
        throw Refused{c10::str(name, ": expected a tensor with memory, got ", said(t))};
    return p;
}

// ------------------------------------------------------------------ calls
PyObject *g_failed = nullptr;  // (function name, status): raises

class WithoutGil {  // until it is destroyed, also by an exception
    PyThreadState *state_ = PyEval_SaveThread();

  public:
    WithoutGil() = default;
    WithoutGil(const WithoutGil &) = delete;
    ~WithoutGil() { PyEval_RestoreThread(state_); }
};

// f(stream), the library call, without the GIL: it touches no Python object and no
// tensor, whose addresses are taken before (and may raise).
template <typename F>
bool called(const char *name, int index, F f) {
    spava_status rc;
    {
        c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
        void *stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
        WithoutGil released;
        rc = f(stream);
    }
    if (rc == SPAVA_OK) return true;
    if (!g_failed) {
        PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, int(rc));
    } else if (PyObject *r = PyObject_CallFunction(g_failed, "si", name, int(rc))) {
        Py_DECREF(r);
        PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, int(rc));
    }
    return false;
}

template <typename F>
PyObject *guarded(F f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refused &r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

bool arguments(Py_ssize_t n, Py_ssize_t want, const char *name) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%s: expected %zd arguments, got %zd", name, want, n);
    return false;
}

PyObject *pair(const at::Tensor &a, PyObject *b) {  // steals b
    PyObject *x = THPVariable_Wrap(a);
    if (!x || !b) {
        Py_XDECREF(x);
        Py_XDECREF(b);
        return nullptr;
    }
    PyObject *t = PyTuple_New(2);
    if (!t) {
        Py_DECREF(x);
        Py_DECREF(b);
        return nullptr;
    }
    PyTuple_SET_ITEM(t, 0, x);
    PyTuple_SET_ITEM(t, 1, b);
    return t;
}

// ------------------------------------------------------------------ kept tensors
// Both objects keep Python tensors, not addresses: a tensor's memory may be
// replaced (``weight.data = ...``, a module that moves), so every call checks it
// and takes its address anew.
// A constructor's tensor as a new reference; null for None or 0.
bool kept(PyObject *o, PyObject **to, const char *name) {
    if (o == Py_None || (PyLong_Check(o) && PyObject_IsTrue(o) == 0)) {
        Py_CLEAR(*to);
        return true;
    }
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_ValueError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
        return false;
    }
    Py_INCREF(o);
    Py_XSETREF(*to, o);
    return true;
}

void *kept_ptr(PyObject *o, at::IntArrayRef shape, at::ScalarType type, int index, const char *name) {
    if (!o) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    check(t, shape, type, index, name);
    return ptr(t, name);
}

// T: {PyObject_HEAD; PyObject *tensors[N]; ...}
template <typename T>
int visit_kept(PyObject *self, visitproc visit, void *arg) {
    for (PyObject *o : reinterpret_cast<T *>(self)->tensors) Py_VISIT(o);
    return 0;
}
template <typename T>
int clear_kept(PyObject *self) {
    for (PyObject *&o : reinterpret_cast<T *>(self)->tensors) Py_CLEAR(o);
    return 0;
}
template <typename T>
void dealloc(PyObject *self) {
    PyObject_GC_UnTrack(self);
    clear_kept<T>(self);
    Py_TYPE(self)->tp_free(self);
}
#define SPAVA_KEPT(type, name, i) \
    {name, T_OBJECT, offsetof(type, tensors) + (i) * sizeof(PyObject *), READONLY, nullptr}

// ------------------------------------------------------------------ Rope
struct Rope {
    PyObject_HEAD
    PyObject *tensors[3];  // q_weight, k_weight, inv_freq
    spava_rope_config cfg;
    int index;
};
PyMemberDef rope_members[] = {SPAVA_KEPT(Rope, "q_weight", 0), SPAVA_KEPT(Rope, "k_weight", 1),
                              SPAVA_KEPT(Rope, "inv_freq", 2), {nullptr, 0, 0, 0, nullptr}};

// (address of a spava_rope_config, q_weight, k_weight, inv_freq, device)
int rope_init(PyObject *self, PyObject *args, PyObject *) {
    Rope *r = reinterpret_cast<Rope *>(self);
    unsigned long long cfg;
    PyObject *q, *k, *f;
    if (!PyArg_ParseTuple(args, "KOOOi", &cfg, &q, &k, &f, &r->index)) return -1;
    if (!cfg) {
        PyErr_SetString(PyExc_ValueError, "Rope: no configuration");
        return -1;
    }
    r->cfg = *reinterpret_cast<const spava_rope_config *>(cfg);
    return kept(q, &r->tensors[0], "q_weight") && kept(k, &r->tensors[1], "k_weight") &&
                   kept(f, &r->tensors[2], "inv_freq") ? 0 : -1;
}

struct RopeTables {
    const void *q_weight, *k_weight;
    const float *inv_freq;
};
RopeTables tables_of(const Rope *r) {
    const int64_t d = r->cfg.head_dim, half = r->cfg.rope_dim / 2;
    return {kept_ptr(r->tensors[0], d, at::kBFloat16, r->index, "q_weight"),
            kept_ptr(r->tensors[1], d, at::kBFloat16, r->index, "k_weight"),
            half ? static_cast<const float *>(kept_ptr(r->tensors[2], half, at::kFloat, r->index, "inv_freq")) : nullptr};
}

const int32_t *positions_of(const Rope *r, PyObject *o, int64_t rows) {
    if (r->cfg.rope_dim == 0) return nullptr;
    if (o == Py_None) throw Refused{"positions: a rotation needs them"};
    const at::Tensor &t = tensor(o, "positions");
    const int64_t axes = r->cfg.n_axes;
    const bool shaped = t.dim() == 2 ? t.size(0) == axes && t.size(1) == rows : axes == 1 && t.dim() == 1 && t.size(0) == rows;
    if (t.scalar_type() != at::kInt || !shaped || !on(t, r->index) || !t.is_contiguous())
        throw Refused{c10::str("positions: expected contiguous Int [", axes, ", ", rows, "] on cuda:", r->index, ", got ",
                               said(t))};
    return static_cast<const int32_t *>(ptr(t, "positions"));
}

// apply(q, k, positions, q_out, k_out)
PyObject *rope_apply(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 5, "apply")) return nullptr;
    return guarded([&]() -> PyObject * {
        const Rope *r = reinterpret_cast<Rope *>(self);
        const spava_rope_config &c = r->cfg;
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
        const int64_t rows = rows_of(q, "q");
        const int64_t qs = token_stride(q, rows, c.n_q_heads, c.head_dim, r->index, "q");
        const int64_t ks = token_stride(k, rows, c.n_kv_heads, c.head_dim, r->index, "k");
        const int32_t *pos = positions_of(r, a[2], rows);
        const at::Tensor qo = output(a[3], q.sizes(), at::kBFloat16, r->index, "q_out");
        const at::Tensor ko = output(a[4], k.sizes(), at::kBFloat16, r->index, "k_out");
        const void *qp = ptr(q, "q"), *kp = ptr(k, "k");
        void *qop = ptr(qo, "q_out"), *kop = ptr(ko, "k_out");
        const RopeTables w = tables_of(r);
        if (!called("spava_qk_norm_rope", r->index, [&](void *stream) {
                return spava_qk_norm_rope(&c, rows, qp, qs, kp, ks, w.q_weight, w.k_weight, w.inv_freq, pos, qop, kop,
                                          stream);
            }))
            return nullptr;
        return pair(qo, THPVariable_Wrap(ko));
    });
}

PyMethodDef rope_methods[] = {
    {"apply", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(rope_apply)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyTypeObject RopeType = {PyVarObject_HEAD_INIT(nullptr, 0)};

// ------------------------------------------------------------------ Cache
struct Cache {
    PyObject_HEAD
    PyObject *tensors[5];  // k_pages, v_pages, k_exp, v_exp, workspace
    spava_cache_config cfg;
    int index;
};
PyMemberDef cache_members[] = {SPAVA_KEPT(Cache, "k_pages", 0), SPAVA_KEPT(Cache, "v_pages", 1),
                               SPAVA_KEPT(Cache, "k_exp", 2),   SPAVA_KEPT(Cache, "v_exp", 3),
                               SPAVA_KEPT(Cache, "workspace", 4), {nullptr, 0, 0, 0, nullptr}};

// (address of a spava_cache_config, (k_pages, v_pages), (k_exp, v_exp), workspace, device)
int cache_init(PyObject *self, PyObject *args, PyObject *) {
    Cache *c = reinterpret_cast<Cache *>(self);
    unsigned long long cfg;
    PyObject *pools, *exps, *ws;
    if (!PyArg_ParseTuple(args, "KOOOi", &cfg, &pools, &exps, &ws, &c->index)) return -1;
    if (!cfg || !PyTuple_Check(pools) || PyTuple_GET_SIZE(pools) != 2 || !PyTuple_Check(exps) ||
        PyTuple_GET_SIZE(exps) != 2) {
        PyErr_SetString(PyExc_ValueError, "Cache: no configuration or no pools");
        return -1;
    }
    c->cfg = *reinterpret_cast<const spava_cache_config *>(cfg);
    return kept(PyTuple_GET_ITEM(pools, 0), &c->tensors[0], "k_pages") &&
                   kept(PyTuple_GET_ITEM(pools, 1), &c->tensors[1], "v_pages") &&
                   kept(PyTuple_GET_ITEM(exps, 0), &c->tensors[2], "k_exp") &&
                   kept(PyTuple_GET_ITEM(exps, 1), &c->tensors[3], "v_exp") && kept(ws, &c->tensors[4], "workspace")
               ? 0
               : -1;
}

spava_cache_pools pools_of(const Cache *c) {
    const int64_t shape[4] = {c->cfg.n_pages, c->cfg.n_kv_heads, c->cfg.page_size, c->cfg.head_dim};
    const at::IntArrayRef rows(shape, 3);
    const bool e4m3 = c->cfg.type == SPAVA_CACHE_E4M3;
    const at::ScalarType type = e4m3 ? at::kFloat8_e4m3fn : at::kBFloat16;
    spava_cache_pools p{kept_ptr(c->tensors[0], shape, type, c->index, "k_pages"),
                        kept_ptr(c->tensors[1], shape, type, c->index, "v_pages"), nullptr, nullptr};
    if (e4m3) {
        p.k_exp = static_cast<int8_t *>(kept_ptr(c->tensors[2], rows, at::kChar, c->index, "k_exp"));
        p.v_exp = static_cast<int8_t *>(kept_ptr(c->tensors[3], rows, at::kChar, c->index, "v_exp"));
    }
    return p;
}

struct Space {
    void *ws;
    size_t bytes;
};
Space space_of(const Cache *c, PyObject *given) {
    if (given == Py_None) given = c->tensors[4];
    if (!given) return {nullptr, 0};
    const at::Tensor &t = tensor(given, "workspace");
    if (t.scalar_type() != at::kByte || !on(t, c->index) || !t.is_contiguous())
        throw Refused{c10::str("workspace: expected contiguous Byte on cuda:", c->index, ", got ", said(t))};
    return {ptr(t, "workspace"), static_cast<size_t>(t.numel())};
}

spava_cache_batch batch_of(const Cache *c, PyObject *table, PyObject *lens) {
    const at::Tensor &t = tensor(table, "table"), &l = tensor(lens, "lens");
    if (t.scalar_type() != at::kInt || l.scalar_type() != at::kInt || t.dim() != 2 || l.dim() != 1 ||
        t.size(0) != l.size(0) || !on(t, c->index) || !on(l, c->index) || !t.is_contiguous() || !l.is_contiguous())
        throw Refused{c10::str("table, lens: expected contiguous Int [sequences, max_pages] and [sequences] on cuda:",
                               c->index, ", got ", said(t), " and ", said(l))};
    return {t.size(0), t.size(1), static_cast<const int32_t *>(ptr(t, "table")), static_cast<const int32_t *>(ptr(l, "lens"))};
}

// write(k, v, table, lens, workspace)
PyObject *cache_write(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 5, "write")) return nullptr;
    return guarded([&]() -> PyObject * {
        const Cache *c = reinterpret_cast<Cache *>(self);
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        const spava_cache_batch batch = batch_of(c, a[2], a[3]);
        const int64_t rows = rows_of(k, "k"), fresh = new_rows_of(rows, batch.n_seqs, "k");
        const int64_t ks = token_stride(k, rows, c->cfg.n_kv_heads, c->cfg.head_dim, c->index, "k");
        const int64_t vs = token_stride(v, rows, c->cfg.n_kv_heads, c->cfg.head_dim, c->index, "v");
        const Space s = space_of(c, a[4]);
        const spava_cache_pools pools = pools_of(c);
        const void *kp = ptr(k, "k"), *vp = ptr(v, "v");
        if (!called("spava_cache_write", c->index, [&](void *stream) {
                return spava_cache_write(&c->cfg, &pools, &batch, fresh, kp, ks, vp, vs, s.ws, s.bytes, stream);
            }))
            return nullptr;
        Py_RETURN_NONE;
    });
}

// append(rope, q, k, v, positions, table, lens, q_out, workspace)
PyObject *cache_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 9, "append")) return nullptr;
    return guarded([&]() -> PyObject * {
        const Cache *c = reinterpret_cast<Cache *>(self);
        if (!PyObject_TypeCheck(a[0], &RopeType)) throw Refused{"rope: expected a QKNormRope"};
        const Rope *r = reinterpret_cast<Rope *>(a[0]);
        if (r->index != c->index)
            throw Refused{c10::str("rope: expected on cuda:", c->index, ", is on cuda:", r->index)};
        const at::Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
        const spava_cache_batch batch = batch_of(c, a[5], a[6]);
        const int64_t rows = rows_of(q, "q"), fresh = new_rows_of(rows, batch.n_seqs, "q");
        const int64_t qs = token_stride(q, rows, c->cfg.n_q_heads, c->cfg.head_dim, c->index, "q");
        const int64_t ks = token_stride(k, rows, c->cfg.n_kv_heads, c->cfg.head_dim, c->index, "k");
        const int64_t vs = token_stride(v, rows, c->cfg.n_kv_heads, c->cfg.head_dim, c->index, "v");
        const int32_t *pos = positions_of(r, a[4], rows);
        const Space s = space_of(c, a[8]);
        const spava_cache_pools pools = pools_of(c);
        const RopeTables w = tables_of(r);
        const at::Tensor qo = output(a[7], q.sizes(), at::kBFloat16, c->index, "q_out");
        const void *qp = ptr(q, "q"), *kp = ptr(k, "k"), *vp = ptr(v, "v");
        void *qop = ptr(qo, "q_out");
        if (!called("spava_cache_append", c->index, [&](void *stream) {
                return spava_cache_append(&r->cfg, &c->cfg, &pools, &batch, fresh, qp, qs, kp, ks, vp, vs, w.q_weight,
                                          w.k_weight, w.inv_freq, pos, qop, s.ws, s.bytes, stream);
            }))
            return nullptr;
        return THPVariable_Wrap(qo);
    });
}

// read(table, lens, rows, first, k_out, v_out, workspace)
PyObject *cache_read(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 7, "read")) return nullptr;
    return guarded([&]() -> PyObject * {
        const Cache *c = reinterpret_cast<Cache *>(self);
        const spava_cache_batch batch = batch_of(c, a[0], a[1]);
        const int64_t rows = PyLong_AsLongLong(a[2]), first = PyLong_AsLongLong(a[3]);
        if (PyErr_Occurred()) return nullptr;
        if (rows < 0 || first < 0) throw Refused{c10::str("rows, first: expected >= 0, got ", rows, " and ", first)};
        const int64_t shape[4] = {batch.n_seqs, rows, c->cfg.n_kv_heads, c->cfg.head_dim};
        const Space s = space_of(c, a[6]);
        const spava_cache_pools pools = pools_of(c);
        const at::Tensor ko = output(a[4], shape, at::kBFloat16, c->index, "k_out");
        const at::Tensor vo = output(a[5], shape, at::kBFloat16, c->index, "v_out");
        void *kop = ptr(ko, "k_out"), *vop = ptr(vo, "v_out");
        if (!called("spava_cache_read", c->index, [&](void *stream) {
                return spava_cache_read(&c->cfg, &pools, &batch, first, rows, kop, vop, s.ws, s.bytes, stream);
            }))
            return nullptr;
        return pair(ko, THPVariable_Wrap(vo));
    });
}

// attn(q, table, lens, o, lse, want_lse, workspace)
PyObject *cache_attn(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (!arguments(n, 7, "attn")) return nullptr;
    return guarded([&]() -> PyObject * {
        const Cache *c = reinterpret_cast<Cache *>(self);
        const at::Tensor &q = tensor(a[0], "q");
        const spava_cache_batch batch = batch_of(c, a[1], a[2]);
        const int64_t shape[3] = {batch.n_seqs, c->cfg.n_q_heads, c->cfg.head_dim};
        check(q, shape, at::kBFloat16, c->index, "q");
        const Space s = space_of(c, a[6]);
        const spava_cache_pools pools = pools_of(c);
        const at::Tensor o = output(a[3], shape, at::kBFloat16, c->index, "o");
        const int64_t lse_shape[2] = {c->cfg.n_q_heads, batch.n_seqs};
        const int want = PyObject_IsTrue(a[5]);
        if (want < 0) return nullptr;
        at::Tensor lse;
        if (want || a[4] != Py_None) lse = output(a[4], lse_shape, at::kFloat, c->index, "lse");
        const void *qp = ptr(q, "q");
        void *op = ptr(o, "o");
        float *lp = lse.defined() ? static_cast<float *>(ptr(lse, "lse")) : nullptr;
        if (!called("spava_cache_attn", c->index, [&](void *stream) {
                return spava_cache_attn(&c->cfg, &pools, &batch, qp, op, lp, s.ws, s.bytes, stream);
            }))
            return nullptr;
        return pair(o, lse.defined() ? THPVariable_Wrap(lse) : Py_NewRef(Py_None));
    });
}

#define SPAVA_METHOD(name, f) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef cache_methods[] = {SPAVA_METHOD("write", cache_write), SPAVA_METHOD("append", cache_append),
                               SPAVA_METHOD("read", cache_read), SPAVA_METHOD("attn", cache_attn),
                               {nullptr, nullptr, 0, nullptr}};

PyTypeObject CacheType = {PyVarObject_HEAD_INIT(nullptr, 0)};

// on_failure(f): f(function name, status) raises what a refused call raises
PyObject *on_failure(PyObject *, PyObject *f) {
    Py_INCREF(f);
    Py_XSETREF(g_failed, f);
    Py_RETURN_NONE;
}

PyMethodDef module_methods[] = {{"on_failure", on_failure, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, module_methods};

template <typename T>
int add_type(PyObject *m, PyTypeObject &t, const char *name, const char *full, PyMethodDef *methods, PyMemberDef *members,
             initproc init) {
    t.tp_name = full;
    t.tp_basicsize = sizeof(T);
    t.tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_HAVE_GC;
    t.tp_methods = methods;
    t.tp_members = members;
    t.tp_init = init;
    t.tp_new = PyType_GenericNew;
    t.tp_traverse = visit_kept<T>;
    t.tp_clear = clear_kept<T>;
    t.tp_dealloc = dealloc<T>;
    if (PyType_Ready(&t) < 0) return -1;
    return PyModule_AddObjectRef(m, name, reinterpret_cast<PyObject *>(&t));
}

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
    PyObject *m = PyModule_Create(&module);
    if (!m) return nullptr;
    if (add_type<Rope>(m, RopeType, "Rope", "_calls.Rope", rope_methods, rope_members, rope_init) < 0 ||
        add_type<Cache>(m, CacheType, "Cache", "_calls.Cache", cache_methods, cache_members, cache_init) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
