// marshal.cpp -- the argument checks and marshalling of the short calls (the gated linear recurrence, the state slots,
// the conv1d's gradient) in C++: what the Python functions of the same names do, at a tenth of the time.
//
// Every function here takes the ordinary case only: exact torch tensors, dense, of the right types and shapes, on the
// current device, on the current stream.  It then calls the C entry and returns the call's result, or the entry's status
// as an int if that is not zero.  In any other case it touches nothing and returns None, and the caller takes the Python
// way, which says what is wrong.  So the rules have one place (the Python functions); this file may be missing.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gdr.h"

namespace {

struct Entries {
    decltype(&gdr_scan_fwd) scan_fwd;
    decltype(&gdr_scan_bwd) scan_bwd;
    decltype(&gdr_scan_step) scan_step;
    decltype(&gdr_conv1d_bwd) conv1d_bwd;
    decltype(&gdr_conv1d_bwd_workspace) conv1d_bwd_workspace;
    decltype(&gdr_slot_copy) slot_copy;
    decltype(&gdr_slot_fork) slot_fork;
    decltype(&gdr_slot_compact) slot_compact;
    decltype(&gdr_slot_free) slot_free;
} entries;

using Sizes = at::IntArrayRef;

// the arguments of one call, and whether all of them are of the ordinary case so far
struct Args {
    PyObject *const *v;
    int dev;
    gdr_stream_t stream;
    bool ok = true;

    const at::Tensor *tensor(int i) {
        if (!THPVariable_CheckExact(v[i])) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(v[i]);
    }
    bool none(int i) const { return v[i] == Py_None; }
    bool flag(int i) {
        if (v[i] != Py_True && v[i] != Py_False) ok = false;
        return v[i] == Py_True;
    }
    bool plain(const at::Tensor &t) const {
        return t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev && t.is_contiguous();
    }
    // address of the tensor i, NULL for None
    void *ptr(int i, at::ScalarType type, Sizes shape) {
        if (none(i)) return nullptr;
        const at::Tensor *t = tensor(i);
        if (!t || !plain(*t) || t->scalar_type() != type || t->sizes() != shape) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    const float *f32(int i, Sizes shape) { return static_cast<const float *>(ptr(i, at::kFloat, shape)); }
    const int32_t *i32(int i, Sizes shape) { return static_cast<const int32_t *>(ptr(i, at::kInt, shape)); }
};

// the device and stream are a call's last two arguments
bool begin(Args &a, PyObject *const *v, Py_ssize_t n, Py_ssize_t want) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return false;
    }
    a.v = v;
    a.dev = (int)PyLong_AsLong(v[n - 2]);
    a.stream = reinterpret_cast<gdr_stream_t>(PyLong_AsVoidPtr(v[n - 1]));
    return !PyErr_Occurred();
}

int code(at::ScalarType t) {
    return t == at::kFloat ? GDR_F32 : t == at::kBFloat16 ? GDR_BF16 : t == at::kHalf ? GDR_F16 : -1;
}
bool fits(int64_t n) { return n >= 0 && n < (1LL << 31); }

// an output: the given tensor (checked) or a new one
struct Out {
    at::Tensor t;
    void *p = nullptr;
    void take(Args &a, int i, const at::Tensor &like, at::ScalarType type, Sizes shape) {
        if (!a.ok) return;
        if (a.none(i)) {
            t = at::empty(shape, like.options().dtype(type).requires_grad(false));
        } else {
            a.ptr(i, type, shape);
            if (!a.ok) return;
            t = *a.tensor(i);
        }
        p = t.data_ptr();
    }
    // the tensor for Python: the caller's own object where one was given
    PyObject *give(const Args &a, int i) const {
        if (a.none(i)) return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
        return Py_NewRef(a.v[i]);
    }
};

template <typename F> int run(F &&f) {
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = f();
    Py_END_ALLOW_THREADS;
    return st;
}

PyObject *tuple(PyObject *a, PyObject *b, PyObject *c = nullptr, PyObject *d = nullptr) {
    const int n = d ? 4 : c ? 3 : 2;
    PyObject *t = PyTuple_New(n);
    if (!t || !a || !b || (n > 2 && !c)) {
        Py_XDECREF(t);
        Py_XDECREF(a);
        Py_XDECREF(b);
        Py_XDECREF(c);
        Py_XDECREF(d);
        return nullptr;
    }
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    if (c) PyTuple_SET_ITEM(t, 2, c);
    if (d) PyTuple_SET_ITEM(t, 3, d);
    return t;
}

// x (B, N, S, D) and g of a recurrence call
struct Scan {
    const at::Tensor *x = nullptr, *g = nullptr;
    int64_t B = 0, N = 0, S = 0, D = 0;
    at::ScalarType type = at::kFloat, gate = at::kFloat;
    void *px = nullptr, *pg = nullptr;
    bool take(Args &a) {
        x = a.tensor(0);
        g = a.tensor(1);
        if (!a.ok || x->dim() != 4) return false;
        B = x->size(0), N = x->size(1), S = x->size(2), D = x->size(3);
        type = x->scalar_type(), gate = g->scalar_type();
        if (code(type) < 0 || (gate != type && gate != at::kFloat) || !fits(B) || !fits(N) || !fits(S) || !fits(D)) return false;
        px = a.ptr(0, type, x->sizes());
        pg = a.ptr(1, gate, x->sizes());
        return a.ok;
    }
    gdr_dtype dt() const { return static_cast<gdr_dtype>(code(type)); }
    gdr_dtype gt() const { return static_cast<gdr_dtype>(code(gate)); }
};

// x, g, initial_state, lengths, out, final_state, checkpoints, mix, want_final, want_checkpoints
PyObject *scan_fwd(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a;
    if (!begin(a, v, n, 12)) return nullptr;
    Scan s;
    if (!s.take(a)) Py_RETURN_NONE;
    const float *init = a.f32(2, {s.B, s.N, s.D});
    const int32_t *lens = a.i32(3, {s.B});
    const bool mix = a.flag(7), want_final = a.flag(8) || !a.none(5), want_ck = a.flag(9) || !a.none(6);
    Out out, fin, ck;
    out.take(a, 4, *s.x, s.type, s.x->sizes());
    if (want_final) fin.take(a, 5, *s.x, at::kFloat, {s.B, s.N, s.D});
    if (want_ck) ck.take(a, 6, *s.x, at::kFloat, {s.B, s.N, (s.S + 63) / 64, s.D});
    if (!a.ok) Py_RETURN_NONE;
    const int st = run([&] {
        return entries.scan_fwd(s.px, s.pg, init, lens, (int)s.B, (int)s.N, (int)s.S, (int)s.D, s.dt(), s.gt(), mix, out.p,
                                static_cast<float *>(fin.p), static_cast<float *>(ck.p), a.stream);
    });
    if (st) return PyLong_FromLong(st);
    return tuple(out.give(a, 4), fin.give(a, 5), ck.give(a, 6));
    END_HANDLE_TH_ERRORS
}

// x, g, checkpoints, dout, dfinal_state, lengths, dx, dg, dinitial_state, mix, want_dinitial
PyObject *scan_bwd(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a;
    if (!begin(a, v, n, 13)) return nullptr;
    Scan s;
    if (!s.take(a) || a.none(2) || a.none(3)) Py_RETURN_NONE;
    const float *ck = a.f32(2, {s.B, s.N, (s.S + 63) / 64, s.D});
    const void *dout = a.ptr(3, s.type, s.x->sizes());
    const float *df = a.f32(4, {s.B, s.N, s.D});
    const int32_t *lens = a.i32(5, {s.B});
    const bool mix = a.flag(9), want = a.flag(10) || !a.none(8);
    Out dx, dg, di;
    dx.take(a, 6, *s.x, s.type, s.x->sizes());
    dg.take(a, 7, *s.x, s.gate, s.x->sizes());
    if (want) di.take(a, 8, *s.x, at::kFloat, {s.B, s.N, s.D});
    if (!a.ok) Py_RETURN_NONE;
    const int st = run([&] {
        return entries.scan_bwd(s.px, s.pg, ck, dout, df, lens, (int)s.B, (int)s.N, (int)s.S, (int)s.D, s.dt(), s.gt(), mix,
                                dx.p, dg.p, static_cast<float *>(di.p), a.stream);
    });
    if (st) return PyLong_FromLong(st);
    return tuple(dx.give(a, 6), dg.give(a, 7), di.give(a, 8));
    END_HANDLE_TH_ERRORS
}

// x, g, state_pool, indices, lengths, accepted, out, mix, per_token
PyObject *scan_step(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a;
    if (!begin(a, v, n, 11)) return nullptr;
    Scan s;
    if (!s.take(a)) Py_RETURN_NONE;
    const at::Tensor *pool = a.tensor(2), *idx = a.tensor(3);
    if (!a.ok || pool->dim() != 3 || !fits(pool->size(0)) || idx->numel() != s.B * s.S) Py_RETURN_NONE;
    void *pp = a.ptr(2, at::kFloat, {pool->size(0), s.N, s.D});
    const int32_t *pi = a.i32(3, idx->sizes()), *lens = a.i32(4, {s.B}), *acc = a.i32(5, {s.B});
    const bool mix = a.flag(7), per_token = a.flag(8);
    Out out;
    out.take(a, 6, *s.x, s.type, s.x->sizes());
    if (!a.ok) Py_RETURN_NONE;
    const int st = run([&] {
        return entries.scan_step(s.px, s.pg, static_cast<float *>(pp), (int)pool->size(0), pi, lens, acc, (int)s.B, (int)s.N,
                                 (int)s.S, (int)s.D, s.dt(), s.gt(), mix, per_token, out.p, a.stream);
    });
    if (st) return PyLong_FromLong(st);
    return tuple(out.give(a, 6), Py_NewRef(v[2]));
    END_HANDLE_TH_ERRORS
}

// x, weight, dq, dk, dv, bias, conv_state, lengths, dconv_state_out, dx, dweight, dbias, dconv_state, workspace
PyObject *conv1d_bwd(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a;
    if (!begin(a, v, n, 16)) return nullptr;
    const at::Tensor *x = a.tensor(0), *w = a.tensor(1), *dq = a.tensor(2), *dv = a.tensor(4);
    if (!a.ok || x->dim() != 3 || w->dim() != 2 || dq->dim() != 4 || dv->dim() != 4 || a.none(3)) Py_RETURN_NONE;
    const int64_t B = x->size(0), S = x->size(1), C = x->size(2), K = w->size(1);
    const int64_t Nk = dq->size(1), Dk = dq->size(3), Nv = dv->size(1), Dv = dv->size(3);
    for (int64_t d : {B, S, C, K, Nk, Dk, Nv, Dv})
        if (!fits(d)) Py_RETURN_NONE;
    const at::ScalarType type = x->scalar_type();
    if (code(type) < 0 || C != 2 * Nk * Dk + Nv * Dv) Py_RETURN_NONE;
    const void *px = a.ptr(0, type, x->sizes()), *pw = a.ptr(1, type, {C, K}), *pq = a.ptr(2, type, {B, Nk, S, Dk}),
               *pk = a.ptr(3, type, {B, Nk, S, Dk}), *pv = a.ptr(4, type, {B, Nv, S, Dv}), *pb = a.ptr(5, type, {C}),
               *ps = a.ptr(6, type, {B, C, K}), *pds = a.ptr(8, type, {B, C, K});
    const int32_t *lens = a.i32(7, {B});
    if (!a.ok) Py_RETURN_NONE;
    const size_t need = entries.conv1d_bwd_workspace((int)B, (int)S, (int)Nk, (int)Nv, (int)Dk, (int)Dv, (int)K);
    size_t have = need;
    if (!a.none(13)) {
        const at::Tensor *ws = a.tensor(13);
        if (!a.ok || (have = (size_t)ws->numel()) < need) Py_RETURN_NONE;
    }
    Out dx, dw, db, ds, ws;
    if (!a.none(13)) ws.take(a, 13, *x, at::kByte, a.tensor(13)->sizes());
    else if (need) ws.take(a, 13, *x, at::kByte, {(int64_t)need});
    dx.take(a, 9, *x, type, x->sizes());
    dw.take(a, 10, *x, at::kFloat, {C, K});
    db.take(a, 11, *x, at::kFloat, {C});
    ds.take(a, 12, *x, type, {B, C, K});
    if (!a.ok) Py_RETURN_NONE;
    const int st = run([&] {
        return entries.conv1d_bwd(px, pw, pb, ps, lens, pq, pk, pv, pds, (int)B, (int)S, (int)Nk, (int)Nv, (int)Dk, (int)Dv,
                                  (int)K, static_cast<gdr_dtype>(code(type)), dx.p, static_cast<float *>(dw.p),
                                  static_cast<float *>(db.p), ds.p, ws.p, have, a.stream);
    });
    if (st) return PyLong_FromLong(st);
    return tuple(dx.give(a, 9), dw.give(a, 10), db.give(a, 11), ds.give(a, 12));
    END_HANDLE_TH_ERRORS
}

// a tensor or a list or tuple of them, all with the same number of slots
struct Pools {
    gdr_pool p[GDR_MAX_POOLS];
    int n = 0;
    int64_t slots = 0;
    bool add(Args &a, PyObject *o) {
        if (!THPVariable_CheckExact(o) || n == GDR_MAX_POOLS) return false;
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.dim() < 1 || !a.plain(t)) return false;
        if (n == 0) slots = t.size(0);
        if (t.size(0) != slots || slots < 1 || !fits(slots)) return false;
        p[n].data = t.data_ptr();
        p[n].slot_bytes = (size_t)(t.numel() / slots) * t.element_size();
        ++n;
        return true;
    }
    bool take(Args &a, PyObject *o) {
        if (!PyList_Check(o) && !PyTuple_Check(o)) return add(a, o);
        const Py_ssize_t k = PySequence_Fast_GET_SIZE(o);
        for (Py_ssize_t i = 0; i < k; ++i)
            if (!add(a, PySequence_Fast_GET_ITEM(o, i))) return false;
        return k > 0;
    }
};
// a one-dimensional int32 tensor of n entries (n < 0: any number, which it becomes)
const int32_t *list(Args &a, int i, int64_t &n) {
    const at::Tensor *t = a.tensor(i);
    if (!t || t->dim() != 1) {
        a.ok = false;
        return nullptr;
    }
    if (n < 0) n = t->size(0);
    if (!fits(n)) a.ok = false;
    return a.i32(i, {n});
}

// pools, src, dst
PyObject *slot_copy(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a;
    Pools p;
    int64_t k = -1;
    if (!begin(a, v, n, 5)) return nullptr;
    if (!p.take(a, v[0])) Py_RETURN_NONE;
    const int32_t *src = list(a, 1, k), *dst = list(a, 2, k);
    if (!a.ok) Py_RETURN_NONE;
    const int st = run([&] { return entries.slot_copy(p.p, p.n, (int)p.slots, src, dst, (int)k, a.stream); });
    return st ? PyLong_FromLong(st) : Py_NewRef(v[0]);
    END_HANDLE_TH_ERRORS
}

// pools, slot_table, parents, new_slot_table
PyObject *slot_fork(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a;
    Pools p;
    int64_t k = -1;
    if (!begin(a, v, n, 6)) return nullptr;
    if (!p.take(a, v[0])) Py_RETURN_NONE;
    const int32_t *table = list(a, 1, k), *parents = list(a, 2, k);
    Out now;
    if (a.ok) now.take(a, 3, *a.tensor(1), at::kInt, {k});
    if (!a.ok) Py_RETURN_NONE;
    const int st = run([&] {
        return entries.slot_fork(p.p, p.n, (int)p.slots, table, parents, (int)k, static_cast<int32_t *>(now.p), a.stream);
    });
    return st ? PyLong_FromLong(st) : now.give(a, 3);
    END_HANDLE_TH_ERRORS
}

// pools, live, new_slot, n_live
PyObject *slot_compact(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a;
    Pools p;
    if (!begin(a, v, n, 6)) return nullptr;
    if (!p.take(a, v[0])) Py_RETURN_NONE;
    const int32_t *live = list(a, 1, p.slots);
    Out now, count;
    if (a.ok) now.take(a, 2, *a.tensor(1), at::kInt, {p.slots});
    if (a.ok) count.take(a, 3, *a.tensor(1), at::kInt, {1});
    if (!a.ok) Py_RETURN_NONE;
    const int st = run([&] {
        return entries.slot_compact(p.p, p.n, (int)p.slots, live, static_cast<int32_t *>(now.p), static_cast<int32_t *>(count.p),
                                    a.stream);
    });
    if (st) return PyLong_FromLong(st);
    return tuple(now.give(a, 2), count.give(a, 3));
    END_HANDLE_TH_ERRORS
}

// pools, idx, live
PyObject *slot_free(PyObject *, PyObject *const *v, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    Args a;
    Pools p;
    int64_t k = -1;
    if (!begin(a, v, n, 5)) return nullptr;
    if (!p.take(a, v[0])) Py_RETURN_NONE;
    const int32_t *idx = list(a, 1, k);
    int32_t *live = a.none(2) ? nullptr : const_cast<int32_t *>(list(a, 2, p.slots));
    if (!a.ok) Py_RETURN_NONE;
    const int st = run([&] { return entries.slot_free(p.p, p.n, (int)p.slots, idx, (int)k, live, a.stream); });
    return st ? PyLong_FromLong(st) : Py_NewRef(v[0]);
    END_HANDLE_TH_ERRORS
}

// the addresses of the C entries, in the order of Entries
PyObject *bind(PyObject *, PyObject *const *v, Py_ssize_t n) {
    void **e = reinterpret_cast<void **>(&entries);
    if (n != (Py_ssize_t)(sizeof(entries) / sizeof(void *))) {
        PyErr_SetString(PyExc_TypeError, "bind() takes the address of every entry");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) e[i] = PyLong_AsVoidPtr(v[i]);
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

#define GDR_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GDR_METHOD(bind),      GDR_METHOD(scan_fwd),  GDR_METHOD(scan_bwd),     GDR_METHOD(scan_step),
                         GDR_METHOD(conv1d_bwd), GDR_METHOD(slot_copy), GDR_METHOD(slot_fork), GDR_METHOD(slot_compact),
                         GDR_METHOD(slot_free),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Marshalling of the short calls of libgdr.so.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// the version of torch whose headers this was compiled with, for the caller to compare before the first call
PyMODINIT_FUNC PyInit__marshal() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", GDR_TORCH) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
