// The attention plans' calls from Python, without the interpreter's share: what
// nearly every call passes (tensors of the plan's type and heads on the current
// device, the current stream) is checked, allocated and launched here; anything
// else returns None, and the binding's own checks in Python take it from there.
// None means that nothing has been launched: a status of the run itself is
// raised, since a run that is made again would take states in place twice.
// 77 tokens take 5.7 us a call so, about what the device takes for them, and 10.0
// with all of it in Python; 128 new tokens into their pages, 12 tensors, 5.1 and 16.
//
// CPython's API is enough: tensors are asked for their shape, strides and address
// through their methods (0.5 us a tensor, 1.2 an allocation).  Where it is built
// with torch's own headers (B2B_TORCH, the version's text), torch's plain tensors are
// looked at and made directly instead; subclasses and stand-ins still go through
// their methods.  Those headers hold the layout of one torch's tensors: beside any
// other the module is not imported, and every call is made in Python.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>
#include <initializer_list>

#ifdef B2B_TORCH
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>
#endif

#include "b2b_attn.h"

namespace {

PyObject *n_shape, *n_stride, *n_data_ptr, *n_dtype, *n_get_device, *n_new_empty;

struct Call {
    PyObject_HEAD
    // the plan, and the library's functions for it
    void *handle, *workspace, *run, *step;
    long heads, kv_heads, dim;
    long page, axes, weights;       // keys a page (0: any); of rotations: axes of the positions, whether norms have weights
    // borrowed from the torch module for as long as it lives, held all the same
    PyObject *dtype, *f32, *i32, *u8, *tensor, *empty_like, *get_device, *raw_stream, *check;
};

struct Ref {       // an owned reference
    PyObject* o;
    explicit Ref(PyObject* p = nullptr) : o(p) {}
    ~Ref() { Py_XDECREF(o); }
    Ref(const Ref&) = delete;
    Ref& operator=(const Ref&) = delete;
    PyObject* take() {
        PyObject* p = o;
        o = nullptr;
        return p;
    }
};

bool as_int(PyObject* o, int64_t* v) {
    if (!o) return false;
    *v = PyLong_AsLongLong(o);
    return *v != -1 || !PyErr_Occurred();
}
bool method_int(PyObject* t, PyObject* name, int64_t* v) {
    Ref r(PyObject_CallMethodNoArgs(t, name));
    return as_int(r.o, v);
}
bool ints(PyObject* tuple, int n, int64_t* v) {
    if (!tuple || !PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != n) return false;
    for (int i = 0; i < n; ++i)
        if (!as_int(PyTuple_GET_ITEM(tuple, i), v + i)) return false;
    return true;
}

#ifdef B2B_TORCH
// torch's own tensor, and no subclass with methods of its own.
bool plain(Call* c, PyObject* t) { return c->tensor == THPVariableClass && THPVariable_CheckExact(t); }

// What may throw, without the interpreter's lock: a tensor that allocates, as a new reference.
template <class F>
PyObject* allocate(F make) {
    struct Unlocked {
        PyThreadState* s = PyEval_SaveThread();
        ~Unlocked() { PyEval_RestoreThread(s); }
    };
    try {
        at::Tensor t;
        {
            Unlocked u;
            t = make();
        }
        return THPVariable_Wrap(std::move(t));
    } catch (...) {         // Python makes the call again and says what it is
        return nullptr;
    }
}
#endif

// A tensor of that type with n dimensions on device `dev` (-1: any, which it
// returns there): its sizes, strides and address.
bool look(Call* c, PyObject* t, PyObject* dtype, int n, int64_t* size, int64_t* stride, void** p, int64_t* dev) {
#ifdef B2B_TORCH
    if (plain(c, t)) {
        try {
            const at::Tensor& x = THPVariable_Unpack(t);
            if ((PyObject*)torch::getTHPDtype(x.scalar_type()) != dtype || x.layout() != at::kStrided || x.dim() != n || !x.is_cuda())
                return false;
            for (int i = 0; i < n; ++i) {
                size[i] = x.size(i);
                stride[i] = x.stride(i);
            }
            const int64_t index = x.get_device();
            if (index < 0 || (*dev >= 0 && index != *dev)) return false;
            *dev = index;
            *p = x.data_ptr();
            return *p != nullptr;
        } catch (...) {
            return false;
        }
    }
#endif
    if (!PyObject_TypeCheck(t, (PyTypeObject*)c->tensor)) return false;
    Ref d(PyObject_GetAttr(t, n_dtype));
    if (d.o != dtype) return false;
    Ref s(PyObject_GetAttr(t, n_shape));
    if (!ints(s.o, n, size)) return false;
    Ref st(PyObject_CallMethodNoArgs(t, n_stride));
    if (!ints(st.o, n, stride)) return false;
    int64_t at, index;
    if (!method_int(t, n_get_device, &index) || index < 0 || (*dev >= 0 && index != *dev)) return false;
    *dev = index;
    if (!method_int(t, n_data_ptr, &at) || !at) return false;
    *p = (void*)at;
    return true;
}

// [rows, heads, dim] that the kernels can address (rows < 0: any number)
bool rows3(Call* c, PyObject* t, int64_t rows, long heads, b2b_rows_t* r, int64_t* n, int64_t* dev) {
    int64_t size[3], st[3];
    void* p;
    if (!look(c, t, c->dtype, 3, size, st, &p, dev)) return false;
    if (size[0] < 1 || (rows >= 0 && size[0] != rows) || size[1] != heads || size[2] != c->dim) return false;
    if (st[2] != 1 || st[0] < c->dim || ((st[0] | st[1] | ((intptr_t)p >> 1)) & 7)) return false;
    *n = size[0];
    *r = b2b_rows_t{p, st[0], st[1]};
    return true;
}

// [requests, rows, kv_heads, dim]
bool rows4(Call* c, PyObject* t, int64_t batch, int64_t rows, b2b_rows_t* r, int64_t* n, int64_t* far, int64_t* dev) {
    int64_t size[4], st[4];
    void* p;
    if (!look(c, t, c->dtype, 4, size, st, &p, dev)) return false;
    if (size[0] != batch || size[1] < 1 || (rows >= 0 && size[1] != rows) || size[2] != c->kv_heads || size[3] != c->dim)
        return false;
    if (st[3] != 1 || st[1] < c->dim || ((st[0] | st[1] | st[2] | ((intptr_t)p >> 1)) & 7)) return false;
    *n = size[1];
    *far = st[0];
    *r = b2b_rows_t{p, st[1], st[2]};
    return true;
}

// Pages [pages, size, kv_heads, dim] of a cache (pages < 0: any number; size 0: any)
bool pages4(Call* c, PyObject* t, int64_t* pages, int64_t* size, b2b_pages_t* x, int64_t* dev) {
    int64_t n[4], st[4];
    void* p;
    if (!look(c, t, c->dtype, 4, n, st, &p, dev)) return false;
    if ((*pages >= 0 && n[0] != *pages) || n[0] < 1 || n[0] > INT32_MAX || (*size && n[1] != *size) || n[1] < 1 ||
        n[1] > INT32_MAX || n[2] != c->kv_heads || n[3] != c->dim)
        return false;
    if (st[3] != 1 || ((st[0] | st[1] | st[2] | ((intptr_t)p >> 1)) & 7)) return false;
    *pages = n[0];
    *size = n[1];
    *x = b2b_pages_t{p, st[0], st[1], st[2]};
    return true;
}

// n contiguous values (n < 0: any number, which it returns there)
bool vec(Call* c, PyObject* t, PyObject* dtype, int64_t* n, void** p, int64_t* dev) {
    int64_t size, st;
    if (!look(c, t, dtype, 1, &size, &st, p, dev) || (st != 1 && size > 1) || (*n >= 0 && size != *n)) return false;
    *n = size;
    return true;
}

// float32 states [n, heads, dim, dim], contiguous, 16-byte aligned
bool states(Call* c, PyObject* t, int64_t n, void** p, int64_t* dev) {
    int64_t size[4], st[4];
    if (!look(c, t, c->f32, 4, size, st, p, dev)) return false;
    return size[0] == n && size[1] == c->heads && size[2] == c->dim && size[3] == c->dim && st[3] == 1 &&
           st[2] == c->dim && st[1] == (int64_t)c->dim * c->dim && (n < 2 || st[0] == st[1] * c->heads) &&
           !((intptr_t)*p & 15);
}

// The current device is the tensors': its current stream.
bool stream_of(Call* c, int64_t dev, void** s) {
    int64_t cur, at;
    {
        Ref r(PyObject_CallNoArgs(c->get_device));
        if (!as_int(r.o, &cur) || cur != dev) return false;
    }
    Ref i(PyLong_FromLongLong(dev));
    Ref r(i.o ? PyObject_CallOneArg(c->raw_stream, i.o) : nullptr);
    if (!as_int(r.o, &at)) return false;
    *s = (void*)at;
    return true;
}

// like.new_empty(size, dtype=dtype), its address
PyObject* fresh(Call* c, PyObject* like, std::initializer_list<int64_t> size, PyObject* dtype, void** p) {
#ifdef B2B_TORCH
    if (plain(c, like)) {
        const at::Tensor& x = THPVariable_Unpack(like);
        PyObject* t = allocate([&] {
            return at::empty(at::IntArrayRef(size), x.options().dtype(((THPDtype*)dtype)->scalar_type));
        });
        if (t) *p = THPVariable_Unpack(t).data_ptr();
        return t;
    }
#endif
    Ref s(PyTuple_New((Py_ssize_t)size.size())), kw(Py_BuildValue("{s:O}", "dtype", dtype));
    if (!s.o || !kw.o) return nullptr;
    Py_ssize_t i = 0;
    for (int64_t n : size) {
        PyObject* v = PyLong_FromLongLong(n);
        if (!v) return nullptr;
        PyTuple_SET_ITEM(s.o, i++, v);
    }
    Ref f(PyObject_GetAttr(like, n_new_empty)), args(PyTuple_Pack(1, s.o));
    if (!f.o || !args.o) return nullptr;
    Ref t(PyObject_Call(f.o, args.o, kw.o));
    int64_t at;
    if (!t.o || !method_int(t.o, n_data_ptr, &at)) return nullptr;
    *p = (void*)at;
    return t.take();
}

// torch.empty_like(like), its address
PyObject* fresh_like(Call* c, PyObject* like, void** p) {
#ifdef B2B_TORCH
    if (plain(c, like)) {
        const at::Tensor& x = THPVariable_Unpack(like);
        PyObject* t = allocate([&] { return at::empty_like(x); });
        if (t) *p = THPVariable_Unpack(t).data_ptr();
        return t;
    }
#endif
    Ref t(PyObject_CallOneArg(c->empty_like, like));
    int64_t at;
    if (!t.o || !method_int(t.o, n_data_ptr, &at)) return nullptr;
    *p = (void*)at;
    return t.take();
}

// The output: the one that was given, or a dense one like Q.
PyObject* output(Call* c, PyObject* given, PyObject* Q, const b2b_rows_t& q, int64_t rows, long heads, b2b_rows_t* o,
                 int64_t* dev) {
    int64_t n;
    if (given != Py_None) {
        if (!rows3(c, given, rows, heads, o, &n, dev)) return nullptr;
        Py_INCREF(given);
        return given;
    }
    if (q.row_stride != heads * c->dim || (heads > 1 && q.head_stride != c->dim)) return nullptr;
    void* p;
    Ref t(fresh_like(c, Q, &p));
    if (!t.o) return nullptr;
    *o = b2b_rows_t{p, (int64_t)heads * c->dim, c->dim};
    return t.take();
}

// Not the usual call: None (any exception on the way is not one of its own).
PyObject* other() {
    PyErr_Clear();
    Py_RETURN_NONE;
}

// What a run that was not accepted ends in: check(status, name), which raises.
PyObject* failed(Call* c, int status, const char* name) {
    Ref r(PyObject_CallFunction(c->check, "is", status, name));
    if (r.o) PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, status);
    return nullptr;
}

PyObject* call_attention(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    Call* c = (Call*)self;
    if (na != 7 || !c->handle) return other();
    PyObject *Q = a[0], *cu_k = a[4] == Py_None ? a[3] : a[4];
    b2b_rows_t q, k, v, o;
    int64_t rows, keys, n, dev = -1, nq = -1, nk = -1;
    void *pq, *pk, *s, *w = nullptr, *l = nullptr;
    if (a[6] != Py_False && a[6] != Py_True) return other();
    if (!rows3(c, Q, -1, c->heads, &q, &rows, &dev) || !rows3(c, a[1], -1, c->kv_heads, &k, &keys, &dev) ||
        !rows3(c, a[2], keys, c->kv_heads, &v, &n, &dev) || !vec(c, a[3], c->i32, &nq, &pq, &dev))
        return other();
    if (cu_k == a[3]) pk = pq;
    else if (!vec(c, cu_k, c->i32, &nk, &pk, &dev) || nk != nq) return other();
    size_t bytes;
    if (nq < 1 || nq > INT32_MAX || !stream_of(c, dev, &s) ||
        ((decltype(&b2b_attn_workspace))c->workspace)((b2b_attn_t)c->handle, (int32_t)(nq - 1), rows, keys, &bytes))
        return other();
    Ref out(output(c, a[5], Q, q, rows, c->heads, &o, &dev));
    if (!out.o) return other();
    Ref ws(bytes ? fresh(c, Q, {(int64_t)bytes}, c->u8, &w) : nullptr);
    if (bytes && !ws.o) return other();
    Ref lse(a[6] == Py_True ? fresh(c, Q, {rows, c->heads}, c->f32, &l) : nullptr);
    if (a[6] == Py_True && !lse.o) return other();
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = ((decltype(&b2b_attn_run))c->run)((b2b_attn_t)c->handle, (int32_t)(nq - 1), rows, keys, q, k, v, o, (int32_t*)pq,
                                           (int32_t*)pk, (float*)l, w, bytes, (hipStream_t)s);
    Py_END_ALLOW_THREADS
    if (st) return failed(c, st, "b2b_attn_run");
    return lse.o ? PyTuple_Pack(2, out.o, lse.o) : out.take();
}

PyObject* call_prefix(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    Call* c = (Call*)self;
    if (na != 7 || !c->handle) return other();
    b2b_rows_t q, kp, vp, k, v, o;
    int64_t batch, prefix, own, n, ks, vs, dev = -1;
    void *lens, *s, *w = nullptr;
    if (!rows3(c, a[0], -1, c->heads, &q, &batch, &dev) || !rows3(c, a[1], -1, c->kv_heads, &kp, &prefix, &dev) ||
        !rows3(c, a[2], prefix, c->kv_heads, &vp, &n, &dev) || !rows4(c, a[3], batch, -1, &k, &own, &ks, &dev) ||
        !rows4(c, a[4], batch, own, &v, &n, &vs, &dev))
        return other();
    n = batch;
    size_t bytes;
    if (!vec(c, a[5], c->i32, &n, &lens, &dev) || batch > INT32_MAX || !stream_of(c, dev, &s) ||
        ((decltype(&b2b_prefix_attn_workspace))c->workspace)((b2b_attn_t)c->handle, (int32_t)batch, prefix, own, &bytes))
        return other();
    Ref out(output(c, a[6], a[0], q, batch, c->heads, &o, &dev));
    if (!out.o) return other();
    Ref ws(bytes ? fresh(c, a[0], {(int64_t)bytes}, c->u8, &w) : nullptr);
    if (bytes && !ws.o) return other();
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = ((decltype(&b2b_prefix_attn_run))c->run)((b2b_attn_t)c->handle, (int32_t)batch, prefix, own, q, kp, vp, k, ks, v, vs,
                                                  (int32_t*)lens, o, w, bytes, (hipStream_t)s);
    Py_END_ALLOW_THREADS
    return st ? failed(c, st, "b2b_prefix_attn_run") : out.take();
}

// Q, K, V, log_decay: what prompts and steps have alike
bool linear_operands(Call* c, PyObject* const* a, b2b_rows_t* q, b2b_rows_t* k, b2b_rows_t* v, int64_t* rows, void** g,
                     int64_t* dev) {
    int64_t n, heads = c->heads;
    return rows3(c, a[0], -1, c->heads, q, rows, dev) && rows3(c, a[1], *rows, c->kv_heads, k, &n, dev) &&
           rows3(c, a[2], *rows, c->kv_heads, v, &n, dev) && vec(c, a[3], c->f32, &heads, g, dev);
}

PyObject* call_linear(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    Call* c = (Call*)self;
    if (na != 8 || !c->handle) return other();
    b2b_rows_t q, k, v, o;
    int64_t rows, dev = -1, ncu = -1;
    void *g, *cu, *s, *s0 = nullptr, *s1, *w = nullptr;
    if (!linear_operands(c, a, &q, &k, &v, &rows, &g, &dev) || !vec(c, a[4], c->i32, &ncu, &cu, &dev) || ncu < 2 ||
        ncu > INT32_MAX || (a[5] != Py_None && !states(c, a[5], ncu - 1, &s0, &dev)) ||
        (a[7] != Py_None && !states(c, a[7], ncu - 1, &s1, &dev)))
        return other();
    size_t bytes;
    if (!stream_of(c, dev, &s) || ((decltype(&b2b_linear_attn_workspace))c->workspace)((b2b_linear_attn_t)c->handle, (int32_t)(ncu - 1), rows, &bytes)) return other();
    Ref out(output(c, a[6], a[0], q, rows, c->heads, &o, &dev));
    if (!out.o) return other();
    Ref after(a[7]);
    if (a[7] != Py_None) Py_INCREF(a[7]);
    else {
        after.o = fresh(c, a[0], {ncu - 1, c->heads, c->dim, c->dim}, c->f32, &s1);
        if (!after.o) return other();
    }
    Ref ws(bytes ? fresh(c, a[0], {(int64_t)bytes}, c->u8, &w) : nullptr);
    if (bytes && !ws.o) return other();
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = ((decltype(&b2b_linear_attn_run))c->run)((b2b_linear_attn_t)c->handle, (int32_t)(ncu - 1), rows, q, k, v, o, (float*)g,
                                                  (int32_t*)cu, (float*)s0, (float*)s1, w, bytes, (hipStream_t)s);
    Py_END_ALLOW_THREADS
    return st ? failed(c, st, "b2b_linear_attn_run") : PyTuple_Pack(2, out.o, after.o);
}

PyObject* call_linear_step(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    Call* c = (Call*)self;
    if (na != 7 || !c->handle) return other();
    b2b_rows_t q, k, v, o;
    int64_t rows, dev = -1;
    void *g, *s, *s0, *s1;
    if (!linear_operands(c, a, &q, &k, &v, &rows, &g, &dev) || rows > INT32_MAX || !states(c, a[4], rows, &s0, &dev) ||
        (a[6] != Py_None && !states(c, a[6], rows, &s1, &dev)) || !stream_of(c, dev, &s))
        return other();
    Ref out(output(c, a[5], a[0], q, rows, c->heads, &o, &dev));
    if (!out.o) return other();
    Ref after(a[6]);
    if (a[6] != Py_None) Py_INCREF(a[6]);
    else {
        after.o = fresh_like(c, a[4], &s1);
        if (!after.o) return other();
    }
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = ((decltype(&b2b_linear_attn_step))c->step)((b2b_linear_attn_t)c->handle, (int32_t)rows, q, k, v, o, (float*)g, (float*)s0,
                                                    (float*)s1, (hipStream_t)s);
    Py_END_ALLOW_THREADS
    return st ? failed(c, st, "b2b_linear_attn_step") : PyTuple_Pack(2, out.o, after.o);
}

// A table of pages [seqs, width], lengths and starts (None: a row each) of new tokens
struct Sequences {
    int64_t seqs, width, ld;
    void *table, *lens, *cu;
};
bool sequences(Call* c, PyObject* table, PyObject* lens, PyObject* cu, int64_t rows, Sequences* s, int64_t* dev) {
    int64_t n[2], st[2], starts;
    if (!look(c, table, c->i32, 2, n, st, &s->table, dev) || n[0] < 1 || n[0] >= INT32_MAX || n[1] < 1 || n[1] > INT32_MAX ||
        st[1] != 1 || (n[0] > 1 && st[0] < n[1]))
        return false;
    s->seqs = n[0];
    s->width = n[1];
    s->ld = n[0] > 1 ? st[0] : n[1];
    s->cu = nullptr;
    starts = n[0] + 1;
    return vec(c, lens, c->i32, &s->seqs, &s->lens, dev) &&
           (cu == Py_None ? rows == n[0] : vec(c, cu, c->i32, &starts, &s->cu, dev));
}

PyObject* call_paged(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    Call* c = (Call*)self;
    if (na != 8 || !c->handle || (a[7] != Py_False && a[7] != Py_True)) return other();
    b2b_rows_t q, o;
    b2b_pages_t k, v;
    Sequences x;
    int64_t rows, pages = -1, size = c->page, dev = -1;
    void *s, *w = nullptr, *l = nullptr;
    if (!rows3(c, a[0], -1, c->heads, &q, &rows, &dev) || !pages4(c, a[1], &pages, &size, &k, &dev) ||
        !pages4(c, a[2], &pages, &size, &v, &dev) || !sequences(c, a[3], a[4], a[5], rows, &x, &dev))
        return other();
    size_t bytes;
    if (!stream_of(c, dev, &s) || ((decltype(&b2b_paged_attn_workspace))c->workspace)((b2b_attn_t)c->handle, (int32_t)x.seqs, rows,
                                                                                      (int32_t)x.width, &bytes))
        return other();
    Ref out(output(c, a[6], a[0], q, rows, c->heads, &o, &dev));
    if (!out.o) return other();
    Ref ws(bytes ? fresh(c, a[0], {(int64_t)bytes}, c->u8, &w) : nullptr);
    if (bytes && !ws.o) return other();
    Ref lse(a[7] == Py_True ? fresh(c, a[0], {rows, c->heads}, c->f32, &l) : nullptr);
    if (a[7] == Py_True && !lse.o) return other();
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = ((decltype(&b2b_paged_attn_run))c->run)((b2b_attn_t)c->handle, (int32_t)x.seqs, rows, q, k, v, (int32_t)pages,
                                                 (int32_t*)x.table, (int32_t)x.width, x.ld, (int32_t*)x.lens, (int32_t*)x.cu, o,
                                                 (float*)l, w, bytes, (hipStream_t)s);
    Py_END_ALLOW_THREADS
    if (st) return failed(c, st, "b2b_paged_attn_run");
    return lse.o ? PyTuple_Pack(2, out.o, lse.o) : out.take();
}

// Q, K, positions and weights: what rotations have alike (positions None: null)
struct Turns {
    b2b_rows_t q, k;
    int64_t rows, ld;
    void *positions, *qw, *kw;
};
bool turns(Call* c, PyObject* Q, PyObject* K, PyObject* positions, PyObject* qw, PyObject* kw, Turns* t, int64_t* dev) {
    int64_t n;
    t->positions = t->qw = t->kw = nullptr;
    if (!rows3(c, Q, -1, c->heads, &t->q, &t->rows, dev) || !rows3(c, K, t->rows, c->kv_heads, &t->k, &n, dev)) return false;
    t->ld = t->rows;
    if (positions != Py_None) {
        if (c->axes == 1) {
            n = t->rows;
            if (!vec(c, positions, c->i32, &n, &t->positions, dev)) return false;
        } else {
            int64_t size[2], st[2];
            if (!look(c, positions, c->i32, 2, size, st, &t->positions, dev) || size[0] != c->axes || size[1] != t->rows ||
                (st[1] != 1 && size[1] > 1))
                return false;
            t->ld = st[0];
        }
    }
    PyObject* w[2] = {qw, kw};
    void** to[2] = {&t->qw, &t->kw};
    for (int i = 0; i < 2; ++i) {
        n = c->dim;
        if (w[i] != Py_None && (!c->weights || !vec(c, w[i], c->dtype, &n, to[i], dev) || ((intptr_t)*to[i] & 15))) return false;
    }
    return true;
}

PyObject* call_rotary(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    Call* c = (Call*)self;
    if (na != 7 || !c->handle || a[2] == Py_None) return other();
    Turns t;
    b2b_rows_t qo, ko;
    int64_t dev = -1;
    void* s;
    if (!turns(c, a[0], a[1], a[2], a[3], a[4], &t, &dev) || !stream_of(c, dev, &s)) return other();
    Ref q(output(c, a[5], a[0], t.q, t.rows, c->heads, &qo, &dev));
    Ref k(q.o ? output(c, a[6], a[1], t.k, t.rows, c->kv_heads, &ko, &dev) : nullptr);
    if (!k.o) return other();
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = ((decltype(&b2b_rotary_run))c->run)((b2b_rotary_t)c->handle, t.rows, t.q, t.k, qo, ko, (int32_t*)t.positions, t.ld, t.qw,
                                             t.kw, (hipStream_t)s);
    Py_END_ALLOW_THREADS
    return st ? failed(c, st, "b2b_rotary_run") : PyTuple_Pack(2, q.o, k.o);
}

PyObject* call_append(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    Call* c = (Call*)self;
    if (na != 12 || !c->handle) return other();
    Turns t;
    Sequences x;
    b2b_rows_t v, qo;
    b2b_pages_t kc, vc;
    int64_t n, pages = -1, size = 0, dev = -1;
    void* s;
    if (!turns(c, a[0], a[1], a[8], a[9], a[10], &t, &dev) || !rows3(c, a[2], t.rows, c->kv_heads, &v, &n, &dev) ||
        !pages4(c, a[3], &pages, &size, &kc, &dev) || !pages4(c, a[4], &pages, &size, &vc, &dev) ||
        !sequences(c, a[5], a[6], a[7], t.rows, &x, &dev) || !stream_of(c, dev, &s))
        return other();
    Ref q(output(c, a[11], a[0], t.q, t.rows, c->heads, &qo, &dev));
    if (!q.o) return other();
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = ((decltype(&b2b_rotary_append))c->step)((b2b_rotary_t)c->handle, (int32_t)x.seqs, t.rows, t.q, t.k, v, qo, kc, vc,
                                                 (int32_t)pages, (int32_t)size, (int32_t*)x.table, (int32_t)x.width, x.ld,
                                                 (int32_t*)x.lens, (int32_t*)x.cu, (int32_t*)t.positions, t.ld, t.qw, t.kw,
                                                 (hipStream_t)s);
    Py_END_ALLOW_THREADS
    return st ? failed(c, st, "b2b_rotary_append") : q.take();
}

PyObject* call_close(PyObject* self, PyObject*) {
    ((Call*)self)->handle = nullptr;
    Py_RETURN_NONE;
}

PyObject** const held(Call* c, int i) {
    PyObject** all[] = {&c->dtype, &c->f32, &c->i32, &c->u8, &c->tensor, &c->empty_like, &c->get_device, &c->raw_stream,
                        &c->check};
    return i < 9 ? all[i] : nullptr;
}

// Call(handle, workspace, run, step, heads, kv_heads, dim, dtype, torch, check, page, axes,
// weights): addresses of the plan and of the library's functions, as integers;
// check(status, name) raises for a status that is not 0.
PyObject* call_new(PyTypeObject* type, PyObject* args, PyObject*) {
    unsigned long long handle, workspace, run, step;
    long heads, kv, dim, page = 0, axes = 1, weights = 0;
    PyObject *dtype, *torch, *check;
    if (!PyArg_ParseTuple(args, "KKKKlllOOO|lll", &handle, &workspace, &run, &step, &heads, &kv, &dim, &dtype, &torch, &check,
                          &page, &axes, &weights))
        return nullptr;
    Call* c = (Call*)type->tp_alloc(type, 0);
    if (!c) return nullptr;
    c->handle = (void*)handle;
    c->workspace = (void*)workspace;
    c->run = (void*)run;
    c->step = (void*)step;
    c->heads = heads;
    c->kv_heads = kv;
    c->dim = dim;
    c->page = page;
    c->axes = axes;
    c->weights = weights;
    Py_INCREF(dtype);
    c->dtype = dtype;
    Py_INCREF(check);
    c->check = check;
    Ref C(PyObject_GetAttrString(torch, "_C"));
    c->f32 = PyObject_GetAttrString(torch, "float32");
    c->i32 = PyObject_GetAttrString(torch, "int32");
    c->u8 = PyObject_GetAttrString(torch, "uint8");
    c->tensor = PyObject_GetAttrString(torch, "Tensor");
    c->empty_like = PyObject_GetAttrString(torch, "empty_like");
    c->get_device = C.o ? PyObject_GetAttrString(C.o, "_cuda_getDevice") : nullptr;
    c->raw_stream = C.o ? PyObject_GetAttrString(C.o, "_cuda_getCurrentRawStream") : nullptr;
    for (int i = 0; held(c, i); ++i)
        if (!*held(c, i)) {
            Py_DECREF(c);
            return nullptr;
        }
    return (PyObject*)c;
}

void call_dealloc(PyObject* self) {
    Call* c = (Call*)self;
    for (int i = 0; held(c, i); ++i) Py_XDECREF(*held(c, i));
    Py_TYPE(self)->tp_free(self);
}

PyMethodDef call_methods[] = {
    {"attention", (PyCFunction)(void (*)(void))call_attention, METH_FASTCALL, "attention(Q, K, V, cu_q, cu_k, O, lse)"},
    {"prefix", (PyCFunction)(void (*)(void))call_prefix, METH_FASTCALL, "prefix(Q, Kp, Vp, K, V, lens, O)"},
    {"linear", (PyCFunction)(void (*)(void))call_linear, METH_FASTCALL, "linear(Q, K, V, log_decay, cu, state, O, state_out)"},
    {"linear_step", (PyCFunction)(void (*)(void))call_linear_step, METH_FASTCALL,
     "linear_step(Q, K, V, log_decay, state, O, state_out)"},
    {"paged", (PyCFunction)(void (*)(void))call_paged, METH_FASTCALL, "paged(Q, K, V, table, lens, cu, O, lse)"},
    {"rotary", (PyCFunction)(void (*)(void))call_rotary, METH_FASTCALL,
     "rotary(Q, K, positions, q_weight, k_weight, Q_out, K_out)"},
    {"append", (PyCFunction)(void (*)(void))call_append, METH_FASTCALL,
     "append(Q, K, V, k_cache, v_cache, table, lens, cu, positions, q_weight, k_weight, Q_out)"},
    {"close", call_close, METH_NOARGS, "the plan is gone: every call returns None"},
    {nullptr, nullptr, 0, nullptr}};

PyTypeObject call_type = {PyVarObject_HEAD_INIT(nullptr, 0) "chip_fusion_amd._attn.Call"};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn", "The attention plans' usual calls.", -1, nullptr, nullptr, nullptr,
                      nullptr, nullptr};

#ifdef B2B_TORCH
// ImportError unless the process's torch is the one whose headers these are.
bool same_torch() {
    Ref torch(PyImport_ImportModule("torch")), about(PyImport_ImportModule("torch.version"));
    if (!torch.o || !about.o) return false;
    Ref v(PyObject_GetAttrString(torch.o, "__version__")), git(PyObject_GetAttrString(about.o, "git_version"));
    if (!v.o || !git.o) return false;
    Ref here(PyUnicode_FromFormat("%S %S", v.o, git.o));
    if (!here.o) return false;
    if (!PyUnicode_CompareWithASCIIString(here.o, B2B_TORCH)) return true;
    PyErr_Format(PyExc_ImportError, "_attn.so is built for torch %s, this is %U", B2B_TORCH, here.o);
    return false;
}
#endif

}  // namespace

PyMODINIT_FUNC PyInit__attn(void) {
    struct {
        PyObject** at;
        const char* name;
    } names[] = {{&n_shape, "shape"},           {&n_stride, "stride"},       {&n_data_ptr, "data_ptr"},
                 {&n_dtype, "dtype"},           {&n_get_device, "get_device"}, {&n_new_empty, "new_empty"}};
    for (auto& n : names)
        if (!(*n.at = PyUnicode_InternFromString(n.name))) return nullptr;
#ifdef B2B_TORCH
    if (!same_torch()) return nullptr;
    const char* built = B2B_TORCH;
#else
    const char* built = nullptr;
#endif
    call_type.tp_basicsize = sizeof(Call);
    call_type.tp_flags = Py_TPFLAGS_DEFAULT;
    call_type.tp_new = call_new;
    call_type.tp_dealloc = call_dealloc;
    call_type.tp_methods = call_methods;
    call_type.tp_doc = "One plan's calls.";
    if (PyType_Ready(&call_type) < 0) return nullptr;
    Ref m(PyModule_Create(&module));
    if (!m.o) return nullptr;
    Py_INCREF(&call_type);
    if (PyModule_AddObject(m.o, "Call", (PyObject*)&call_type) < 0) {
        Py_DECREF(&call_type);
        return nullptr;
    }
    // the torch whose tensors are looked at directly, or None
    Ref torch(Py_BuildValue("z", built));
    if (!torch.o || PyModule_AddObject(m.o, "torch", torch.o) < 0) return nullptr;
    torch.take();
    return m.take();
}
