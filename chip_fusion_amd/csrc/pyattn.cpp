// The attention plans' calls from Python, without the interpreter's share: what
// nearly every call passes (tensors of the plan's type and heads on the current
// device, the current stream) is checked, allocated and launched here; anything
// else returns None, and the binding's own checks in Python take it from there.
// None means that nothing has been launched: a status of the run itself is
// raised, since a run that is made again would take states in place twice.
// 77 tokens take 6.0 us a call so, about what the device takes for them, and 10.0
// with all of it in Python.
//
// CPython's API only: tensors are asked for their shape, strides and address
// through their methods, so nothing depends on torch's headers.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include "b2b_attn.h"

namespace {

PyObject *n_shape, *n_stride, *n_data_ptr, *n_dtype, *n_get_device, *n_new_empty;

struct Call {
    PyObject_HEAD
    // the plan, and the library's functions for it
    void *handle, *workspace, *run, *step;
    long heads, kv_heads, dim;
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

// A tensor of that type with n dimensions on device `dev` (-1: any, which it
// returns there): its sizes, strides and address.
bool look(Call* c, PyObject* t, PyObject* dtype, int n, int64_t* size, int64_t* stride, void** p, int64_t* dev) {
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
PyObject* fresh(PyObject* like, PyObject* size, PyObject* dtype, void** p) {
    Ref s(size), kw(Py_BuildValue("{s:O}", "dtype", dtype));
    if (!s.o || !kw.o) return nullptr;
    Ref f(PyObject_GetAttr(like, n_new_empty)), args(PyTuple_Pack(1, s.o));
    if (!f.o || !args.o) return nullptr;
    Ref t(PyObject_Call(f.o, args.o, kw.o));
    int64_t at;
    if (!t.o || !method_int(t.o, n_data_ptr, &at)) return nullptr;
    *p = (void*)at;
    return t.take();
}

// The output: the one that was given, or a dense one like Q.
PyObject* output(Call* c, PyObject* given, PyObject* Q, const b2b_rows_t& q, int64_t rows, b2b_rows_t* o, int64_t* dev) {
    int64_t n;
    if (given != Py_None) {
        if (!rows3(c, given, rows, c->heads, o, &n, dev)) return nullptr;
        Py_INCREF(given);
        return given;
    }
    if (q.row_stride != c->heads * c->dim || (c->heads > 1 && q.head_stride != c->dim)) return nullptr;
    Ref t(PyObject_CallOneArg(c->empty_like, Q));
    int64_t at;
    if (!t.o || !method_int(t.o, n_data_ptr, &at)) return nullptr;
    *o = b2b_rows_t{(const void*)at, (int64_t)c->heads * c->dim, c->dim};
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
    Ref out(output(c, a[5], Q, q, rows, &o, &dev));
    if (!out.o) return other();
    Ref ws(bytes ? fresh(Q, PyLong_FromSize_t(bytes), c->u8, &w) : nullptr);
    if (bytes && !ws.o) return other();
    Ref lse(a[6] == Py_True ? fresh(Q, Py_BuildValue("(Ll)", (long long)rows, c->heads), c->f32, &l) : nullptr);
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
    Ref out(output(c, a[6], a[0], q, batch, &o, &dev));
    if (!out.o) return other();
    Ref ws(bytes ? fresh(a[0], PyLong_FromSize_t(bytes), c->u8, &w) : nullptr);
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
    Ref out(output(c, a[6], a[0], q, rows, &o, &dev));
    if (!out.o) return other();
    Ref after(a[7]);
    if (a[7] != Py_None) Py_INCREF(a[7]);
    else {
        after.o = fresh(a[0], Py_BuildValue("(Llll)", (long long)(ncu - 1), c->heads, c->dim, c->dim), c->f32, &s1);
        if (!after.o) return other();
    }
    Ref ws(bytes ? fresh(a[0], PyLong_FromSize_t(bytes), c->u8, &w) : nullptr);
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
    int64_t rows, at, dev = -1;
    void *g, *s, *s0, *s1;
    if (!linear_operands(c, a, &q, &k, &v, &rows, &g, &dev) || rows > INT32_MAX || !states(c, a[4], rows, &s0, &dev) ||
        (a[6] != Py_None && !states(c, a[6], rows, &s1, &dev)) || !stream_of(c, dev, &s))
        return other();
    Ref out(output(c, a[5], a[0], q, rows, &o, &dev));
    if (!out.o) return other();
    Ref after(a[6]);
    if (a[6] != Py_None) Py_INCREF(a[6]);
    else {
        after.o = PyObject_CallOneArg(c->empty_like, a[4]);
        if (!after.o || !method_int(after.o, n_data_ptr, &at)) return other();
        s1 = (void*)at;
    }
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = ((decltype(&b2b_linear_attn_step))c->step)((b2b_linear_attn_t)c->handle, (int32_t)rows, q, k, v, o, (float*)g, (float*)s0,
                                                    (float*)s1, (hipStream_t)s);
    Py_END_ALLOW_THREADS
    return st ? failed(c, st, "b2b_linear_attn_step") : PyTuple_Pack(2, out.o, after.o);
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

// Call(handle, workspace, run, step, heads, kv_heads, dim, dtype, torch, check): addresses
// of the plan and of the library's functions, as integers; check(status, name)
// raises for a status that is not 0.
PyObject* call_new(PyTypeObject* type, PyObject* args, PyObject*) {
    unsigned long long handle, workspace, run, step;
    long heads, kv, dim;
    PyObject *dtype, *torch, *check;
    if (!PyArg_ParseTuple(args, "KKKKlllOOO", &handle, &workspace, &run, &step, &heads, &kv, &dim, &dtype, &torch, &check))
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
    {"close", call_close, METH_NOARGS, "the plan is gone: every call returns None"},
    {nullptr, nullptr, 0, nullptr}};

PyTypeObject call_type = {PyVarObject_HEAD_INIT(nullptr, 0) "chip_fusion_amd._attn.Call"};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn", "The attention plans' usual calls.", -1, nullptr, nullptr, nullptr,
                      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn(void) {
    struct {
        PyObject** at;
        const char* name;
    } names[] = {{&n_shape, "shape"},           {&n_stride, "stride"},       {&n_data_ptr, "data_ptr"},
                 {&n_dtype, "dtype"},           {&n_get_device, "get_device"}, {&n_new_empty, "new_empty"}};
    for (auto& n : names)
        if (!(*n.at = PyUnicode_InternFromString(n.name))) return nullptr;
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
    return m.take();
}
