// pa_pyfast.cpp -- argument marshalling of q4.py's calls (module _pa_fast).
//
// A small step's call is mostly host time: through ctypes a call of nine
// tensors costs 8 us, of which the launch is 2 (host time a call, Python's
// checks and here: tables 8.4 and 2.4 us, rotary 9.9 and 2.9, decode 7.6 and
// 3.3; through the tensors' Python methods it was 5.3, 5.5 and 4.9).  Each
// function looks at the same things as q4.py's checks (dtype, shape, device,
// contiguity of every tensor), on the tensors themselves, and in the usual case -- everything in
// order, the tensors' device the current one, its current stream -- makes the C
// call and returns its status.  In any other case it does nothing and returns
// None, and q4.py's own path goes on, which has the messages and the rarer
// forms.  No exception leaves this file, and q4.py works without it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

#include <torch/csrc/autograd/python_variable.h>

#include "../../include/pa_q4.h"

namespace {

using at::ScalarType;

PyObject *current_device, *current_stream;
decltype(&pa_q4_write) f_write;
decltype(&pa_q4_read) f_read;
decltype(&pa_q4_decode) f_decode;
decltype(&pa_extend_tables) f_tables;
decltype(&pa_rope_axes) f_rope;

// A Python int as long long; takes the reference.  0: not one that fits.
int as_ll(PyObject* o, long long* out) {
    if (!o) return 0;
    *out = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return !(*out == -1 && PyErr_Occurred());
}

// An int argument that is neither a bool nor out of a C int's range.
int as_int(PyObject* o, int* out) {
    if (!PyLong_CheckExact(o)) return 0;
    const long v = PyLong_AsLong(o);
    if ((v == -1 && PyErr_Occurred()) || v > INT32_MAX || v < INT32_MIN) return 0;
    *out = (int)v;
    return 1;
}

// An address, for a parameter of whatever pointer type.
struct Address {
    void* p = nullptr;
    template <typename X>
    operator X*() const {
        return static_cast<X*>(p);
    }
};

// The tensor of a torch.Tensor (or Parameter, but no other subclass).
const at::Tensor* tensor_of(PyObject* o) {
    return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

// The dtype's number in pa.h; -1: not a float type.
int float_type(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case ScalarType::Half: return PA_DTYPE_F16;
        case ScalarType::BFloat16: return PA_DTYPE_BF16;
        case ScalarType::Float: return PA_DTYPE_F32;
        default: return -1;
    }
}

ScalarType scalar_type(int type) {
    return type == PA_DTYPE_F16    ? ScalarType::Half
           : type == PA_DTYPE_BF16 ? ScalarType::BFloat16
                                   : ScalarType::Float;
}

int shape_of(PyObject* o, int n, long long* out) {
    const at::Tensor* t = tensor_of(o);
    if (!t || t->dim() != n) return 0;
    for (int i = 0; i < n; ++i) out[i] = t->size(i);
    return 1;
}

// A contiguous tensor of this type and device; its shape is compared (want) or
// given back (get).
int tensor(PyObject* o, ScalarType type, int n, const long long* want, long long* get,
           long long dev, Address* ptr) {
    const at::Tensor* t = tensor_of(o);
    if (!t || t->scalar_type() != type || t->dim() != n || t->get_device() != dev) return 0;
    for (int i = 0; i < n; ++i) {
        if (want && t->size(i) != want[i]) return 0;
        if (get) get[i] = t->size(i);
    }
    if (!t->is_contiguous()) return 0;
    ptr->p = t->data_ptr();
    return ptr->p || t->numel() == 0;  // (a meta tensor has no memory)
}

// Rows [n, heads, dim] with the heads of a token side by side: address and token stride.
int rows(PyObject* o, int type, const long long* want, long long dev, Address* ptr,
         long long* stride) {
    const at::Tensor* t = tensor_of(o);
    if (!t || float_type(*t) != type || t->dim() != 3 || t->get_device() != dev) return 0;
    for (int i = 0; i < 3; ++i)
        if (t->size(i) != want[i]) return 0;
    if (t->stride(2) != 1 || (t->stride(1) != want[2] && want[1] != 1)) return 0;
    *stride = want[0] > 1 ? t->stride(0) : want[1] * want[2];
    ptr->p = t->data_ptr();
    return ptr->p || t->numel() == 0;  // (a meta tensor has no memory)
}

// The tensor's device if it is the current one, and that device's current stream.
int device_and_stream(PyObject* o, long long* dev, void** stream) {
    const at::Tensor* t = tensor_of(o);
    long long now;
    if (!t) return 0;
    *dev = t->get_device();  // (-1 without one, which is never the current one)
    if (!as_ll(PyObject_CallNoArgs(current_device), &now) || now != *dev) return 0;
    PyObject* d = PyLong_FromLongLong(*dev);
    if (!d) return 0;
    PyObject* r = PyObject_CallOneArg(current_stream, d);
    Py_DECREF(d);
    if (!r) return 0;
    const unsigned long long v = PyLong_AsUnsignedLongLong(r);
    Py_DECREF(r);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) return 0;
    *stream = (void*)(uintptr_t)v;
    return 1;
}

int fits(const long long* v, int n) {
    for (int i = 0; i < n; ++i)
        if (v[i] < 0 || v[i] > INT32_MAX) return 0;
    return 1;
}

PyObject* not_taken(void) {
    PyErr_Clear();
    Py_RETURN_NONE;
}

// q4_write(k, v, slots, cache) and q4_read(cache, slots, k, v): `order` gives the
// places of k, v, slots, cache among the arguments.
PyObject* cache_call(PyObject* const* a, Py_ssize_t n_args, const int* order, int write) {
    if (n_args != 4) return not_taken();
    PyObject *k = a[order[0]], *v = a[order[1]], *sl = a[order[2]], *c = a[order[3]];
    long long dev, s[3], cs[3], ks, vs;
    void* stream;
    Address kp, vp, sp, cp;
    const at::Tensor* kt = tensor_of(k);
    const int type = kt ? float_type(*kt) : -1;
    if (type < 0 || !device_and_stream(k, &dev, &stream) || !shape_of(k, 3, s)) return not_taken();
    if (!tensor(c, ScalarType::Byte, 3, NULL, cs, dev, &cp) || cs[1] != s[1] || cs[2] != 20 * s[2] ||
        !fits(s, 3) || !fits(cs, 3) || !rows(k, type, s, dev, &kp, &ks) ||
        !rows(v, type, s, dev, &vp, &vs) || !tensor(sl, ScalarType::Long, 1, s, NULL, dev, &sp))
        return not_taken();
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = write ? f_write((int)s[0], (int)s[1], (int)s[2], 16, (int)cs[0], type, kp, ks, vp, vs,
                             sp, cp, NULL, stream)
                   : f_read((int)s[0], (int)s[1], (int)s[2], 16, (int)cs[0], type, cp, sp, kp, ks,
                            vp, vs, NULL, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

PyObject* q4_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    static const int order[4] = {0, 1, 2, 3};
    return cache_call(a, n, order, 1);
}

PyObject* q4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    static const int order[4] = {2, 3, 1, 0};
    return cache_call(a, n, order, 0);
}

// q4_decode(plan, q, cache, block_tables, context_lens, scale, window, out, lse, workspace)
PyObject* q4_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 10 || !PyFloat_CheckExact(a[5])) return not_taken();
    Py_buffer buf;
    if (PyObject_GetBuffer(a[0], &buf, PyBUF_SIMPLE) != 0) return not_taken();
    pa_q4_plan_t plan;
    const int whole = buf.len == (Py_ssize_t)sizeof(plan);
    if (whole) memcpy(&plan, buf.buf, sizeof(plan));
    PyBuffer_Release(&buf);
    if (!whole || plan.dtype < PA_DTYPE_F16 || plan.dtype > PA_DTYPE_BF16) return not_taken();
    const float scale = (float)PyFloat_AS_DOUBLE(a[5]);
    const long long B = plan.batch, Hq = plan.num_q_heads, D = plan.head_dim;
    const long long qs[3] = {B, Hq, D}, ls[2] = {B, Hq};
    const long long cs[3] = {plan.num_pages, plan.num_kv_heads, 20 * D};
    const long long ts[2] = {B, plan.max_pages_per_seq};
    long long dev, ws_n;
    int window;
    void* stream;
    Address q, c, bt, cl, out, lse, ws;
    if (!as_int(a[6], &window) || !device_and_stream(a[1], &dev, &stream) ||
        !tensor(a[1], scalar_type(plan.dtype), 3, qs, NULL, dev, &q) ||
        !tensor(a[2], ScalarType::Byte, 3, cs, NULL, dev, &c) ||
        !tensor(a[3], ScalarType::Int, 2, ts, NULL, dev, &bt) ||
        !tensor(a[4], ScalarType::Int, 1, &B, NULL, dev, &cl) ||
        !tensor(a[7], scalar_type(plan.dtype), 3, qs, NULL, dev, &out) ||
        !tensor(a[8], ScalarType::Float, 2, ls, NULL, dev, &lse) ||
        !tensor(a[9], ScalarType::Byte, 1, NULL, &ws_n, dev, &ws) || ws_n < 0 ||
        (size_t)ws_n < plan.workspace_bytes)
        return not_taken();
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = f_decode(&plan, q, c, bt, cl, scale, window, out, lse, ws, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

// extend_tables(past, new, free, num_pages, block_tables, context_lens, starts, slots,
// positions, pages_taken)
PyObject* extend_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
    int pages;
    long long dev, B, B1, cap, nfree, ts[2];
    const long long one = 1;
    void* stream;
    Address past, fresh, free_pages, bt, cl, starts, slots, pos, taken;
    if (n != 10 || !as_int(a[3], &pages) || !device_and_stream(a[0], &dev, &stream) ||
        !tensor(a[0], ScalarType::Int, 1, NULL, &B, dev, &past) ||
        !tensor(a[1], ScalarType::Int, 1, &B, NULL, dev, &fresh) ||
        !tensor(a[2], ScalarType::Int, 1, NULL, &nfree, dev, &free_pages) ||
        !tensor(a[4], ScalarType::Int, 2, NULL, ts, dev, &bt) || ts[0] != B ||
        !tensor(a[5], ScalarType::Int, 1, &B, NULL, dev, &cl))
        return not_taken();
    B1 = B + 1;
    if (!tensor(a[6], ScalarType::Int, 1, &B1, NULL, dev, &starts) ||
        !tensor(a[7], ScalarType::Long, 1, NULL, &cap, dev, &slots) ||
        !tensor(a[8], ScalarType::Int, 1, &cap, NULL, dev, &pos) ||
        !tensor(a[9], ScalarType::Int, 1, &one, NULL, dev, &taken) || !fits(&B, 1) ||
        !fits(&cap, 1) || !fits(&nfree, 1) || !fits(ts, 2))
        return not_taken();
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = f_tables((int)B, (int)ts[1], 16, pages, (int)nfree, (int)cap, past, fresh, free_pages,
                      bt, cl, starts, slots, pos, taken, NULL, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

// rope_axes(q, k, positions, sections, theta, q_out, k_out, rotary_dim, interleaved, inverse),
// with q and k both there; q_out, k_out, rotary_dim may be None.
PyObject* rope_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 10 || !PyTuple_CheckExact(a[3]) || !PyFloat_CheckExact(a[4]) || !PyBool_Check(a[8]) ||
        !PyBool_Check(a[9]))
        return not_taken();
    const Py_ssize_t axes = PyTuple_GET_SIZE(a[3]);
    int sections[PA_ROPE_MAX_AXES], rot;
    if (axes < 1 || axes > PA_ROPE_MAX_AXES) return not_taken();
    for (Py_ssize_t i = 0; i < axes; ++i)
        if (!as_int(PyTuple_GET_ITEM(a[3], i), &sections[i])) return not_taken();
    const float theta = (float)PyFloat_AS_DOUBLE(a[4]);
    long long dev, s[2][3], st[4], ps[2];
    void* stream;
    Address p[4], pos;
    const at::Tensor* qt = tensor_of(a[0]);
    const int type = qt ? float_type(*qt) : -1;
    if (type < 0 || !device_and_stream(a[0], &dev, &stream)) return not_taken();
    for (int i = 0; i < 2; ++i) {  // q, then k
        if (!shape_of(a[i], 3, s[i]) || !rows(a[i], type, s[i], dev, &p[i], &st[i]))
            return not_taken();
        p[2 + i] = p[i];
        st[2 + i] = st[i];
        if (a[5 + i] != Py_None && !rows(a[5 + i], type, s[i], dev, &p[2 + i], &st[2 + i]))
            return not_taken();
    }
    ps[0] = axes;
    ps[1] = s[0][0];
    if (s[1][0] != s[0][0] || s[1][2] != s[0][2] || !fits(s[0], 3) || !fits(s[1], 3) ||
        !tensor(a[2], ScalarType::Int, 2, ps, NULL, dev, &pos))
        return not_taken();
    rot = (int)s[0][2];
    if (a[7] != Py_None && !as_int(a[7], &rot)) return not_taken();
    const int interleaved = a[8] == Py_True, inverse = a[9] == Py_True;
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = f_rope((int)s[0][0], (int)s[0][1], (int)s[1][1], (int)s[0][2], rot, (int)axes, sections,
                    interleaved, inverse, theta, type, p[0], st[0], p[1], st[1], pos, p[2], st[2],
                    p[3], st[3], stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

// setup(functions, current_device, current_stream): the addresses of the five C functions,
// and torch's two callables.
PyObject* setup(PyObject*, PyObject* args) {
    PyObject *f, *dev, *stream;
    void* fn[5];
    if (!PyArg_ParseTuple(args, "O!OO", &PyTuple_Type, &f, &dev, &stream)) return NULL;
    if (PyTuple_GET_SIZE(f) != 5) {
        PyErr_SetString(PyExc_ValueError, "setup: five addresses");
        return NULL;
    }
    for (int i = 0; i < 5; ++i) {
        fn[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(f, i));
        if (!fn[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "setup: a null address");
            return NULL;
        }
    }
    memcpy(&f_write, &fn[0], sizeof(void*));
    memcpy(&f_read, &fn[1], sizeof(void*));
    memcpy(&f_decode, &fn[2], sizeof(void*));
    memcpy(&f_tables, &fn[3], sizeof(void*));
    memcpy(&f_rope, &fn[4], sizeof(void*));
    Py_INCREF(dev);
    Py_XSETREF(current_device, dev);
    Py_INCREF(stream);
    Py_XSETREF(current_stream, stream);
    Py_RETURN_NONE;
}

// An entry point, with what torch throws (a tensor without memory, say) kept inside.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject* m, PyObject* const* a, Py_ssize_t n) {
    try {
        return F(m, a, n);
    } catch (...) {
        return not_taken();
    }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyCFunction method() {
    return (PyCFunction)(void (*)(void))entry<F>;
}

PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"q4_write", method<q4_write>(), METH_FASTCALL, NULL},
    {"q4_read", method<q4_read>(), METH_FASTCALL, NULL},
    {"q4_decode", method<q4_decode>(), METH_FASTCALL, NULL},
    {"extend_tables", method<extend_tables>(), METH_FASTCALL, NULL},
    {"rope_axes", method<rope_axes>(), METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_fast", NULL, -1, methods, NULL, NULL, NULL, NULL};

}  // namespace

PyMODINIT_FUNC PyInit__pa_fast(void) { return PyModule_Create(&module); }
