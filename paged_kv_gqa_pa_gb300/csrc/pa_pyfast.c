/*
 * pa_pyfast.c -- argument marshalling of q4.py's calls in C (module _pa_fast).
 *
 * A small step's call is mostly host time: through ctypes a call of nine
 * tensors costs 8 us, of which the launch is 2.  Each function here looks at
 * the same things as q4.py's checks (dtype, shape, device, contiguity of every
 * tensor), and in the usual case -- everything in order, the tensors' device
 * the current one, its current stream -- makes the C call and returns its
 * status.  In any other case it does nothing and returns None, and q4.py's
 * own path goes on, which has the messages and the rarer forms.  No Python
 * exception leaves this file, and q4.py works without it.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "../../include/pa_q4.h"

enum { F16, BF16, F32, I32, I64, U8, NUM_TYPES };

static PyObject *s_dtype, *s_shape, *s_get_device, *s_data_ptr, *s_is_contiguous, *s_stride;
static PyObject* types[NUM_TYPES]; /* torch dtypes, compared by identity */
static PyObject *current_device, *current_stream;
static int (*f_write)(int, int, int, int, int, int, const void*, long long, const void*, long long,
                      const int64_t*, void*, uint32_t*, void*);
static int (*f_read)(int, int, int, int, int, int, const void*, const int64_t*, void*, long long,
                     void*, long long, uint32_t*, void*);
static int (*f_decode)(const pa_q4_plan_t*, const void*, const void*, const int32_t*,
                       const int32_t*, float, int, void*, float*, void*, void*);
static int (*f_tables)(int, int, int, int, int, int, const int32_t*, const int32_t*,
                       const int32_t*, int32_t*, int32_t*, int32_t*, int64_t*, int32_t*, int32_t*,
                       uint32_t*, void*);
static int (*f_rope)(int, int, int, int, int, int, const int*, int, int, float, int, const void*,
                     long long, const void*, long long, const int32_t*, void*, long long, void*,
                     long long, void*);

/* A Python int as long long; takes the reference.  0: not one that fits. */
static int as_ll(PyObject* o, long long* out) {
    if (!o) return 0;
    *out = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return !(*out == -1 && PyErr_Occurred());
}

static int call_ll(PyObject* t, PyObject* method, long long* out) {
    return as_ll(PyObject_CallMethodNoArgs(t, method), out);
}

/* An int argument that is neither a bool nor out of a C int's range. */
static int as_int(PyObject* o, int* out) {
    if (!PyLong_CheckExact(o)) return 0;
    const long v = PyLong_AsLong(o);
    if ((v == -1 && PyErr_Occurred()) || v > INT32_MAX || v < INT32_MIN) return 0;
    *out = (int)v;
    return 1;
}

/* The ints of a tuple (a torch.Size); takes the reference. */
static int tuple_ll(PyObject* o, int n, long long* out) {
    int ok = o && PyTuple_Check(o) && PyTuple_GET_SIZE(o) == n;
    for (int i = 0; ok && i < n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
        ok = !(out[i] == -1 && PyErr_Occurred());
    }
    Py_XDECREF(o);
    return ok;
}

static int shape_of(PyObject* t, int n, long long* out) {
    return tuple_ll(PyObject_GetAttr(t, s_shape), n, out);
}

static int has_type(PyObject* t, int type) {
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    const int ok = d && d == types[type];
    Py_XDECREF(d);
    return ok;
}

/* F16, BF16 or F32; -1: another type. */
static int float_type(PyObject* t) {
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    int type = -1;
    for (int i = F16; i <= F32; ++i)
        if (d && d == types[i]) type = i;
    Py_XDECREF(d);
    return type;
}

static int address(PyObject* t, void** out) {
    PyObject* o = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!o) return 0;
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    Py_DECREF(o);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) return 0;
    *out = (void*)(uintptr_t)v;
    return 1;
}

static int on_device(PyObject* t, long long dev) {
    long long d;
    return call_ll(t, s_get_device, &d) && d == dev;
}

/* A contiguous tensor of this type and device; its shape is compared (want) or
 * given back (get). */
static int tensor(PyObject* t, int type, int n, const long long* want, long long* get,
                  long long dev, void** ptr) {
    long long s[4];
    if (!has_type(t, type) || !shape_of(t, n, s) || !on_device(t, dev)) return 0;
    for (int i = 0; i < n; ++i) {
        if (want && s[i] != want[i]) return 0;
        if (get) get[i] = s[i];
    }
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    const int ok = c == Py_True;
    Py_XDECREF(c);
    return ok && address(t, ptr);
}

/* Rows [n, heads, dim] with the heads of a token side by side: address and token stride. */
static int rows(PyObject* t, int type, const long long* want, long long dev, void** ptr,
                long long* stride) {
    long long s[3], st[3];
    if (!has_type(t, type) || !shape_of(t, 3, s) || !on_device(t, dev)) return 0;
    if (s[0] != want[0] || s[1] != want[1] || s[2] != want[2]) return 0;
    if (!tuple_ll(PyObject_CallMethodNoArgs(t, s_stride), 3, st)) return 0;
    if (st[2] != 1 || (st[1] != s[2] && s[1] != 1)) return 0;
    *stride = s[0] > 1 ? st[0] : s[1] * s[2];
    return address(t, ptr);
}

/* The tensor's device if it is the current one, and that device's current stream. */
static int device_and_stream(PyObject* t, long long* dev, void** stream) {
    long long now;
    if (!call_ll(t, s_get_device, dev) || *dev < 0) return 0;
    if (!as_ll(PyObject_CallNoArgs(current_device), &now) || now != *dev) return 0;
    PyObject* d = PyLong_FromLongLong(*dev);
    if (!d) return 0;
    PyObject* o = PyObject_CallOneArg(current_stream, d);
    Py_DECREF(d);
    if (!o) return 0;
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    Py_DECREF(o);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) return 0;
    *stream = (void*)(uintptr_t)v;
    return 1;
}

static int fits(const long long* v, int n) {
    for (int i = 0; i < n; ++i)
        if (v[i] < 0 || v[i] > INT32_MAX) return 0;
    return 1;
}

static PyObject* not_taken(void) {
    PyErr_Clear();
    Py_RETURN_NONE;
}

/* q4_write(k, v, slots, cache) and q4_read(cache, slots, k, v): `order` gives the
 * places of k, v, slots, cache among the arguments. */
static PyObject* cache_call(PyObject* const* a, Py_ssize_t n_args, const int* order, int write) {
    if (n_args != 4) return not_taken();
    PyObject *k = a[order[0]], *v = a[order[1]], *sl = a[order[2]], *c = a[order[3]];
    long long dev, s[3], cs[3], ks, vs;
    void *stream, *kp, *vp, *sp, *cp;
    const int type = float_type(k);
    if (type < 0 || !device_and_stream(k, &dev, &stream) || !shape_of(k, 3, s)) return not_taken();
    if (!tensor(c, U8, 3, NULL, cs, dev, &cp) || cs[1] != s[1] || cs[2] != 20 * s[2] ||
        !fits(s, 3) || !fits(cs, 3) || !rows(k, type, s, dev, &kp, &ks) ||
        !rows(v, type, s, dev, &vp, &vs) || !tensor(sl, I64, 1, s, NULL, dev, &sp))
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

static PyObject* q4_write(PyObject* m, PyObject* const* a, Py_ssize_t n) {
    static const int order[4] = {0, 1, 2, 3};
    (void)m;
    return cache_call(a, n, order, 1);
}

static PyObject* q4_read(PyObject* m, PyObject* const* a, Py_ssize_t n) {
    static const int order[4] = {2, 3, 1, 0};
    (void)m;
    return cache_call(a, n, order, 0);
}

/* q4_decode(plan, q, cache, block_tables, context_lens, scale, window, out, lse, workspace) */
static PyObject* q4_decode(PyObject* m, PyObject* const* a, Py_ssize_t n) {
    (void)m;
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
    void *stream, *q, *c, *bt, *cl, *out, *lse, *ws;
    if (!as_int(a[6], &window) || !device_and_stream(a[1], &dev, &stream) ||
        !tensor(a[1], plan.dtype, 3, qs, NULL, dev, &q) || !tensor(a[2], U8, 3, cs, NULL, dev, &c) ||
        !tensor(a[3], I32, 2, ts, NULL, dev, &bt) || !tensor(a[4], I32, 1, &B, NULL, dev, &cl) ||
        !tensor(a[7], plan.dtype, 3, qs, NULL, dev, &out) ||
        !tensor(a[8], F32, 2, ls, NULL, dev, &lse) ||
        !tensor(a[9], U8, 1, NULL, &ws_n, dev, &ws) || ws_n < 0 ||
        (size_t)ws_n < plan.workspace_bytes)
        return not_taken();
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = f_decode(&plan, q, c, bt, cl, scale, window, out, lse, ws, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

/* extend_tables(past, new, free, num_pages, block_tables, context_lens, starts, slots,
 * positions, pages_taken) */
static PyObject* extend_tables(PyObject* m, PyObject* const* a, Py_ssize_t n) {
    (void)m;
    int pages;
    long long dev, B, B1, cap, nfree, ts[2];
    const long long one = 1;
    void *stream, *past, *fresh, *free_pages, *bt, *cl, *starts, *slots, *pos, *taken;
    if (n != 10 || !as_int(a[3], &pages) || !device_and_stream(a[0], &dev, &stream) ||
        !tensor(a[0], I32, 1, NULL, &B, dev, &past) || !tensor(a[1], I32, 1, &B, NULL, dev, &fresh) ||
        !tensor(a[2], I32, 1, NULL, &nfree, dev, &free_pages) ||
        !tensor(a[4], I32, 2, NULL, ts, dev, &bt) || ts[0] != B ||
        !tensor(a[5], I32, 1, &B, NULL, dev, &cl))
        return not_taken();
    B1 = B + 1;
    if (!tensor(a[6], I32, 1, &B1, NULL, dev, &starts) ||
        !tensor(a[7], I64, 1, NULL, &cap, dev, &slots) ||
        !tensor(a[8], I32, 1, &cap, NULL, dev, &pos) ||
        !tensor(a[9], I32, 1, &one, NULL, dev, &taken) || !fits(&B, 1) || !fits(&cap, 1) ||
        !fits(&nfree, 1) || !fits(ts, 2))
        return not_taken();
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = f_tables((int)B, (int)ts[1], 16, pages, (int)nfree, (int)cap, past, fresh, free_pages,
                      bt, cl, starts, slots, pos, taken, NULL, stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

/* rope_axes(q, k, positions, sections, theta, q_out, k_out, rotary_dim, interleaved, inverse),
 * with q and k both there; q_out, k_out, rotary_dim may be None. */
static PyObject* rope_axes(PyObject* m, PyObject* const* a, Py_ssize_t n) {
    (void)m;
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
    void *stream, *p[4], *pos;
    const int type = float_type(a[0]);
    if (type < 0 || !device_and_stream(a[0], &dev, &stream)) return not_taken();
    for (int i = 0; i < 2; ++i) { /* q, then k */
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
        !tensor(a[2], I32, 2, ps, NULL, dev, &pos))
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

/* setup(types, functions, current_device, current_stream): the six dtypes, the addresses of
 * the five C functions, and torch's two callables. */
static PyObject* setup(PyObject* m, PyObject* args) {
    PyObject *t, *f, *dev, *stream;
    void* fn[5];
    (void)m;
    if (!PyArg_ParseTuple(args, "O!O!OO", &PyTuple_Type, &t, &PyTuple_Type, &f, &dev, &stream))
        return NULL;
    if (PyTuple_GET_SIZE(t) != NUM_TYPES || PyTuple_GET_SIZE(f) != 5) {
        PyErr_SetString(PyExc_ValueError, "setup: six dtypes and five addresses");
        return NULL;
    }
    for (int i = 0; i < 5; ++i) {
        fn[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(f, i));
        if (!fn[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "setup: a null address");
            return NULL;
        }
    }
    for (int i = 0; i < NUM_TYPES; ++i) {
        Py_INCREF(PyTuple_GET_ITEM(t, i));
        Py_XSETREF(types[i], PyTuple_GET_ITEM(t, i));
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

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"q4_write", (PyCFunction)(void (*)(void))q4_write, METH_FASTCALL, NULL},
    {"q4_read", (PyCFunction)(void (*)(void))q4_read, METH_FASTCALL, NULL},
    {"q4_decode", (PyCFunction)(void (*)(void))q4_decode, METH_FASTCALL, NULL},
    {"extend_tables", (PyCFunction)(void (*)(void))extend_tables, METH_FASTCALL, NULL},
    {"rope_axes", (PyCFunction)(void (*)(void))rope_axes, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_fast", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pa_fast(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_stride = PyUnicode_InternFromString("stride");
    if (!s_dtype || !s_shape || !s_get_device || !s_data_ptr || !s_is_contiguous || !s_stride)
        return NULL;
    return PyModule_Create(&module);
}
