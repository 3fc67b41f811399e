/* The layer norm calls' arguments taken from torch tensors in C.
 *
 * A layer norm of a few hundred rows takes the GPU about five microseconds, and
 * the same call through ctypes takes the CPU eight to ten: two thirds of it
 * Python code that asks tensors for pointers, strides and types and converts
 * them one by one.  These functions take the usual case (contiguous tensors of
 * the types that belong together, all large enough, and torch's stream) in less
 * than two microseconds.  Everything else they leave to the binding, which takes
 * it or says what is wrong with it: they return SLOW before anything was called.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "cc_dp.h"

enum { SLOW = -1000 };

typedef int (*forward_fn)(const void *, size_t, const void *, size_t, const void *, const void *,
                          void *, size_t, void *, size_t, float *, float *, size_t, size_t, float,
                          int, int, void *);
typedef int (*backward_fn)(const void *, size_t, const void *, size_t, const void *, const float *,
                           const float *, const void *, size_t, void *, size_t, void *, void *,
                           size_t, size_t, int, int, void *, size_t, void *);

static forward_fn g_forward;
static backward_fn g_backward;
static PyObject *g_dtypes[3];              /* by CC_DTYPE_* code */
static PyObject *g_get_device, *g_get_stream;
static PyObject *s_data_ptr, *s_is_contiguous, *s_dtype, *s_nbytes;

/* Each of these says whether the usual case goes on; no error is left set. */
static int no(void) {
    PyErr_Clear();
    return 0;
}

/* A tensor's address: contiguous, of this type and of `count` elements at least. */
static int pointer(PyObject *t, int code, size_t count, void **out) {
    *out = NULL;
    if (t == Py_None) return 1;
    if (PyLong_Check(t)) return 0;
    PyObject *r = PyObject_GetAttr(t, s_dtype);
    if (!r) return no();
    Py_DECREF(r);
    if (r != g_dtypes[code]) return 0;
    r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!r) return no();
    Py_DECREF(r);
    if (r != Py_True) return 0;
    r = PyObject_GetAttr(t, s_nbytes);
    if (!r) return no();
    const size_t bytes = PyLong_AsSize_t(r);
    Py_DECREF(r);
    if (PyErr_Occurred()) return no();
    if (bytes / (code == CC_DTYPE_F32 ? 4 : 2) < count) return 0;
    r = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!r) return no();
    const unsigned long long v = PyLong_AsUnsignedLongLong(r);
    Py_DECREF(r);
    if (PyErr_Occurred()) return no();
    *out = (void *)(uintptr_t)v;
    return 1;
}

/* Workspace: whatever its type, of these bytes. */
static int workspace(PyObject *t, size_t bytes, void **out) {
    *out = NULL;
    if (t == Py_None) return 1;
    if (PyLong_Check(t)) return 0;
    PyObject *r = PyObject_GetAttr(t, s_nbytes);
    if (!r) return no();
    const size_t has = PyLong_AsSize_t(r);
    Py_DECREF(r);
    if (PyErr_Occurred()) return no();
    if (has < bytes) return 0;
    r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!r) return no();
    Py_DECREF(r);
    if (r != Py_True) return 0;
    r = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!r) return no();
    const unsigned long long v = PyLong_AsUnsignedLongLong(r);
    Py_DECREF(r);
    if (PyErr_Occurred()) return no();
    *out = (void *)(uintptr_t)v;
    return 1;
}

static int size(PyObject *o, size_t *out) {
    if (!PyLong_Check(o)) return 0;
    *out = PyLong_AsSize_t(o);
    return PyErr_Occurred() ? no() : 1;
}

/* The type's code of the first tensor that is there; else as it was. */
static int dtype(PyObject *const *t, int count, int *out) {
    for (int i = 0; i < count; ++i) {
        if (t[i] == Py_None) continue;
        PyObject *d = PyObject_GetAttr(t[i], s_dtype);
        if (!d) return no();
        Py_DECREF(d);
        for (int k = 0; k < 3; ++k)
            if (d == g_dtypes[k]) {
                *out = k;
                return 1;
            }
        return 0;
    }
    return 1;
}

static int stream(void **out) {
    PyObject *d = PyObject_CallNoArgs(g_get_device);
    if (!d) return no();
    PyObject *s = PyObject_CallOneArg(g_get_stream, d);
    Py_DECREF(d);
    if (!s) return no();
    const unsigned long long v = PyLong_AsUnsignedLongLong(s);
    Py_DECREF(s);
    if (PyErr_Occurred()) return no();
    *out = (void *)(uintptr_t)v;
    return 1;
}

/* x, weight, bias, y, mean, rstd, rows, cols, eps, residual, sum_out */
static PyObject *layernorm_forward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    void *x, *w, *b, *y, *mean, *rstd, *residual, *sum, *on;
    size_t rows, cols, all;
    int act = -1, par;
    if (!g_forward || n != 11 || a[0] == Py_None || !size(a[6], &rows) || !size(a[7], &cols) ||
        __builtin_mul_overflow(rows, cols, &all) || !PyFloat_Check(a[8]) || !dtype(a, 1, &act))
        return PyLong_FromLong(SLOW);
    par = act;
    if (!dtype(a + 1, 2, &par) || !pointer(a[0], act, all, &x) || !pointer(a[1], par, cols, &w) ||
        !pointer(a[2], par, cols, &b) || !pointer(a[3], act, all, &y) ||
        !pointer(a[4], CC_DTYPE_F32, rows, &mean) || !pointer(a[5], CC_DTYPE_F32, rows, &rstd) ||
        !pointer(a[9], act, all, &residual) || !pointer(a[10], act, all, &sum) || !stream(&on))
        return PyLong_FromLong(SLOW);
    const float eps = (float)PyFloat_AS_DOUBLE(a[8]);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = g_forward(x, cols, residual, cols, w, b, y, cols, sum, cols, mean, rstd, rows, cols, eps,
                   act, par, on);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* dy, x, weight, mean, rstd, dx, dweight, dbias, rows, cols, workspace,
 * workspace_bytes, dsum */
static PyObject *layernorm_backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    void *dy, *x, *w, *mean, *rstd, *dx, *dw, *db, *ws, *dsum, *on;
    size_t rows, cols, all, bytes;
    int act = -1, par;
    if (!g_backward || n != 13 || a[1] == Py_None || !size(a[8], &rows) || !size(a[9], &cols) ||
        __builtin_mul_overflow(rows, cols, &all) || !size(a[11], &bytes) || !dtype(a + 1, 1, &act))
        return PyLong_FromLong(SLOW);
    par = act;
    PyObject *const params[3] = {a[2], a[6], a[7]};
    if (!dtype(params, 3, &par) || !pointer(a[0], act, all, &dy) || !pointer(a[1], act, all, &x) ||
        !pointer(a[2], par, cols, &w) || !pointer(a[3], CC_DTYPE_F32, rows, &mean) ||
        !pointer(a[4], CC_DTYPE_F32, rows, &rstd) || !pointer(a[5], act, all, &dx) ||
        !pointer(a[6], par, cols, &dw) || !pointer(a[7], par, cols, &db) ||
        !workspace(a[10], bytes, &ws) || !pointer(a[12], act, all, &dsum) || !stream(&on))
        return PyLong_FromLong(SLOW);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = g_backward(dy, cols, x, cols, w, (const float *)mean, (const float *)rstd, dsum, cols, dx,
                    cols, dw, db, rows, cols, act, par, ws, bytes, on);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* (forward address, backward address, (bf16, fp16, fp32), get_device, get_stream) */
static PyObject *setup(PyObject *self, PyObject *args) {
    (void)self;
    unsigned long long forward, backward;
    PyObject *d[3], *get_device, *get_stream;
    if (!PyArg_ParseTuple(args, "KK(OOO)OO", &forward, &backward, &d[0], &d[1], &d[2], &get_device,
                          &get_stream))
        return NULL;
    for (int k = 0; k < 3; ++k) Py_XSETREF(g_dtypes[k], Py_NewRef(d[k]));
    Py_XSETREF(g_get_device, Py_NewRef(get_device));
    Py_XSETREF(g_get_stream, Py_NewRef(get_stream));
    g_forward = (forward_fn)(uintptr_t)forward;
    g_backward = (backward_fn)(uintptr_t)backward;
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"layernorm_forward", (PyCFunction)(void (*)(void))layernorm_forward, METH_FASTCALL, NULL},
    {"layernorm_backward", (PyCFunction)(void (*)(void))layernorm_backward, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_nbytes = PyUnicode_InternFromString("nbytes");
    if (!s_data_ptr || !s_is_contiguous || !s_dtype || !s_nbytes) return NULL;
    return PyModule_Create(&module);
}
