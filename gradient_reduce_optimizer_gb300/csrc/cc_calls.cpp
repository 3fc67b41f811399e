/* The layer norm calls' arguments taken from torch tensors in C++.
 *
 * A layer norm of a few hundred rows takes the GPU about five microseconds, and
 * the same call through ctypes takes the CPU eight to ten: two thirds of it
 * Python code that asks tensors for types, sizes, strides and pointers and
 * converts them one by one.  These functions take the usual case (contiguous
 * tensors of the types that belong together, all large enough, and torch's
 * stream) in less than a microsecond.  Everything else they leave to the binding,
 * which takes it or says what is wrong with it: they return SLOW before anything
 * was called.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "cc_dp.h"

namespace {

constexpr long SLOW = -1000;

using forward_fn = decltype(&cc_layernorm_forward);
using backward_fn = decltype(&cc_layernorm_backward);

forward_fn g_forward;
backward_fn g_backward;
PyObject *g_get_device, *g_get_stream;

/* Each of these says whether the usual case goes on; no error is left set. */
bool no() {
    PyErr_Clear();
    return false;
}

bool size(PyObject *o, size_t *out) {
    if (!PyLong_Check(o)) return false;
    *out = PyLong_AsSize_t(o);
    return !PyErr_Occurred() || no();
}

bool is_tensor(PyObject *o) { return THPVariable_CheckExact(o); }

/* The type's code of the first tensor that is there; else as it was. */
bool dtype(PyObject *const *t, int count, int *out) {
    for (int i = 0; i < count; ++i) {
        if (t[i] == Py_None) continue;
        if (!is_tensor(t[i])) return false;
        switch (THPVariable_Unpack(t[i]).scalar_type()) {
            case at::kBFloat16: *out = CC_DTYPE_BF16; return true;
            case at::kHalf: *out = CC_DTYPE_F16; return true;
            case at::kFloat: *out = CC_DTYPE_F32; return true;
            default: return false;
        }
    }
    return true;
}

/* The address of a contiguous tensor of `bytes` bytes at least. */
bool address(const at::Tensor &t, size_t bytes, void **out) {
    if (t.layout() != at::kStrided || !t.is_contiguous() || t.nbytes() < bytes) return false;
    *out = t.data_ptr();
    return true;
}

/* A tensor of this type and of `count` elements at least, or None. */
bool pointer(PyObject *o, int code, size_t count, void **out) {
    *out = nullptr;
    if (o == Py_None) return true;
    int own = -1;
    size_t bytes;
    return is_tensor(o) && dtype(&o, 1, &own) && own == code &&
           !__builtin_mul_overflow(count, static_cast<size_t>(code == CC_DTYPE_F32 ? 4 : 2),
                                   &bytes) &&
           address(THPVariable_Unpack(o), bytes, out);
}

/* Workspace: whatever its type, of these bytes. */
bool workspace(PyObject *o, size_t bytes, void **out) {
    *out = nullptr;
    return o == Py_None || (is_tensor(o) && address(THPVariable_Unpack(o), bytes, out));
}

bool stream(void **out) {
    PyObject *d = PyObject_CallNoArgs(g_get_device);
    if (!d) return no();
    PyObject *s = PyObject_CallOneArg(g_get_stream, d);
    Py_DECREF(d);
    if (!s) return no();
    const unsigned long long v = PyLong_AsUnsignedLongLong(s);
    Py_DECREF(s);
    if (PyErr_Occurred()) return no();
    *out = reinterpret_cast<void *>(static_cast<uintptr_t>(v));
    return true;
}

long forward(PyObject *const *a) {
    void *x, *w, *b, *y, *mean, *rstd, *residual, *sum, *on;
    size_t rows, cols, all;
    int act = -1;
    if (!g_forward || a[0] == Py_None || !size(a[6], &rows) || !size(a[7], &cols) ||
        __builtin_mul_overflow(rows, cols, &all) || !PyFloat_Check(a[8]) || !dtype(a, 1, &act))
        return SLOW;
    int par = act;
    if (!dtype(a + 1, 2, &par) || !pointer(a[0], act, all, &x) || !pointer(a[1], par, cols, &w) ||
        !pointer(a[2], par, cols, &b) || !pointer(a[3], act, all, &y) ||
        !pointer(a[4], CC_DTYPE_F32, rows, &mean) || !pointer(a[5], CC_DTYPE_F32, rows, &rstd) ||
        !pointer(a[9], act, all, &residual) || !pointer(a[10], act, all, &sum) || !stream(&on))
        return SLOW;
    const float eps = static_cast<float>(PyFloat_AS_DOUBLE(a[8]));
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = g_forward(x, cols, residual, cols, w, b, y, cols, sum, cols, static_cast<float *>(mean),
                   static_cast<float *>(rstd), rows, cols, eps, act, par, on);
    Py_END_ALLOW_THREADS
    return st;
}

long backward(PyObject *const *a) {
    void *dy, *x, *w, *mean, *rstd, *dx, *dw, *db, *ws, *dsum, *on;
    size_t rows, cols, all, bytes;
    int act = -1;
    if (!g_backward || a[1] == Py_None || !size(a[8], &rows) || !size(a[9], &cols) ||
        __builtin_mul_overflow(rows, cols, &all) || !size(a[11], &bytes) || !dtype(a + 1, 1, &act))
        return SLOW;
    int par = act;
    PyObject *const params[3] = {a[2], a[6], a[7]};
    if (!dtype(params, 3, &par) || !pointer(a[0], act, all, &dy) || !pointer(a[1], act, all, &x) ||
        !pointer(a[2], par, cols, &w) || !pointer(a[3], CC_DTYPE_F32, rows, &mean) ||
        !pointer(a[4], CC_DTYPE_F32, rows, &rstd) || !pointer(a[5], act, all, &dx) ||
        !pointer(a[6], par, cols, &dw) || !pointer(a[7], par, cols, &db) ||
        !workspace(a[10], bytes, &ws) || !pointer(a[12], act, all, &dsum) || !stream(&on))
        return SLOW;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = g_backward(dy, cols, x, cols, w, static_cast<const float *>(mean),
                    static_cast<const float *>(rstd), dsum, cols, dx, cols, dw, db, rows, cols, act,
                    par, ws, bytes, on);
    Py_END_ALLOW_THREADS
    return st;
}

/* torch's own functions may throw; what does is not the usual case. */
template <long (*CALL)(PyObject *const *), Py_ssize_t COUNT>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
    long st = SLOW;
    try {
        if (n == COUNT) st = CALL(a);
    } catch (...) {
        st = SLOW;
    }
    return PyLong_FromLong(st);
}

/* (forward address, backward address, get_device, get_stream) */
PyObject *setup(PyObject *, PyObject *args) {
    unsigned long long forward_at, backward_at;
    PyObject *get_device, *get_stream;
    if (!PyArg_ParseTuple(args, "KKOO", &forward_at, &backward_at, &get_device, &get_stream))
        return nullptr;
    Py_XSETREF(g_get_device, Py_NewRef(get_device));
    Py_XSETREF(g_get_stream, Py_NewRef(get_stream));
    g_forward = reinterpret_cast<forward_fn>(static_cast<uintptr_t>(forward_at));
    g_backward = reinterpret_cast<backward_fn>(static_cast<uintptr_t>(backward_at));
    Py_RETURN_NONE;
}

template <typename F> PyCFunction method(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

/* x, weight, bias, y, mean, rstd, rows, cols, eps, residual, sum_out;
 * dy, x, weight, mean, rstd, dx, dweight, dbias, rows, cols, workspace,
 * workspace_bytes, dsum */
PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, nullptr},
    {"layernorm_forward", method(entry<forward, 11>), METH_FASTCALL, nullptr},
    {"layernorm_backward", method(entry<backward, 13>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
