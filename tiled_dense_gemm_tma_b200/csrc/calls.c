/*
 * calls.c -- CPython functions over the entry points that a layer makes several
 * times a step (8-bit and 4-bit linear layers, the experts' operators): one per
 * entry point of include/tg_gemm.h, with its arguments in its order, addresses
 * as integers or None, returning the tg_status.  A foreign-function call of 10 to
 * 20 converted arguments takes 1.5 us of host time, these 0.2, of some 9 us that a
 * small call takes in all.
 *
 * The functions check nothing but that the arguments are numbers: binding.py
 * has checked the tensors, and the library checks its arguments.  The
 * interpreter's lock is released during the call.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>

#include "tg_gemm.h"

#define MOST 24

/* The integers of args[0 .. n); args[skip] is left out (a float). */
static int read_args(PyObject *const *args, Py_ssize_t n, Py_ssize_t want, Py_ssize_t skip, int64_t *v) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
        return 0;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (i == skip || args[i] == Py_None) {
            v[i] = 0;
            continue;
        }
        v[i] = PyLong_AsLongLong(args[i]);
        if (v[i] == -1 && PyErr_Occurred()) return 0;
    }
    return 1;
}

/* What does not fit an int becomes the nearest that does, which the library refuses. */
static int narrow(int64_t x) { return x > INT_MAX ? INT_MAX : x < INT_MIN ? INT_MIN : (int)x; }

#define P(i) ((void *)(intptr_t)v[i])
#define I(i) v[i]
#define N(i) narrow(v[i])

#define CALL(name, want, ...)                                                              \
    static PyObject *py_##name(PyObject *self, PyObject *const *args, Py_ssize_t n) {      \
        int64_t v[MOST];                                                                   \
        tg_status s;                                                                       \
        (void)self;                                                                        \
        if (!read_args(args, n, want, -1, v)) return NULL;                                 \
        Py_BEGIN_ALLOW_THREADS s = name(__VA_ARGS__);                                      \
        Py_END_ALLOW_THREADS return PyLong_FromLong(s);                                    \
    }

/* The same with a float at `at`, passed as f. */
#define CALL_F(name, want, at, ...)                                                        \
    static PyObject *py_##name(PyObject *self, PyObject *const *args, Py_ssize_t n) {      \
        int64_t v[MOST];                                                                   \
        tg_status s;                                                                       \
        float f;                                                                           \
        (void)self;                                                                        \
        if (!read_args(args, n, want, at, v)) return NULL;                                 \
        f = (float)PyFloat_AsDouble(args[at]);                                             \
        if (f == -1.0f && PyErr_Occurred()) return NULL;                                   \
        Py_BEGIN_ALLOW_THREADS s = name(__VA_ARGS__);                                      \
        Py_END_ALLOW_THREADS return PyLong_FromLong(s);                                    \
    }

CALL(tg_quant_i8, 9, I(0), I(1), P(2), I(3), N(4), P(5), I(6), P(7), P(8))
CALL(tg_gemm_w8a8, 15, I(0), I(1), I(2), P(3), I(4), P(5), P(6), I(7), N(8), P(9), P(10), I(11), N(12), N(13), P(14))
CALL(tg_gemm_grouped_f16, 15, I(0), I(1), I(2), N(3), P(4), I(5), P(6), P(7), I(8), I(9), N(10), P(11), I(12), N(13),
     P(14))
CALL(tg_gemm_grouped_bf16, 15, I(0), I(1), I(2), N(3), P(4), I(5), P(6), P(7), I(8), I(9), N(10), P(11), I(12), N(13),
     P(14))
CALL(tg_gemm_grouped_wgrad_f16, 13, I(0), I(1), I(2), N(3), P(4), I(5), P(6), I(7), P(8), P(9), I(10), I(11), P(12))
CALL(tg_gemm_grouped_wgrad_bf16, 13, I(0), I(1), I(2), N(3), P(4), I(5), P(6), I(7), P(8), P(9), I(10), I(11), P(12))
CALL(tg_gemm_grouped_w8a8, 19, I(0), I(1), I(2), N(3), P(4), I(5), P(6), P(7), P(8), I(9), I(10), N(11), P(12), I(13),
     P(14), I(15), N(16), N(17), P(18))
CALL(tg_expert_sort, 10, I(0), N(1), N(2), P(3), N(4), P(5), P(6), P(7), P(8), P(9))
CALL(tg_expert_gather, 13, I(0), N(1), I(2), N(3), P(4), I(5), P(6), P(7), P(8), P(9), I(10), P(11), P(12))
CALL(tg_expert_combine, 12, I(0), N(1), I(2), N(3), P(4), I(5), P(6), P(7), P(8), P(9), I(10), P(11))
CALL(tg_expert_combine_grad, 15, I(0), N(1), I(2), N(3), P(4), I(5), P(6), I(7), P(8), P(9), P(10), P(11), I(12),
     P(13), P(14))
CALL(tg_quant_mxfp4, 10, I(0), I(1), P(2), I(3), N(4), P(5), I(6), P(7), I(8), P(9))
CALL(tg_dequant_mxfp4, 10, I(0), I(1), P(2), I(3), P(4), I(5), P(6), I(7), N(8), P(9))
CALL(tg_expert_quant_mxfp4, 13, I(0), N(1), I(2), P(3), I(4), N(5), P(6), P(7), P(8), I(9), P(10), I(11), P(12))
CALL(tg_gemm_mxfp4, 16, I(0), I(1), I(2), P(3), I(4), P(5), I(6), P(7), I(8), P(9), I(10), P(11), I(12), N(13), N(14),
     P(15))
CALL(tg_gemm_grouped_mxfp4, 20, I(0), I(1), I(2), N(3), P(4), I(5), P(6), I(7), P(8), P(9), I(10), I(11), P(12), I(13),
     I(14), P(15), I(16), N(17), N(18), P(19))
CALL_F(tg_expert_route, 15, 11, I(0), N(1), P(2), I(3), N(4), P(5), N(6), N(7), N(8), N(9), N(10), f, P(12), P(13),
       P(14))
CALL_F(tg_expert_route_grad, 14, 8, I(0), N(1), P(2), I(3), N(4), N(5), N(6), N(7), f, P(9), P(10), P(11), I(12),
       P(13))

#define ENTRY(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}

static PyMethodDef methods[] = {
    ENTRY(tg_quant_i8), ENTRY(tg_gemm_w8a8), ENTRY(tg_gemm_grouped_f16), ENTRY(tg_gemm_grouped_bf16),
    ENTRY(tg_gemm_grouped_wgrad_f16), ENTRY(tg_gemm_grouped_wgrad_bf16), ENTRY(tg_gemm_grouped_w8a8),
    ENTRY(tg_expert_sort), ENTRY(tg_expert_gather), ENTRY(tg_expert_combine), ENTRY(tg_expert_combine_grad),
    ENTRY(tg_quant_mxfp4), ENTRY(tg_dequant_mxfp4), ENTRY(tg_expert_quant_mxfp4), ENTRY(tg_gemm_mxfp4),
    ENTRY(tg_gemm_grouped_mxfp4), ENTRY(tg_expert_route), ENTRY(tg_expert_route_grad), {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tg_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tg_calls(void) { return PyModule_Create(&module); }
