/* pycall.c -- direct CPython calls of libmoe entry points that decode steps make many times.
 *
 * ctypes converts a call's 20 to 30 arguments in about 3 us, more than the launch itself takes;
 * these wrappers take 0.3.  Same names, same argument order as include/moe.h; pointers are integers
 * or None.  The library is the one that the binding has loaded: bind(name, address) hands over each
 * function.  Python's lock is given up for the call, which may wait for a full queue. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/moe.h"

typedef moe_status_t (*route_fn)(const void*, moe_dtype_t, int64_t, const float*, const float*, int, int, int, moe_score_t,
                                 int, int, int, int, int, float, int32_t*, float*, cudaStream_t);
typedef moe_status_t (*lora_fn)(const void*, moe_dtype_t, int64_t, const uint16_t*, const uint16_t*, const float*,
                                const int32_t*, const int32_t*, const int32_t*, const int32_t*, const int32_t*, int, int,
                                const void*, int64_t, void*, moe_dtype_t, int64_t, int, int, int, int, cudaStream_t);
typedef moe_status_t (*norm_fn)(const void*, moe_dtype_t, int64_t, int, int, const void*, const void*, moe_dtype_t, float,
                                float, const void*, moe_dtype_t, int64_t, int, moe_gate_act_t, const void*, int64_t, float,
                                float, void*, moe_dtype_t, int64_t, void*, moe_dtype_t, int64_t, int, int, cudaStream_t);

static route_fn route = NULL;
static lora_fn lora = NULL;
static norm_fn norm = NULL;

/* Arguments in turn; a failed conversion leaves Python's error set and is looked for once at the end. */
typedef struct {
    PyObject* const* at;
} Args;

static void* ptr(Args* a) {
    PyObject* o = *a->at++;
    return o == Py_None ? NULL : PyLong_AsVoidPtr(o);
}
static int64_t i64(Args* a) { return PyLong_AsLongLong(*a->at++); }
static int i32(Args* a) {
    const long long v = PyLong_AsLongLong(*a->at++);
    if (v < INT_MIN || v > INT_MAX) PyErr_SetString(PyExc_OverflowError, "argument does not fit an int");
    return (int)v;
}
static float f32(Args* a) { return (float)PyFloat_AsDouble(*a->at++); }

static int ready(const char* name, const void* fn, Py_ssize_t n, Py_ssize_t want) {
    if (n != want) PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
    else if (!fn) PyErr_Format(PyExc_RuntimeError, "%s is not bound", name);
    else return 1;
    return 0;
}

static PyObject* call_route(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    if (!ready("moe_route_grouped", (const void*)route, n, 18)) return NULL;
    Args a = {args};
    const void* logits = ptr(&a);
    const int type = i32(&a);
    const int64_t ld = i64(&a);
    const void *bias = ptr(&a), *shared_w = ptr(&a);
    int v[9];
    for (int i = 0; i < 9; ++i) v[i] = i32(&a);
    const float scale = f32(&a);
    void *ids = ptr(&a), *w = ptr(&a), *stream = ptr(&a);
    if (PyErr_Occurred()) return NULL;
    moe_status_t status;
    Py_BEGIN_ALLOW_THREADS
    status = route(logits, (moe_dtype_t)type, ld, bias, shared_w, v[0], v[1], v[2], (moe_score_t)v[3], v[4], v[5], v[6], v[7],
                   v[8], scale, ids, w, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

static PyObject* call_lora(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    if (!ready("moe_lora", (const void*)lora, n, 23)) return NULL;
    Args a = {args};
    const void* x = ptr(&a);
    const int x_type = i32(&a);
    const int64_t ldx = i64(&a);
    const void* p[8];
    for (int i = 0; i < 8; ++i) p[i] = ptr(&a);
    const int tile_m = i32(&a), adapters = i32(&a);
    const void* residual = ptr(&a);
    const int64_t ldr = i64(&a);
    void* out = ptr(&a);
    const int out_type = i32(&a);
    const int64_t ldo = i64(&a);
    const int T = i32(&a), N = i32(&a), K = i32(&a), R = i32(&a);
    void* stream = ptr(&a);
    if (PyErr_Occurred()) return NULL;
    moe_status_t status;
    Py_BEGIN_ALLOW_THREADS
    status = lora(x, (moe_dtype_t)x_type, ldx, p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], tile_m, adapters, residual, ldr,
                  out, (moe_dtype_t)out_type, ldo, T, N, K, R, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

static PyObject* call_norm(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    if (!ready("moe_combine_norm", (const void*)norm, n, 28)) return NULL;
    Args a = {args};
    const void* y = ptr(&a);
    const int y_type = i32(&a);
    const int64_t ldy = i64(&a);
    const int slots = i32(&a), post = i32(&a);
    const void *post_w = ptr(&a), *pre_w = ptr(&a);
    const int w_type = i32(&a);
    const float offset = f32(&a), eps = f32(&a);
    const void* gate = ptr(&a);
    const int gate_type = i32(&a);
    const int64_t ldg = i64(&a);
    const int cols = i32(&a), act = i32(&a);
    const void* h = ptr(&a);
    const int64_t ldh = i64(&a);
    const float alpha = f32(&a), beta = f32(&a);
    void* h_out = ptr(&a);
    const int h_type = i32(&a);
    const int64_t ldho = i64(&a);
    void* n_out = ptr(&a);
    const int n_type = i32(&a);
    const int64_t ldn = i64(&a);
    const int T = i32(&a), H = i32(&a);
    void* stream = ptr(&a);
    if (PyErr_Occurred()) return NULL;
    moe_status_t status;
    Py_BEGIN_ALLOW_THREADS
    status = norm(y, (moe_dtype_t)y_type, ldy, slots, post, post_w, pre_w, (moe_dtype_t)w_type, offset, eps, gate,
                  (moe_dtype_t)gate_type, ldg, cols, (moe_gate_act_t)act, h, ldh, alpha, beta, h_out, (moe_dtype_t)h_type, ldho,
                  n_out, (moe_dtype_t)n_type, ldn, T, H, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

static PyObject* bind(PyObject* self, PyObject* args) {
    const char* name;
    unsigned long long at;
    if (!PyArg_ParseTuple(args, "sK", &name, &at)) return NULL;
    if (!strcmp(name, "moe_route_grouped")) route = (route_fn)(uintptr_t)at;
    else if (!strcmp(name, "moe_lora")) lora = (lora_fn)(uintptr_t)at;
    else if (!strcmp(name, "moe_combine_norm")) norm = (norm_fn)(uintptr_t)at;
    else return PyErr_Format(PyExc_ValueError, "no wrapper of %s", name);
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, NULL},
                                {"moe_route_grouped", (PyCFunction)(void (*)(void))call_route, METH_FASTCALL, NULL},
                                {"moe_lora", (PyCFunction)(void (*)(void))call_lora, METH_FASTCALL, NULL},
                                {"moe_combine_norm", (PyCFunction)(void (*)(void))call_norm, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pycall(void) { return PyModule_Create(&module); }
