/*
 * Argument marshalling of the dense operators' Python entry points (ops.py):
 * reads pointers, types, strides and sizes off the tensors, checks that they
 * fit the call, and makes it.  The same checks in Python took longer (5 us a
 * call) than the launch itself (2.3 us); here they take about 1.5 us.
 *
 * Every function returns the call's moe_status_t as an int; a tensor of
 * another type, shape, device or inner stride than the call takes gives
 * MOE_ERR_INVALID_ARG and nothing is launched.  Tensors are read through
 * their Python attributes only (dtype, shape, stride, get_device, data_ptr).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "moe.h"

enum { BF16 = 1, F32 = 2, U8 = 4, E4M3 = 8, I32 = 16 };
static PyObject* g_dtypes[5];                 /* in the order of the bits above */
static PyObject *g_device, *g_raw_stream;     /* current device; handle of a device's current stream */
static PyObject *s_dtype, *s_shape, *s_stride, *s_get_device, *s_data_ptr, *s_numel, *s_is_contiguous, *s_cuda_stream;

/* 1: fits, 0: refused, -1: a Python error is set */
#define TRY(call)                                                        \
    do {                                                                 \
        const int r_ = (call);                                           \
        if (r_ < 0) return NULL;                                         \
        if (r_ == 0) return PyLong_FromLong(MOE_ERR_INVALID_ARG);        \
    } while (0)

static int call_ll(PyObject* o, PyObject* method, long long* v) {
    PyObject* r = PyObject_CallMethodNoArgs(o, method);
    if (r == NULL) return -1;
    *v = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return *v == -1 && PyErr_Occurred() ? -1 : 1;
}

static int dtype_bit(PyObject* t, int* bit) {
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    if (d == NULL) return -1;
    *bit = 0;
    for (int i = 0; i < 5; ++i)
        if (d == g_dtypes[i]) *bit = 1 << i;
    Py_DECREF(d);
    return 1;
}

static int address(PyObject* t, void** p) {
    PyObject* r = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (r == NULL) return -1;
    *p = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return *p == NULL && PyErr_Occurred() ? -1 : 1;
}

static int on_device(PyObject* t, long long dev) {
    long long d;
    const int r = call_ll(t, s_get_device, &d);      /* -1 for host memory */
    return r < 0 ? r : d == dev;
}

typedef struct {
    void* p;
    int type;              /* moe_type_t */
    int64_t ld, m, n;
} Mat;

/* A [m, n] matrix (-1: any) of one of the types; all zero for None. */
static int mat(PyObject* t, long long dev, int types, int64_t m, int64_t n, Mat* o) {
    memset(o, 0, sizeof(*o));
    if (t == Py_None) return 1;
    int bit, r = dtype_bit(t, &bit);
    if (r <= 0) return r;
    if (!(bit & types)) return 0;
    if ((r = on_device(t, dev)) <= 0) return r;
    PyObject* shape = PyObject_GetAttr(t, s_shape);
    if (shape == NULL) return -1;
    PyObject* stride = NULL;
    r = 0;
    if (PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 2) {
        r = -1;
        stride = PyObject_CallMethodNoArgs(t, s_stride);
        if (stride != NULL) r = PyTuple_Check(stride) && PyTuple_GET_SIZE(stride) == 2;
    }
    if (r > 0) {
        o->m = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
        o->n = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1));
        o->ld = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 0));
        const int64_t step = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 1));
        if (PyErr_Occurred()) {
            r = -1;
        } else {
            if (o->m <= 1 && o->ld < o->n) o->ld = o->n;
            r = o->ld >= o->n && (step == 1 || o->n == 1) && (m < 0 || o->m == m) && (n < 0 || o->n == n);
        }
    }
    Py_DECREF(shape);
    Py_XDECREF(stride);
    if (r <= 0) return r;
    o->type = bit == F32 ? MOE_TYPE_F32 : MOE_TYPE_BF16;
    return address(t, &o->p);
}

/* A contiguous tensor of n elements; NULL for None. */
static int flat(PyObject* t, long long dev, int types, int64_t n, void** p, int* type) {
    *p = NULL;
    if (t == Py_None) return 1;
    int bit, r = dtype_bit(t, &bit);
    if (r <= 0) return r;
    if (!(bit & types)) return 0;
    if ((r = on_device(t, dev)) <= 0) return r;
    long long k;
    if ((r = call_ll(t, s_numel, &k)) <= 0) return r;
    if (k != n) return 0;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (c == NULL) return -1;
    r = c == Py_True;
    Py_DECREF(c);
    if (r <= 0) return r;
    if (type != NULL) *type = bit == F32 ? MOE_TYPE_F32 : MOE_TYPE_BF16;
    return address(t, p);
}

/* A workspace: uint8, any length. */
static int workspace(PyObject* t, long long dev, void** p, size_t* bytes) {
    *p = NULL;
    *bytes = 0;
    if (t == Py_None) return 1;
    long long k;
    const int r = call_ll(t, s_numel, &k);
    if (r <= 0) return r;
    *bytes = (size_t)k;
    return flat(t, dev, U8, k, p, NULL);
}

static int current_device(long long* dev) {
    PyObject* r = PyObject_CallNoArgs(g_device);
    if (r == NULL) return -1;
    *dev = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return *dev == -1 && PyErr_Occurred() ? -1 : 1;
}

/* The handle of a torch stream, of the device's current one for None. */
static int handle(PyObject* stream, long long dev, void** h) {
    PyObject* r;
    if (stream == Py_None) {
        PyObject* d = PyLong_FromLongLong(dev);
        if (d == NULL) return -1;
        r = PyObject_CallOneArg(g_raw_stream, d);
        Py_DECREF(d);
    } else {
        r = PyObject_GetAttr(stream, s_cuda_stream);
    }
    if (r == NULL) return -1;
    *h = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return *h == NULL && PyErr_Occurred() ? -1 : 1;
}

static int arity(Py_ssize_t got, Py_ssize_t want) {
    if (got == want) return 1;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return -1;
}

#define MAKE(call)                               \
    do {                                         \
        moe_status_t st_;                        \
        Py_BEGIN_ALLOW_THREADS                   \
        st_ = (call);                            \
        Py_END_ALLOW_THREADS                     \
        return PyLong_FromLong(st_);             \
    } while (0)

/* (x, w, res, eps, y, r, rstd, codes, scales, sf_layout, stream) */
static PyObject* norm_fwd(PyObject* self, PyObject* const* a, Py_ssize_t k) {
    long long dev;
    Mat x, res, y, r;
    void *w, *rstd, *codes, *scales, *st;
    int wt = 0;
    TRY(arity(k, 11));
    TRY(current_device(&dev));
    TRY(mat(a[0], dev, BF16 | F32, -1, -1, &x));
    TRY(flat(a[1], dev, BF16 | F32, x.n, &w, &wt));
    TRY(mat(a[2], dev, BF16 | F32, x.m, x.n, &res));
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1. && PyErr_Occurred()) return NULL;
    TRY(mat(a[4], dev, BF16 | F32, x.m, x.n, &y));
    TRY(mat(a[5], dev, BF16 | F32, x.m, x.n, &r));
    TRY(flat(a[6], dev, F32, x.m, &rstd, NULL));
    const long layout = PyLong_AsLong(a[9]);
    if (PyErr_Occurred()) return NULL;
    const int64_t rows = layout == MOE_SF_ATOMS ? (x.m + 127) / 128 * 128 : x.m;
    TRY(flat(a[7], dev, U8 | E4M3, rows * x.n, &codes, NULL));
    TRY(flat(a[8], dev, U8, rows * (x.n / 32), &scales, NULL));
    TRY(a[0] != Py_None && a[1] != Py_None && (a[7] == Py_None) == (a[8] == Py_None));
    /* r has the residual's type; its own when there is no residual */
    TRY(a[2] == Py_None || a[5] == Py_None || r.type == res.type);
    TRY(handle(a[10], dev, &st));
    const int rt = a[2] != Py_None ? res.type : (a[5] != Py_None ? r.type : x.type);
    TRY(x.n <= INT32_MAX);
    MAKE(rmsnorm_residual_fwd(x.p, x.type, x.ld, res.p, rt, res.ld, w, wt, (float)eps, x.m, (int)x.n, r.p, r.ld, y.p,
                              y.type, y.ld, rstd, codes, scales, (int)layout, st));
}

/* (dy, r, w, rstd, dres, dx, dw, ws, stream) */
static PyObject* norm_bwd(PyObject* self, PyObject* const* a, Py_ssize_t k) {
    long long dev;
    Mat dy, r, dres, dx;
    void *w, *rstd, *dw, *ws, *st;
    size_t bytes;
    int wt = 0;
    TRY(arity(k, 9));
    TRY(current_device(&dev));
    TRY(mat(a[1], dev, BF16 | F32, -1, -1, &r));
    TRY(mat(a[0], dev, BF16 | F32, r.m, r.n, &dy));
    TRY(flat(a[2], dev, BF16 | F32, r.n, &w, &wt));
    TRY(flat(a[3], dev, F32, r.m, &rstd, NULL));
    TRY(mat(a[4], dev, BF16 | F32, r.m, r.n, &dres));
    TRY(mat(a[5], dev, BF16 | F32, r.m, r.n, &dx));
    TRY(flat(a[6], dev, F32, r.n, &dw, NULL));
    TRY(workspace(a[7], dev, &ws, &bytes));
    for (int i = 0; i < 6; ++i) TRY(i == 4 || a[i] != Py_None);
    TRY(dx.type == r.type && (a[4] == Py_None || dres.type == r.type) && r.n <= INT32_MAX);
    TRY(handle(a[8], dev, &st));
    MAKE(rmsnorm_residual_bwd(dy.p, dy.type, dy.ld, r.p, r.type, r.ld, w, wt, rstd, dres.p, dres.ld, r.m, (int)r.n,
                              dx.p, dx.ld, dw, ws, bytes, st));
}

/* (x, w, bias, act, res, y, z, err, stream) */
static PyObject* lin_fwd(PyObject* self, PyObject* const* a, Py_ssize_t k) {
    long long dev;
    Mat x, w, res, y, z;
    void *bias, *err, *st;
    TRY(arity(k, 9));
    TRY(current_device(&dev));
    TRY(mat(a[0], dev, BF16, -1, -1, &x));
    TRY(mat(a[1], dev, BF16, x.n, -1, &w));
    TRY(flat(a[2], dev, BF16, w.n, &bias, NULL));
    const long act = PyLong_AsLong(a[3]);
    if (act == -1 && PyErr_Occurred()) return NULL;
    TRY(mat(a[4], dev, BF16, x.m, w.n, &res));
    TRY(mat(a[5], dev, BF16, x.m, w.n, &y));
    TRY(mat(a[6], dev, BF16, x.m, w.n, &z));
    TRY(flat(a[7], dev, I32, 1, &err, NULL));
    TRY(a[0] != Py_None && a[1] != Py_None && a[5] != Py_None && w.n <= INT32_MAX);
    TRY(handle(a[8], dev, &st));
    MAKE(linear_fwd(x.p, x.ld, w.p, w.ld, bias, (int)act, res.p, res.ld, x.m, (int)w.n, x.n, y.p, y.ld, z.p, z.ld,
                    err, st));
}

/* (dy, x, w, z, act, dx, dw, dbias, ws, err, stream) */
static PyObject* lin_bwd(PyObject* self, PyObject* const* a, Py_ssize_t k) {
    long long dev;
    Mat dy, x, w, z, dx, dw;
    void *dbias, *ws, *err, *st;
    size_t bytes;
    TRY(arity(k, 11));
    TRY(current_device(&dev));
    TRY(mat(a[0], dev, BF16, -1, -1, &dy));
    TRY(mat(a[1], dev, BF16, dy.m, -1, &x));
    TRY(mat(a[2], dev, BF16, x.n, dy.n, &w));
    TRY(mat(a[3], dev, BF16, dy.m, dy.n, &z));
    const long act = PyLong_AsLong(a[4]);
    if (act == -1 && PyErr_Occurred()) return NULL;
    TRY(mat(a[5], dev, BF16, dy.m, x.n, &dx));
    TRY(mat(a[6], dev, BF16 | F32, x.n, dy.n, &dw));
    TRY(flat(a[7], dev, F32, dy.n, &dbias, NULL));
    TRY(workspace(a[8], dev, &ws, &bytes));
    TRY(flat(a[9], dev, I32, 1, &err, NULL));
    TRY(a[0] != Py_None && a[1] != Py_None && a[2] != Py_None && dy.n <= INT32_MAX);
    TRY(handle(a[10], dev, &st));
    MAKE(linear_bwd(dy.p, dy.ld, x.p, x.ld, w.p, w.ld, z.p, z.ld, (int)act, dy.m, (int)dy.n, x.n, dx.p, dx.ld, dw.p,
                    dw.type, dw.ld, dbias, ws, bytes, err, st));
}

/* (x, w1, act, h, a, err, stream) */
static PyObject* ffn_fwd(PyObject* self, PyObject* const* a, Py_ssize_t k) {
    long long dev;
    Mat x, w, h, g;
    void *err, *st;
    TRY(arity(k, 7));
    TRY(current_device(&dev));
    TRY(mat(a[0], dev, BF16, -1, -1, &x));
    TRY(mat(a[1], dev, BF16, x.n, -1, &w));
    const long act = PyLong_AsLong(a[2]);
    if (act == -1 && PyErr_Occurred()) return NULL;
    TRY(w.n % 2 == 0 && w.n <= INT32_MAX);
    TRY(mat(a[3], dev, BF16, x.m, w.n / 2, &h));
    TRY(mat(a[4], dev, BF16, x.m, w.n, &g));
    TRY(flat(a[5], dev, I32, 1, &err, NULL));
    TRY(a[0] != Py_None && a[1] != Py_None && a[3] != Py_None);
    TRY(handle(a[6], dev, &st));
    MAKE(gated_ffn_fwd(x.p, x.ld, w.p, w.ld, (int)act, x.m, (int)(w.n / 2), x.n, h.p, h.ld, g.p, g.ld, err, st));
}

/* (dh, a, x, w1, act, da, dx, dw1, err, stream) */
static PyObject* ffn_bwd(PyObject* self, PyObject* const* a, Py_ssize_t k) {
    long long dev;
    Mat dh, g, x, w, da, dx, dw;
    void *err, *st;
    TRY(arity(k, 10));
    TRY(current_device(&dev));
    TRY(mat(a[0], dev, BF16, -1, -1, &dh));
    TRY(dh.n <= INT32_MAX / 2);
    TRY(mat(a[1], dev, BF16, dh.m, 2 * dh.n, &g));
    TRY(mat(a[2], dev, BF16, dh.m, -1, &x));
    TRY(mat(a[3], dev, BF16, x.n, 2 * dh.n, &w));
    const long act = PyLong_AsLong(a[4]);
    if (act == -1 && PyErr_Occurred()) return NULL;
    TRY(mat(a[5], dev, BF16, dh.m, 2 * dh.n, &da));
    TRY(mat(a[6], dev, BF16, dh.m, x.n, &dx));
    TRY(mat(a[7], dev, BF16 | F32, x.n, 2 * dh.n, &dw));
    TRY(flat(a[8], dev, I32, 1, &err, NULL));
    for (int i = 0; i < 6; ++i) TRY(i == 4 || a[i] != Py_None);
    TRY(handle(a[9], dev, &st));
    MAKE(gated_ffn_bwd(dh.p, dh.ld, g.p, g.ld, x.p, x.ld, w.p, w.ld, (int)act, dh.m, (int)dh.n, x.n, da.p, da.ld, dx.p,
                       dx.ld, dw.p, dw.type, dw.ld, err, st));
}

/* (table address, its device, tensors, tiles, p_type, g_type, state_bits, lr, beta1, beta2, eps, step, grad_scale, seed,
   stream); lr and step: a number or a device tensor */
static PyObject* adamw(PyObject* self, PyObject* const* a, Py_ssize_t k) {
    long long dev;
    moe_adamw_opts_t o;
    void *p, *st;
    memset(&o, 0, sizeof(o));
    TRY(arity(k, 15));
    TRY(current_device(&dev));
    void* table = PyLong_AsVoidPtr(a[0]);
    const long long table_dev = PyLong_AsLongLong(a[1]), tiles = PyLong_AsLongLong(a[3]);
    const long tensors = PyLong_AsLong(a[2]), pt = PyLong_AsLong(a[4]), gt = PyLong_AsLong(a[5]);
    const long bits = PyLong_AsLong(a[6]);
    o.beta1 = PyFloat_AsDouble(a[8]);
    o.beta2 = PyFloat_AsDouble(a[9]);
    o.eps = PyFloat_AsDouble(a[10]);
    o.seed = (uint32_t)PyLong_AsUnsignedLongLongMask(a[13]);
    if (PyErr_Occurred()) return NULL;
    TRY(table_dev == dev);      /* every tensor of the plan is where its table is (ops.adamw_plan) */
    if (PyFloat_Check(a[7]) || PyLong_Check(a[7])) {
        o.lr = PyFloat_AsDouble(a[7]);
        if (o.lr == -1. && PyErr_Occurred()) return NULL;
    } else {
        TRY(flat(a[7], dev, F32, 1, &p, NULL));
        TRY(p != NULL);
        o.lr_dev = (const float*)p;
    }
    if (PyLong_Check(a[11])) {
        o.step = PyLong_AsLongLong(a[11]);
    } else {
        TRY(flat(a[11], dev, I32, 1, &p, NULL));
        TRY(p != NULL);
        o.step_dev = (int32_t*)p;
    }
    if (PyErr_Occurred()) return NULL;
    TRY(flat(a[12], dev, F32, 1, &p, NULL));
    o.grad_scale = (const float*)p;
    TRY(handle(a[14], dev, &st));
    MAKE(adamw_step(table, (int)tensors, tiles, (int)pt, (int)gt, (int)bits, &o, st));
}

/* (bfloat16, float32, uint8, float8_e4m3fn, int32, current device, current stream's handle) */
static PyObject* setup(PyObject* self, PyObject* const* a, Py_ssize_t k) {
    TRY(arity(k, 7));
    for (int i = 0; i < 5; ++i) Py_XSETREF(g_dtypes[i], Py_NewRef(a[i]));
    Py_XSETREF(g_device, Py_NewRef(a[5]));
    Py_XSETREF(g_raw_stream, Py_NewRef(a[6]));
    Py_RETURN_NONE;
}

#define FAST(name, fn) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST("setup", setup),
                                FAST("rmsnorm_residual_fwd", norm_fwd),
                                FAST("rmsnorm_residual_bwd", norm_bwd),
                                FAST("linear_fwd", lin_fwd),
                                FAST("linear_bwd", lin_bwd),
                                FAST("gated_ffn_fwd", ffn_fwd),
                                FAST("gated_ffn_bwd", ffn_bwd),
                                FAST("adamw_step", adamw),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
    struct {
        PyObject** s;
        const char* name;
    } const names[] = {{&s_dtype, "dtype"},       {&s_shape, "shape"},   {&s_stride, "stride"},
                       {&s_get_device, "get_device"}, {&s_data_ptr, "data_ptr"}, {&s_numel, "numel"},
                       {&s_is_contiguous, "is_contiguous"}, {&s_cuda_stream, "cuda_stream"}};
    for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
        if ((*names[i].s = PyUnicode_InternFromString(names[i].name)) == NULL) return NULL;
    return PyModule_Create(&module);
}
