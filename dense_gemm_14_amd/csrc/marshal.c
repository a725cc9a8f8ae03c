/*
 * marshal.c -- argument marshalling of the layer calls (CPython C API): the
 * checks of __init__.py's _typed_addr, _workspace and _stream and the call itself,
 * without the interpreter between them. A small product's launch takes 2.3 us;
 * marshalled in Python its call took 4.9 us, and that, not the kernel, was the
 * time of every layer of up to about a million weights.
 *
 * What is not an exact torch.Tensor of BF16 values or their bits on the current
 * device, large enough and contiguous, goes to the Python functions, which know
 * the other kinds of arguments and word the refusals.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>

typedef int (*linear_fn)(int, int, int, const void *, const void *, const void *, int, const void *, void *, void *,
                         void *, size_t, void *);
typedef int (*gated_fn)(int, int, int, const void *, const void *, const void *, int, void *, void *, void *, size_t,
                        void *);
typedef int (*backward_fn)(int, int, int, const void *, const void *, const void *, int, const void *, void *, void *,
                           void *, void *, size_t, void *);

static linear_fn linear_call;
static gated_fn gated_call;
static backward_fn backward_call[2];   /* linear, gated */
static PyObject *tensor_type, *current_device, *raw_stream, *slow_ptr, *slow_workspace, *slow_stream, *bf16, *bits16;
static PyObject *s_get_device, *s_nbytes, *s_is_contiguous, *s_data_ptr, *s_dtype;

static int to_int(PyObject *o, int *out)
{
    long v;
    if (PyLong_Check(o)) {
        v = PyLong_AsLong(o);
    } else {
        PyObject *n = PyNumber_Long(o);
        if (!n)
            return -1;
        v = PyLong_AsLong(n);
        Py_DECREF(n);
    }
    if (v == -1 && PyErr_Occurred())
        return -1;
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_SetString(PyExc_OverflowError, "size beyond 32 bits");
        return -1;
    }
    *out = (int)v;
    return 0;
}

static int long_of(PyObject *o, long long *out)   /* steals o */
{
    if (!o)
        return -1;
    *out = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int address_of(PyObject *o, void **out)    /* steals o: an address or None */
{
    if (!o)
        return -1;
    *out = o == Py_None ? NULL : PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

/* Whether x is a tensor of `need` bytes as the kernels take it; its size. */
static int fits(PyObject *x, size_t need, long device, long long *bytes)
{
    long long v;
    PyObject *c;
    if ((PyObject *)Py_TYPE(x) != tensor_type)
        return 0;
    if (long_of(PyObject_CallMethodNoArgs(x, s_get_device), &v) < 0)
        return -1;
    if (v != device)
        return 0;
    if (long_of(PyObject_GetAttr(x, s_nbytes), bytes) < 0)
        return -1;
    if ((unsigned long long)*bytes < need)
        return 0;
    c = PyObject_CallMethodNoArgs(x, s_is_contiguous);
    if (!c)
        return -1;
    Py_DECREF(c);
    return c == Py_True;
}

/* Whether the tensor x holds BF16 values, under that type or as 16-bit integers. */
static int holds_bf16(PyObject *x)
{
    PyObject *t = PyObject_GetAttr(x, s_dtype);
    if (!t)
        return -1;
    Py_DECREF(t);   /* torch keeps its types */
    return t == bf16 || t == bits16;
}

static int pointer(PyObject *x, size_t need, const char *what, long device, void **out)
{
    long long bytes;
    int ok;
    *out = NULL;
    if (x == Py_None)
        return 0;
    ok = fits(x, need, device, &bytes);
    if (ok > 0)
        ok = holds_bf16(x);
    if (ok < 0)
        return -1;
    if (ok)
        return address_of(PyObject_CallMethodNoArgs(x, s_data_ptr), out);
    return address_of(PyObject_CallFunction(slow_ptr, "Onsl", x, (Py_ssize_t)need, what, device), out);
}

static int workspace(PyObject *ws, PyObject *nbytes, long device, void **out, size_t *size)
{
    long long bytes;
    int ok = 0;
    PyObject *pair;
    *out = NULL;
    *size = 0;
    if (ws == Py_None && nbytes == Py_None)
        return 0;
    if (nbytes == Py_None && (ok = fits(ws, 0, device, &bytes)) < 0)
        return -1;
    if (ok) {
        *size = (size_t)bytes;
        return address_of(PyObject_CallMethodNoArgs(ws, s_data_ptr), out);
    }
    pair = PyObject_CallFunction(slow_workspace, "OOl", ws, nbytes, device);
    if (!pair)
        return -1;
    ok = -1;
    if (PyTuple_Check(pair) && PyTuple_GET_SIZE(pair) == 2) {
        PyObject *p = PyTuple_GET_ITEM(pair, 0);
        Py_INCREF(p);
        ok = address_of(p, out);
        if (ok == 0) {
            *size = PyLong_AsSize_t(PyTuple_GET_ITEM(pair, 1));
            ok = PyErr_Occurred() ? -1 : 0;
        }
    }
    Py_DECREF(pair);
    return ok;
}

static int stream_of(PyObject *s, PyObject *device, void **out)
{
    if (s == Py_None)
        return address_of(PyObject_CallOneArg(raw_stream, device), out);
    return address_of(PyObject_CallFunctionObjArgs(slow_stream, s, device, NULL), out);
}

#define EXPECT(n)                                                                    \
    if (count != (n)) {                                                              \
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", (n), count); \
        return NULL;                                                                 \
    }

/* forward(gated, M, N, K, A, B, bias, activation, R, Z, C, workspace, workspace_bytes, stream) -> status */
static PyObject *forward(PyObject *self, PyObject *const *a, Py_ssize_t count)
{
    int gated, M, N, K, act, status;
    void *A, *B, *bias, *R, *Z, *C, *ws, *stream;
    size_t size, mn, rows;
    long dev;
    PyObject *device;
    EXPECT(14)
    if (to_int(a[0], &gated) || to_int(a[1], &M) || to_int(a[2], &N) || to_int(a[3], &K) || to_int(a[7], &act))
        return NULL;
    device = PyObject_CallNoArgs(current_device);
    if (!device)
        return NULL;
    dev = PyLong_AsLong(device);
    /* (sizes that the call refuses, or that leave nothing to do, need no bytes) */
    rows = M > 0 && N > 0 && K >= 0 ? (gated ? 2 : 1) * (size_t)N : 0;
    mn = rows ? (size_t)M * (size_t)N * 2 : 0;
    status = pointer(a[4], rows ? (size_t)M * (size_t)K * 2 : 0, "A", dev, &A) ||
             pointer(a[5], rows ? rows * (size_t)K * 2 : 0, "B", dev, &B) ||
             pointer(a[6], rows * 2, "bias", dev, &bias) || pointer(a[8], mn, "R", dev, &R) ||
             pointer(a[9], gated ? 2 * mn : mn, "Z", dev, &Z) || pointer(a[10], mn, "C", dev, &C) ||
             workspace(a[11], a[12], dev, &ws, &size) || stream_of(a[13], device, &stream);
    Py_DECREF(device);
    if (status)
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    status = gated ? gated_call(M, N, K, A, B, bias, act, Z, C, ws, size, stream)
                   : linear_call(M, N, K, A, B, bias, act, R, Z, C, ws, size, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* backward(gated, M, N, K, A, B, Z, activation, dC, dA, dB, dbias, workspace, workspace_bytes, stream) -> status */
static PyObject *backward(PyObject *self, PyObject *const *a, Py_ssize_t count)
{
    int gated, M, N, K, act, status, ok;
    void *A, *B, *Z, *dC, *dA, *dB, *dbias, *ws, *stream;
    size_t size, rows, mk, rk;
    long dev;
    PyObject *device;
    EXPECT(15)
    if (to_int(a[0], &gated) || to_int(a[1], &M) || to_int(a[2], &N) || to_int(a[3], &K) || to_int(a[7], &act))
        return NULL;
    device = PyObject_CallNoArgs(current_device);
    if (!device)
        return NULL;
    dev = PyLong_AsLong(device);
    ok = M >= 0 && N >= 0 && K >= 0;   /* (else the call refuses the sizes) */
    rows = ok ? (gated ? 2 : 1) * (size_t)N : 0;
    mk = ok ? (size_t)M * (size_t)K * 2 : 0;
    rk = ok ? rows * (size_t)K * 2 : 0;
    status = pointer(a[4], mk, "A", dev, &A) || pointer(a[5], rk, "B", dev, &B) ||
             pointer(a[6], ok ? (size_t)M * rows * 2 : 0, "Z", dev, &Z) ||
             pointer(a[8], ok ? (size_t)M * (size_t)N * 2 : 0, "dC", dev, &dC) || pointer(a[9], mk, "dA", dev, &dA) ||
             pointer(a[10], rk, "dB", dev, &dB) || pointer(a[11], rows * 2, "dbias", dev, &dbias) ||
             workspace(a[12], a[13], dev, &ws, &size) || stream_of(a[14], device, &stream);
    Py_DECREF(device);
    if (status)
        return NULL;
    Py_BEGIN_ALLOW_THREADS
    status = backward_call[gated != 0](M, N, K, A, B, Z, act, dC, dA, dB, dbias, ws, size, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(status);
}

/* bind(tensor type, current_device, raw_stream, _typed_addr, _workspace, _stream, bfloat16, int16, four addresses) */
static PyObject *bind(PyObject *self, PyObject *args)
{
    unsigned long long f[4];
    PyObject *o[8];
    if (!PyArg_ParseTuple(args, "OOOOOOOOKKKK", &o[0], &o[1], &o[2], &o[3], &o[4], &o[5], &o[6], &o[7], &f[0], &f[1],
                          &f[2], &f[3]))
        return NULL;
    for (int i = 0; i < 8; ++i)
        Py_INCREF(o[i]);   /* kept for the life of the process */
    tensor_type = o[0];
    current_device = o[1];
    raw_stream = o[2];
    slow_ptr = o[3];
    slow_workspace = o[4];
    slow_stream = o[5];
    bf16 = o[6];
    bits16 = o[7];
    linear_call = (linear_fn)(uintptr_t)f[0];
    gated_call = (gated_fn)(uintptr_t)f[1];
    backward_call[0] = (backward_fn)(uintptr_t)f[2];
    backward_call[1] = (backward_fn)(uintptr_t)f[3];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL},
    {"forward", (PyCFunction)(void (*)(void))forward, METH_FASTCALL, NULL},
    {"backward", (PyCFunction)(void (*)(void))backward, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void)
{
    s_get_device = PyUnicode_InternFromString("get_device");
    s_nbytes = PyUnicode_InternFromString("nbytes");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_dtype = PyUnicode_InternFromString("dtype");
    if (!s_get_device || !s_nbytes || !s_is_contiguous || !s_data_ptr || !s_dtype)
        return NULL;
    return PyModule_Create(&module);
}
