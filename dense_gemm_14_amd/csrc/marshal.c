/*
 * marshal.c -- argument marshalling of the layer calls (CPython C API): the
 * checks of __init__.py's _typed_addr, _workspace and _stream and the call itself,
 * without the interpreter between them. A small product's launch takes 2.3 us;
 * marshalled in Python its call took 4.9 us, and that, not the kernel, was the
 * time of every layer of up to about a million weights.
 *
 * What is not a plain torch.Tensor (or Parameter) of BF16 values or their bits on the current
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
static PyObject *tensor_type, *parameter_type, *current_device, *raw_stream, *slow_ptr, *slow_workspace, *slow_stream, *bf16, *bits16;
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

static int is_tensor(PyObject *x)
{
    PyObject *type = (PyObject *)Py_TYPE(x);
    return type == tensor_type || type == parameter_type;
}

/* Whether x is a tensor of `need` bytes as the kernels take it; its size. */
static int fits(PyObject *x, size_t need, long device, long long *bytes)
{
    long long v;
    PyObject *c;
    if (!is_tensor(x))
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

/*
 * The calls at a network's ends (embedding, layer norm, cross entropy). Their
 * arrays are of several types, so the marshalling here takes only what is plain in
 * every respect -- tensors of a type that the call knows, on the current device,
 * large enough and contiguous, sizes that are ints -- and otherwise answers None:
 * __init__.py then goes through the arguments one by one and words the refusal.
 */
enum { BF16 = 0, FP32 = 1, INT32 = 0, INT64 = 1 };   /* the C ABI's types */

typedef int (*embedding_fn)(int, int, int, int, const void *, int, const void *, float, int, void *, void *);
typedef int (*embedding_bwd_fn)(int, int, int, int, const void *, int, const void *, float, int, const void *, void *,
                                void *, size_t, void *);
typedef int (*norm_fn)(int, int, int, const void *, int, const void *, const void *, float, void *, void *, void *, void *);
typedef int (*norm_bwd_fn)(int, int, int, const void *, int, const void *, const void *, const void *, const void *,
                           const void *, void *, void *, void *, void *, size_t, void *);
typedef int (*entropy_fn)(int, int, int, const void *, const void *, int, const void *, void *, void *, void *, size_t,
                          void *);
typedef int (*entropy_bwd_fn)(int, int, int, const void *, const void *, int, const void *, const void *, const void *,
                              void *, void *, void *, size_t, void *);
static embedding_fn embedding_call;
static embedding_bwd_fn embedding_bwd_call;
static norm_fn norm_call;
static norm_bwd_fn norm_bwd_call;
static entropy_fn entropy_call;
static entropy_bwd_fn entropy_bwd_call;
static PyObject *fp32, *int32, *int64;

/* One call's arguments as they are taken: `plain` falls to 0 with the first that
 * is not. */
struct taken {
    PyObject *device;
    long dev;
    int plain;
};

static int size_arg(struct taken *t, PyObject *o)
{
    long v;
    if (!t->plain || !PyLong_CheckExact(o)) {
        t->plain = 0;
        return 0;
    }
    v = PyLong_AsLong(o);
    if (v < 0 || v > INT_MAX) {      /* (an error, too, is left to the long way) */
        PyErr_Clear();
        t->plain = 0;
        return 0;
    }
    return (int)v;
}

static float float_arg(struct taken *t, PyObject *o)
{
    double v = 0.0;
    if (t->plain && PyFloat_CheckExact(o))
        v = PyFloat_AS_DOUBLE(o);
    else if (t->plain && PyLong_CheckExact(o))
        v = PyLong_AsDouble(o);
    else
        t->plain = 0;
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        t->plain = 0;
    }
    return (float)v;
}

/* Address of x, a tensor of `count` elements of either type of a pair; *kind: -1 on
 * the way in for a type that is still open, else the one that it has to be. */
static void *array_arg(struct taken *t, PyObject *x, size_t count, PyObject *type0, size_t size0, PyObject *type1,
                       size_t size1, int *kind)
{
    PyObject *type;
    long long bytes;
    void *p = NULL;
    int is;
    if (!t->plain || x == Py_None)
        return NULL;
    t->plain = 0;
    if (!is_tensor(x) || !(type = PyObject_GetAttr(x, s_dtype)))
        goto out;
    Py_DECREF(type);   /* torch keeps its types */
    is = type == type0 ? 0 : type == type1 ? 1 : -1;
    if (is < 0 || (*kind >= 0 && is != *kind))
        goto out;
    *kind = is;
    if (fits(x, count * (is ? size1 : size0), t->dev, &bytes) <= 0)
        goto out;
    if (address_of(PyObject_CallMethodNoArgs(x, s_data_ptr), &p) == 0)
        t->plain = 1;
out:
    PyErr_Clear();
    return p;
}
static void *values(struct taken *t, PyObject *x, size_t count, int *kind) { return array_arg(t, x, count, bf16, 2, fp32, 4, kind); }
static void *halves(struct taken *t, PyObject *x, size_t count)
{
    int kind = BF16;
    return values(t, x, count, &kind);
}
static void *floats(struct taken *t, PyObject *x, size_t count)
{
    int kind = FP32;
    return values(t, x, count, &kind);
}
static void *id_array(struct taken *t, PyObject *x, size_t count, int *kind) { return array_arg(t, x, count, int32, 4, int64, 8, kind); }

static int begin(struct taken *t)
{
    t->device = PyObject_CallNoArgs(current_device);
    if (!t->device)
        return -1;
    t->dev = PyLong_AsLong(t->device);
    t->plain = 1;
    return 0;
}

/* Workspace and stream, the last arguments; 0 where the call can be made. */
static int finish(struct taken *t, PyObject *ws, PyObject *nbytes, void **w, size_t *size, PyObject *s, void **stream)
{
    int bad = !t->plain || (ws && workspace(ws, nbytes, t->dev, w, size) < 0) || stream_of(s, t->device, stream) < 0;
    Py_DECREF(t->device);
    return bad;
}
#define UNLESS_PLAIN              \
    {                             \
        if (PyErr_Occurred())     \
            return NULL;          \
        Py_RETURN_NONE;           \
    }
#define CALL(...)                 \
    Py_BEGIN_ALLOW_THREADS        \
    status = __VA_ARGS__;         \
    Py_END_ALLOW_THREADS          \
    return PyLong_FromLong(status)

/* embedding(tokens, vocab, cols, ids, E, Y, scale, stream) */
static PyObject *embedding(PyObject *self, PyObject *const *a, Py_ssize_t count)
{
    struct taken t;
    int status, id = -1, et = -1, yt = -1;
    void *stream;
    EXPECT(8)
    if (begin(&t))
        return NULL;
    const int T = size_arg(&t, a[0]), V = size_arg(&t, a[1]), K = size_arg(&t, a[2]);
    void *ids = id_array(&t, a[3], T, &id), *E = values(&t, a[4], (size_t)V * K, &et), *Y = values(&t, a[5], (size_t)T * K, &yt);
    const float scale = float_arg(&t, a[6]);
    if (finish(&t, NULL, NULL, NULL, NULL, a[7], &stream) || id < 0 || et < 0 || yt < 0)
        UNLESS_PLAIN
    CALL(embedding_call(T, V, K, id, ids, et, E, scale, yt, Y, stream));
}

/* embedding_bwd(tokens, vocab, cols, ids, dY, R, dE, scale, workspace, workspace_bytes, stream) */
static PyObject *embedding_bwd(PyObject *self, PyObject *const *a, Py_ssize_t count)
{
    struct taken t;
    int status, id = -1, et = -1, yt = -1;
    void *stream, *ws;
    size_t size;
    EXPECT(11)
    if (begin(&t))
        return NULL;
    const int T = size_arg(&t, a[0]), V = size_arg(&t, a[1]), K = size_arg(&t, a[2]);
    void *ids = id_array(&t, a[3], T, &id), *dY = values(&t, a[4], (size_t)T * K, &yt);
    void *dE = values(&t, a[6], (size_t)V * K, &et), *R = values(&t, a[5], (size_t)V * K, &et);
    const float scale = float_arg(&t, a[7]);
    if (finish(&t, a[8], a[9], &ws, &size, a[10], &stream) || id < 0 || et < 0 || yt < 0)
        UNLESS_PLAIN
    CALL(embedding_bwd_call(T, V, K, id, ids, yt, dY, scale, et, R, dE, ws, size, stream));
}

/* layer_norm(rows, cols, X, gamma, beta, Y, mean, rstd, eps, stream) */
static PyObject *layer_norm(PyObject *self, PyObject *const *a, Py_ssize_t count)
{
    struct taken t;
    int status, xt = -1, wt = -1;
    void *stream;
    EXPECT(10)
    if (begin(&t))
        return NULL;
    const int M = size_arg(&t, a[0]), N = size_arg(&t, a[1]);
    const size_t n = (size_t)M * N;
    void *X = values(&t, a[2], n, &xt), *gamma = values(&t, a[3], N, &wt), *beta = values(&t, a[4], N, &wt);
    void *Y = halves(&t, a[5], n), *mean = floats(&t, a[6], M), *rstd = floats(&t, a[7], M);
    const float eps = float_arg(&t, a[8]);
    if (finish(&t, NULL, NULL, NULL, NULL, a[9], &stream) || xt < 0)
        UNLESS_PLAIN
    CALL(norm_call(M, N, xt, X, wt < 0 ? BF16 : wt, gamma, beta, eps, Y, mean, rstd, stream));
}

/* layer_norm_bwd(rows, cols, X, gamma, mean, rstd, dY, R, dX, dgamma, dbeta, workspace, workspace_bytes, stream) */
static PyObject *layer_norm_bwd(PyObject *self, PyObject *const *a, Py_ssize_t count)
{
    struct taken t;
    int status, xt = -1, wt = -1;
    void *stream, *ws;
    size_t size;
    EXPECT(14)
    if (begin(&t))
        return NULL;
    const int M = size_arg(&t, a[0]), N = size_arg(&t, a[1]);
    const size_t n = (size_t)M * N;
    void *X = values(&t, a[2], n, &xt), *gamma = values(&t, a[3], N, &wt);
    void *mean = floats(&t, a[4], M), *rstd = floats(&t, a[5], M), *dY = halves(&t, a[6], n);
    void *R = values(&t, a[7], n, &xt), *dX = values(&t, a[8], n, &xt);
    void *dgamma = values(&t, a[9], N, &wt), *dbeta = values(&t, a[10], N, &wt);
    if (finish(&t, a[11], a[12], &ws, &size, a[13], &stream) || xt < 0)
        UNLESS_PLAIN
    CALL(norm_bwd_call(M, N, xt, X, wt < 0 ? BF16 : wt, gamma, mean, rstd, dY, R, dX, dgamma, dbeta, ws, size, stream));
}

/* entropy(M, V, K, A, B, targets, loss, lse, workspace, workspace_bytes, stream) */
static PyObject *entropy(PyObject *self, PyObject *const *a, Py_ssize_t count)
{
    struct taken t;
    int status, id = -1;
    void *stream, *ws;
    size_t size;
    EXPECT(11)
    if (begin(&t))
        return NULL;
    const int M = size_arg(&t, a[0]), V = size_arg(&t, a[1]), K = size_arg(&t, a[2]);
    void *A = halves(&t, a[3], (size_t)M * K), *B = halves(&t, a[4], (size_t)V * K), *ids = id_array(&t, a[5], M, &id);
    void *loss = floats(&t, a[6], M), *lse = floats(&t, a[7], M);
    if (finish(&t, a[8], a[9], &ws, &size, a[10], &stream) || id < 0)
        UNLESS_PLAIN
    CALL(entropy_call(M, V, K, A, B, id, ids, loss, lse, ws, size, stream));
}

/* entropy_bwd(M, V, K, A, B, targets, lse, dloss, dA, dB, workspace, workspace_bytes, stream) */
static PyObject *entropy_bwd(PyObject *self, PyObject *const *a, Py_ssize_t count)
{
    struct taken t;
    int status, id = -1;
    void *stream, *ws;
    size_t size;
    EXPECT(13)
    if (begin(&t))
        return NULL;
    const int M = size_arg(&t, a[0]), V = size_arg(&t, a[1]), K = size_arg(&t, a[2]);
    const size_t mk = (size_t)M * K, vk = (size_t)V * K;
    void *A = halves(&t, a[3], mk), *B = halves(&t, a[4], vk), *ids = id_array(&t, a[5], M, &id);
    void *lse = floats(&t, a[6], M), *dloss = floats(&t, a[7], M), *dA = halves(&t, a[8], mk), *dB = halves(&t, a[9], vk);
    if (finish(&t, a[10], a[11], &ws, &size, a[12], &stream) || id < 0)
        UNLESS_PLAIN
    CALL(entropy_bwd_call(M, V, K, A, B, id, ids, lse, dloss, dA, dB, ws, size, stream));
}

/* bind_ends(parameter type, float32, int32, int64, six addresses) */
static PyObject *bind_ends(PyObject *self, PyObject *args)
{
    unsigned long long f[6];
    PyObject *o[4];
    if (!PyArg_ParseTuple(args, "OOOOKKKKKK", &o[0], &o[1], &o[2], &o[3], &f[0], &f[1], &f[2], &f[3], &f[4], &f[5]))
        return NULL;
    for (int i = 0; i < 4; ++i)
        Py_INCREF(o[i]);   /* kept for the life of the process */
    parameter_type = o[0];
    fp32 = o[1];
    int32 = o[2];
    int64 = o[3];
    embedding_call = (embedding_fn)(uintptr_t)f[0];
    embedding_bwd_call = (embedding_bwd_fn)(uintptr_t)f[1];
    norm_call = (norm_fn)(uintptr_t)f[2];
    norm_bwd_call = (norm_bwd_fn)(uintptr_t)f[3];
    entropy_call = (entropy_fn)(uintptr_t)f[4];
    entropy_bwd_call = (entropy_bwd_fn)(uintptr_t)f[5];
    Py_RETURN_NONE;
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
    {"bind_ends", bind_ends, METH_VARARGS, NULL},
    {"embedding", (PyCFunction)(void (*)(void))embedding, METH_FASTCALL, NULL},
    {"embedding_bwd", (PyCFunction)(void (*)(void))embedding_bwd, METH_FASTCALL, NULL},
    {"layer_norm", (PyCFunction)(void (*)(void))layer_norm, METH_FASTCALL, NULL},
    {"layer_norm_bwd", (PyCFunction)(void (*)(void))layer_norm_bwd, METH_FASTCALL, NULL},
    {"entropy", (PyCFunction)(void (*)(void))entropy, METH_FASTCALL, NULL},
    {"entropy_bwd", (PyCFunction)(void (*)(void))entropy_bwd, METH_FASTCALL, NULL},
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
