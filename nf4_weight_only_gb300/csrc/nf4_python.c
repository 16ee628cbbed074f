/*
 * The Python binding's short way into libnf4.so for the calls that a decode loop makes many times a token.
 *
 * A call through ctypes with its tensors checked in Python costs 3 to 5 microseconds of the host's time beside
 * the launch itself (2 us), which is what the smallest calls take on the GPU; here the same checks and the call
 * are compiled.  Every function returns the status as an int, or None if a tensor is not what the call
 * wants (type, shape, contiguity, device): the Python wrapper then takes its own checks, which say what is
 * wrong.  Nothing is kept from one call to the next but the types and functions given to init().
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdint.h>

typedef struct nf4_kv_cache nf4_kv_cache;
typedef void* cudaStream;

static int (*p_append)(const nf4_kv_cache*, const void*, const void*, const void*, int64_t, cudaStream);
static int (*p_read)(const nf4_kv_cache*, const void*, int64_t, void*, void*, cudaStream);
static int (*p_attention)(const nf4_kv_cache*, const void*, const void*, int64_t, const void*, int64_t, int64_t, float,
                          int64_t, void*, void*, int64_t, cudaStream);
static int (*p_rope)(const void*, int64_t, const void*, int64_t, int64_t, int64_t, const void*, int, const int32_t*,
                     const void*, int64_t, int, float, void*, void*, cudaStream);
static int (*p_rmsnorm)(const void*, const void*, const void*, int64_t, int64_t, float, void*, void*, void*, void*,
                        cudaStream);

enum { BF16, FP8, F32, I32, I64, U8, TYPES };
static PyObject* g_types[TYPES];
static PyObject *g_raw_stream, *g_current_device;
static PyObject *s_dtype, *s_shape, *s_is_contiguous, *s_is_cuda, *s_data_ptr, *s_cuda_stream;

static int is_true(PyObject* v) { /* steals v */
    const int yes = v == Py_True;
    if (!v) PyErr_Clear();
    Py_XDECREF(v);
    return yes;
}

/* Whether t is a contiguous CUDA tensor of that type and shape; a negative dim takes the tensor's.  *at: its address. */
static int tensor(PyObject* t, int type, int nd, int64_t* dims, void** at) {
    PyObject* v = PyObject_GetAttr(t, s_dtype);
    int ok = v == g_types[type];
    if (!v) PyErr_Clear();
    Py_XDECREF(v);
    if (!ok) return 0;
    v = PyObject_GetAttr(t, s_shape);
    ok = v && PyTuple_Check(v) && PyTuple_GET_SIZE(v) == nd;
    for (int i = 0; ok && i < nd; i++) {
        const int64_t d = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
        if (dims[i] < 0) dims[i] = d;
        ok = d >= 0 && dims[i] == d;
    }
    if (PyErr_Occurred()) PyErr_Clear();
    Py_XDECREF(v);
    if (!ok || !is_true(PyObject_CallMethodNoArgs(t, s_is_contiguous)) || !is_true(PyObject_GetAttr(t, s_is_cuda)))
        return 0;
    v = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!v) {
        PyErr_Clear();
        return 0;
    }
    *at = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return 1;
}

static int maybe(PyObject* t, int type, int nd, int64_t* dims, void** at) {
    *at = NULL;
    return t == Py_None || tensor(t, type, nd, dims, at);
}

/* The handle of `stream` (a torch stream or an int), or of the current device's current stream; 0: an exception. */
static int stream_of(PyObject* stream, cudaStream* at) {
    PyObject* v;
    if (stream == Py_None) {
        PyObject* device = PyObject_CallNoArgs(g_current_device);
        if (!device) return 0;
        v = PyObject_CallOneArg(g_raw_stream, device);
        Py_DECREF(device);
    } else if (PyLong_Check(stream)) {
        v = Py_NewRef(stream);
    } else {
        v = PyObject_GetAttr(stream, s_cuda_stream);
    }
    if (!v) return 0;
    *at = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return !PyErr_Occurred();
}

#define CALL(expr)                 \
    int status;                    \
    Py_BEGIN_ALLOW_THREADS         \
    status = (expr);               \
    Py_END_ALLOW_THREADS           \
    return PyLong_FromLong(status)

#define ARGS(n)                                                            \
    if (nargs != (n)) {                                                    \
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");    \
        return NULL;                                                       \
    }

/* append(cache address, kv_heads, head_dim, k, v, slots, stream) */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
    (void)self;
    ARGS(7)
    int64_t t[1] = {-1};
    void *k, *v, *slots;
    cudaStream stream;
    if (!tensor(a[5], I64, 1, t, &slots)) Py_RETURN_NONE;
    int64_t shape[3] = {t[0], PyLong_AsLongLong(a[1]), PyLong_AsLongLong(a[2])};
    if (!tensor(a[3], BF16, 3, shape, &k) || !tensor(a[4], BF16, 3, shape, &v)) Py_RETURN_NONE;
    const nf4_kv_cache* cache = PyLong_AsVoidPtr(a[0]);
    if (!stream_of(a[6], &stream) || PyErr_Occurred()) return NULL;
    CALL(p_append(cache, k, v, slots, t[0], stream));
}

/* read(cache address, kv_heads, head_dim, slots, k, v, stream) */
static PyObject* read_(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
    (void)self;
    ARGS(7)
    int64_t t[1] = {-1};
    void *k, *v, *slots;
    cudaStream stream;
    if (!tensor(a[3], I64, 1, t, &slots)) Py_RETURN_NONE;
    int64_t shape[3] = {t[0], PyLong_AsLongLong(a[1]), PyLong_AsLongLong(a[2])};
    if (!maybe(a[4], BF16, 3, shape, &k) || !maybe(a[5], BF16, 3, shape, &v)) Py_RETURN_NONE;
    const nf4_kv_cache* cache = PyLong_AsVoidPtr(a[0]);
    if (!stream_of(a[6], &stream) || PyErr_Occurred()) return NULL;
    CALL(p_read(cache, slots, t[0], k, v, stream));
}

/* attention(cache address, head_dim, q, page_table, lengths, out, workspace, scale or None, window, stream) */
static PyObject* attention(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
    (void)self;
    ARGS(10)
    const int64_t d = PyLong_AsLongLong(a[1]);
    int64_t shape[3] = {-1, -1, d}, table[2], size[1] = {-1};
    void *q, *pages, *lengths, *out, *workspace;
    cudaStream stream;
    if (!tensor(a[2], BF16, 3, shape, &q)) Py_RETURN_NONE;
    table[0] = shape[0], table[1] = -1;
    if (!tensor(a[3], I32, 2, table, &pages) || !tensor(a[4], I32, 1, shape, &lengths) ||
        !tensor(a[5], BF16, 3, shape, &out) || !tensor(a[6], U8, 1, size, &workspace))
        Py_RETURN_NONE;
    const double scale = a[7] == Py_None ? pow((double)d, -0.5) : PyFloat_AsDouble(a[7]);
    const int64_t window = PyLong_AsLongLong(a[8]);
    const nf4_kv_cache* cache = PyLong_AsVoidPtr(a[0]);
    if (PyErr_Occurred() || !stream_of(a[9], &stream)) return NULL;
    CALL(p_attention(cache, q, pages, table[1], lengths, shape[0], shape[1], (float)scale, window, out, workspace, size[0],
                     stream));
}

/* rope(q, k, positions, inv_freq, q_out, k_out, sections or None, interleaved, magnitude, stream) */
static PyObject* rope(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
    (void)self;
    ARGS(10)
    int64_t q_shape[3] = {-1, -1, -1}, k_shape[3] = {-1, -1, -1}, at[2] = {-1, -1}, pairs[1] = {-1};
    void *q, *k, *qo = NULL, *ko = NULL, *positions, *inv_freq;
    int32_t counts[4];
    cudaStream stream;
    if (!maybe(a[0], BF16, 3, q_shape, &q)) Py_RETURN_NONE;
    if (a[0] != Py_None) k_shape[0] = q_shape[0], k_shape[2] = q_shape[2];
    if (!maybe(a[1], BF16, 3, k_shape, &k) || (a[0] == Py_None && a[1] == Py_None)) Py_RETURN_NONE;
    const int64_t *any = a[0] != Py_None ? q_shape : k_shape, t = any[0], d = any[2];
    if ((a[0] != Py_None && !tensor(a[4], BF16, 3, q_shape, &qo)) || (a[1] != Py_None && !tensor(a[5], BF16, 3, k_shape, &ko)))
        Py_RETURN_NONE;
    at[1] = t;
    if (!tensor(a[2], I32, 2, at, &positions) || !tensor(a[3], F32, 1, pairs, &inv_freq)) Py_RETURN_NONE;
    const int64_t axes = at[0];
    if (axes < 1 || axes > 4) Py_RETURN_NONE;
    if (a[6] == Py_None) {
        if (axes != 1 || pairs[0] > INT32_MAX) Py_RETURN_NONE;
        counts[0] = (int32_t)pairs[0];
    } else {
        PyObject* seq = PySequence_Fast(a[6], "sections: want a sequence");
        if (!seq) return NULL;
        int ok = PySequence_Fast_GET_SIZE(seq) == axes;
        for (int64_t i = 0; ok && i < axes; i++) {
            const int64_t n = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
            ok = n >= INT32_MIN && n <= INT32_MAX;
            counts[i] = (int32_t)n;
        }
        Py_DECREF(seq);
        if (PyErr_Occurred()) return NULL;
        if (!ok) Py_RETURN_NONE;
    }
    const int interleaved = PyObject_IsTrue(a[7]);
    const double magnitude = PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred() || !stream_of(a[9], &stream)) return NULL;
    const int64_t hq = a[0] != Py_None ? q_shape[1] : 0, hk = a[1] != Py_None ? k_shape[1] : 0;
    CALL(p_rope(q, hq, k, hk, t, d, positions, (int)axes, counts, inv_freq, 2 * pairs[0], interleaved, (float)magnitude, qo,
                ko, stream));
}

/* rmsnorm(x, weight, eps, residual, residual_out, y, y8, y8_scales, stream) */
static PyObject* rmsnorm(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
    (void)self;
    ARGS(9)
    int64_t shape[2] = {-1, -1};
    void *x, *w, *r, *ro, *y, *y8, *scales;
    cudaStream stream;
    if (!tensor(a[0], BF16, 2, shape, &x) || !tensor(a[1], BF16, 1, shape + 1, &w) || !maybe(a[3], BF16, 2, shape, &r) ||
        !maybe(a[4], BF16, 2, shape, &ro) || !maybe(a[5], BF16, 2, shape, &y) || !maybe(a[6], FP8, 2, shape, &y8) ||
        !maybe(a[7], F32, 1, shape, &scales))
        Py_RETURN_NONE;
    const double eps = PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred() || !stream_of(a[8], &stream)) return NULL;
    CALL(p_rmsnorm(x, r, w, shape[0], shape[1], (float)eps, ro, y, y8, scales, stream));
}

/* init(addresses of the five functions, the six types, raw-stream and current-device functions) */
static PyObject* init(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
    (void)self;
    ARGS(5 + TYPES + 2)
    void* f[5];
    for (int i = 0; i < 5; i++) f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return NULL;
    p_append = f[0], p_read = f[1], p_attention = f[2], p_rope = f[3], p_rmsnorm = f[4];
    for (int i = 0; i < TYPES; i++) Py_XSETREF(g_types[i], Py_NewRef(a[5 + i]));
    Py_XSETREF(g_raw_stream, Py_NewRef(a[5 + TYPES]));
    Py_XSETREF(g_current_device, Py_NewRef(a[6 + TYPES]));
    Py_RETURN_NONE;
}

#define METHOD(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD("init", init), METHOD("append", append), METHOD("read", read_),
                                METHOD("attention", attention), METHOD("rope", rope), METHOD("rmsnorm", rmsnorm),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "nf4_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_nf4_calls(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    return PyModule_Create(&module);
}
