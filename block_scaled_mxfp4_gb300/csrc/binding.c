// Fast path of the Python binding for the calls of a decoding step, where the
// time to marshal a call's arguments in Python (3 us on the host of a GB300)
// is a good part of the call.  The module holds no arithmetic and links
// nothing: each function takes the arguments of the C entry of its name (device
// pointers as tensors, integers or None; an optional stream), calls it at the
// address that bind() was given, and raises through the package's own error.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

static PyObject *g_data_ptr;        // "data_ptr"
static PyObject *g_stream_attr;     // "cuda_stream"
static PyObject *g_pointer;         // the package's pointer conversion, for other objects
static PyObject *g_current_stream;  // -> the current stream's handle
static PyObject *g_raise;           // (status, name): raises

static void *as_pointer(PyObject *o, int *bad)
{
    if (o == Py_None || *bad)
        return NULL;
    PyObject *v;
    if (PyLong_Check(o)) {
        v = Py_NewRef(o);
    } else {
        v = PyObject_CallMethodNoArgs(o, g_data_ptr);
        if (!v && PyErr_ExceptionMatches(PyExc_AttributeError)) {
            PyErr_Clear();
            v = PyObject_CallOneArg(g_pointer, o);
        }
        if (!v) {
            *bad = 1;
            return NULL;
        }
    }
    void *p = v == Py_None ? NULL : (void *)(uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    if (!p && PyErr_Occurred())
        *bad = 1;
    return p;
}

static int64_t as_int64(PyObject *o, int *bad)
{
    if (*bad)
        return 0;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        *bad = 1;
    return v;
}

static int as_int(PyObject *o, int *bad)
{
    const int64_t v = as_int64(o, bad);
    if (!*bad && (v < INT32_MIN || v > INT32_MAX)) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
        *bad = 1;
    }
    return (int)v;
}

static size_t as_size(PyObject *o, int *bad)
{
    const int64_t v = as_int64(o, bad);
    if (!*bad && v < 0) {
        PyErr_SetString(PyExc_OverflowError, "a size is negative");
        *bad = 1;
    }
    return (size_t)v;
}

static float as_float(PyObject *o, int *bad)
{
    if (*bad)
        return 0.0f;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        *bad = 1;
    return (float)v;
}

static void *as_stream(PyObject *o, int *bad)
{
    if (*bad)
        return NULL;
    PyObject *v = !o || o == Py_None ? PyObject_CallNoArgs(g_current_stream)
                  : PyLong_Check(o)  ? Py_NewRef(o)
                                     : PyObject_GetAttr(o, g_stream_attr);
    if (!v) {
        *bad = 1;
        return NULL;
    }
    void *p = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    if (!p && PyErr_Occurred())
        *bad = 1;
    return p;
}

// The stream is the argument after the entry's own, by place or by name.
static int stream_argument(const char *name, Py_ssize_t want, PyObject *const *a, Py_ssize_t n, PyObject *kw,
                           PyObject **stream)
{
    const Py_ssize_t named = kw ? PyTuple_GET_SIZE(kw) : 0;
    if (named == 1 && n == want && PyUnicode_CompareWithASCIIString(PyTuple_GET_ITEM(kw, 0), "stream") == 0) {
        *stream = a[n];
        return 1;
    }
    if (named == 0 && (n == want || n == want + 1)) {
        *stream = n > want ? a[want] : NULL;
        return 1;
    }
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments and an optional stream", name, want);
    return 0;
}

static PyObject *finish(int status, const char *name)
{
    if (status == 0)
        return PyLong_FromLong(0);
    return PyObject_CallFunction(g_raise, "is", status, name);
}

static int (*mxfp4_moe_route_at)(void *, void *, void *, void *, void *, void *, int64_t, int, void
    *, int, int, int, int, float, void *, size_t, void *);

static PyObject *call_mxfp4_moe_route(PyObject *self, PyObject *const *a, Py_ssize_t n, PyObject *kw)
{
    (void)self;
    PyObject *so;
    int bad = 0;
    if (!stream_argument("mxfp4_moe_route", 16, a, n, kw, &so))
        return NULL;
    void *ids = as_pointer(a[0], &bad);
    void *gates = as_pointer(a[1], &bad);
    void *offsets = as_pointer(a[2], &bad);
    void *row_token = as_pointer(a[3], &bad);
    void *slot_row = as_pointer(a[4], &bad);
    void *logits = as_pointer(a[5], &bad);
    int64_t ldl = as_int64(a[6], &bad);
    int logits_type = as_int(a[7], &bad);
    void *token_mask = as_pointer(a[8], &bad);
    int T = as_int(a[9], &bad);
    int E = as_int(a[10], &bad);
    int k = as_int(a[11], &bad);
    int gate_mode = as_int(a[12], &bad);
    float gate_scale = as_float(a[13], &bad);
    void *workspace = as_pointer(a[14], &bad);
    size_t workspace_bytes = as_size(a[15], &bad);
    void *stream = as_stream(so, &bad);
    if (bad)
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = mxfp4_moe_route_at(ids, gates, offsets, row_token, slot_row, logits, ldl,
        logits_type, token_mask, T, E, k, gate_mode, gate_scale, workspace, workspace_bytes,
        stream);
    Py_END_ALLOW_THREADS
    return finish(status, "mxfp4_moe_route");
}

static int (*mxfp4_group_quantize_at)(void *, int64_t, void *, void *, int64_t, int, int, void *,
    void *, int, void *, int, int, void *);

static PyObject *call_mxfp4_group_quantize(PyObject *self, PyObject *const *a, Py_ssize_t n, PyObject *kw)
{
    (void)self;
    PyObject *so;
    int bad = 0;
    if (!stream_argument("mxfp4_group_quantize", 13, a, n, kw, &so))
        return NULL;
    void *Q = as_pointer(a[0], &bad);
    int64_t ldq = as_int64(a[1], &bad);
    void *S = as_pointer(a[2], &bad);
    void *X = as_pointer(a[3], &bad);
    int64_t ldx = as_int64(a[4], &bad);
    int T = as_int(a[5], &bad);
    int K = as_int(a[6], &bad);
    void *slot_row = as_pointer(a[7], &bad);
    void *ids = as_pointer(a[8], &bad);
    int k = as_int(a[9], &bad);
    void *offsets = as_pointer(a[10], &bad);
    int groups = as_int(a[11], &bad);
    int rows = as_int(a[12], &bad);
    void *stream = as_stream(so, &bad);
    if (bad)
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = mxfp4_group_quantize_at(Q, ldq, S, X, ldx, T, K, slot_row, ids, k, offsets, groups,
        rows, stream);
    Py_END_ALLOW_THREADS
    return finish(status, "mxfp4_group_quantize");
}

static int (*mxfp8_group_quantize_at)(void *, int64_t, void *, void *, int64_t, int, int, void *,
    void *, int, void *, int, int, int, void *);

static PyObject *call_mxfp8_group_quantize(PyObject *self, PyObject *const *a, Py_ssize_t n, PyObject *kw)
{
    (void)self;
    PyObject *so;
    int bad = 0;
    if (!stream_argument("mxfp8_group_quantize", 14, a, n, kw, &so))
        return NULL;
    void *Q = as_pointer(a[0], &bad);
    int64_t ldq = as_int64(a[1], &bad);
    void *S = as_pointer(a[2], &bad);
    void *X = as_pointer(a[3], &bad);
    int64_t ldx = as_int64(a[4], &bad);
    int T = as_int(a[5], &bad);
    int K = as_int(a[6], &bad);
    void *slot_row = as_pointer(a[7], &bad);
    void *ids = as_pointer(a[8], &bad);
    int k = as_int(a[9], &bad);
    void *offsets = as_pointer(a[10], &bad);
    int groups = as_int(a[11], &bad);
    int rows = as_int(a[12], &bad);
    int fmt = as_int(a[13], &bad);
    void *stream = as_stream(so, &bad);
    if (bad)
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = mxfp8_group_quantize_at(Q, ldq, S, X, ldx, T, K, slot_row, ids, k, offsets, groups,
        rows, fmt, stream);
    Py_END_ALLOW_THREADS
    return finish(status, "mxfp8_group_quantize");
}

static int (*mxfp4_grouped_gemm_at)(void *, int64_t, void *, int64_t, void *, void *, int64_t,
    int64_t, void *, void *, int, int, int, int, float, void *, size_t, void *);

static PyObject *call_mxfp4_grouped_gemm(PyObject *self, PyObject *const *a, Py_ssize_t n, PyObject *kw)
{
    (void)self;
    PyObject *so;
    int bad = 0;
    if (!stream_argument("mxfp4_grouped_gemm", 17, a, n, kw, &so))
        return NULL;
    void *D = as_pointer(a[0], &bad);
    int64_t ldd = as_int64(a[1], &bad);
    void *A = as_pointer(a[2], &bad);
    int64_t lda = as_int64(a[3], &bad);
    void *SA = as_pointer(a[4], &bad);
    void *B = as_pointer(a[5], &bad);
    int64_t ldb = as_int64(a[6], &bad);
    int64_t stride_b = as_int64(a[7], &bad);
    void *SB = as_pointer(a[8], &bad);
    void *offsets = as_pointer(a[9], &bad);
    int groups = as_int(a[10], &bad);
    int rows = as_int(a[11], &bad);
    int N = as_int(a[12], &bad);
    int K = as_int(a[13], &bad);
    float alpha = as_float(a[14], &bad);
    void *workspace = as_pointer(a[15], &bad);
    size_t workspace_bytes = as_size(a[16], &bad);
    void *stream = as_stream(so, &bad);
    if (bad)
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = mxfp4_grouped_gemm_at(D, ldd, A, lda, SA, B, ldb, stride_b, SB, offsets, groups,
        rows, N, K, alpha, workspace, workspace_bytes, stream);
    Py_END_ALLOW_THREADS
    return finish(status, "mxfp4_grouped_gemm");
}

static int (*mxfp8_grouped_gemm_at)(void *, int64_t, void *, int64_t, void *, void *, int64_t,
    int64_t, void *, void *, int, int, int, int, int, int, float, void *, size_t, void *);

static PyObject *call_mxfp8_grouped_gemm(PyObject *self, PyObject *const *a, Py_ssize_t n, PyObject *kw)
{
    (void)self;
    PyObject *so;
    int bad = 0;
    if (!stream_argument("mxfp8_grouped_gemm", 19, a, n, kw, &so))
        return NULL;
    void *D = as_pointer(a[0], &bad);
    int64_t ldd = as_int64(a[1], &bad);
    void *A = as_pointer(a[2], &bad);
    int64_t lda = as_int64(a[3], &bad);
    void *SA = as_pointer(a[4], &bad);
    void *B = as_pointer(a[5], &bad);
    int64_t ldb = as_int64(a[6], &bad);
    int64_t stride_b = as_int64(a[7], &bad);
    void *SB = as_pointer(a[8], &bad);
    void *offsets = as_pointer(a[9], &bad);
    int groups = as_int(a[10], &bad);
    int rows = as_int(a[11], &bad);
    int N = as_int(a[12], &bad);
    int K = as_int(a[13], &bad);
    int fmt_a = as_int(a[14], &bad);
    int fmt_b = as_int(a[15], &bad);
    float alpha = as_float(a[16], &bad);
    void *workspace = as_pointer(a[17], &bad);
    size_t workspace_bytes = as_size(a[18], &bad);
    void *stream = as_stream(so, &bad);
    if (bad)
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = mxfp8_grouped_gemm_at(D, ldd, A, lda, SA, B, ldb, stride_b, SB, offsets, groups,
        rows, N, K, fmt_a, fmt_b, alpha, workspace, workspace_bytes, stream);
    Py_END_ALLOW_THREADS
    return finish(status, "mxfp8_grouped_gemm");
}

static int (*mxfp4_grouped_swiglu_at)(void *, int64_t, void *, void *, int64_t, void *, void *,
    int64_t, int64_t, void *, void *, int, int, int, int, float, void *, size_t, void *);

static PyObject *call_mxfp4_grouped_swiglu(PyObject *self, PyObject *const *a, Py_ssize_t n, PyObject *kw)
{
    (void)self;
    PyObject *so;
    int bad = 0;
    if (!stream_argument("mxfp4_grouped_swiglu", 18, a, n, kw, &so))
        return NULL;
    void *H = as_pointer(a[0], &bad);
    int64_t ldh = as_int64(a[1], &bad);
    void *SH = as_pointer(a[2], &bad);
    void *A = as_pointer(a[3], &bad);
    int64_t lda = as_int64(a[4], &bad);
    void *SA = as_pointer(a[5], &bad);
    void *B = as_pointer(a[6], &bad);
    int64_t ldb = as_int64(a[7], &bad);
    int64_t stride_b = as_int64(a[8], &bad);
    void *SB = as_pointer(a[9], &bad);
    void *offsets = as_pointer(a[10], &bad);
    int groups = as_int(a[11], &bad);
    int rows = as_int(a[12], &bad);
    int F = as_int(a[13], &bad);
    int K = as_int(a[14], &bad);
    float alpha = as_float(a[15], &bad);
    void *workspace = as_pointer(a[16], &bad);
    size_t workspace_bytes = as_size(a[17], &bad);
    void *stream = as_stream(so, &bad);
    if (bad)
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = mxfp4_grouped_swiglu_at(H, ldh, SH, A, lda, SA, B, ldb, stride_b, SB, offsets,
        groups, rows, F, K, alpha, workspace, workspace_bytes, stream);
    Py_END_ALLOW_THREADS
    return finish(status, "mxfp4_grouped_swiglu");
}

static int (*mxfp8_grouped_swiglu_at)(void *, int64_t, void *, void *, int64_t, void *, void *,
    int64_t, int64_t, void *, void *, int, int, int, int, int, int, int, float, void *, size_t, void *);

static PyObject *call_mxfp8_grouped_swiglu(PyObject *self, PyObject *const *a, Py_ssize_t n, PyObject *kw)
{
    (void)self;
    PyObject *so;
    int bad = 0;
    if (!stream_argument("mxfp8_grouped_swiglu", 21, a, n, kw, &so))
        return NULL;
    void *H = as_pointer(a[0], &bad);
    int64_t ldh = as_int64(a[1], &bad);
    void *SH = as_pointer(a[2], &bad);
    void *A = as_pointer(a[3], &bad);
    int64_t lda = as_int64(a[4], &bad);
    void *SA = as_pointer(a[5], &bad);
    void *B = as_pointer(a[6], &bad);
    int64_t ldb = as_int64(a[7], &bad);
    int64_t stride_b = as_int64(a[8], &bad);
    void *SB = as_pointer(a[9], &bad);
    void *offsets = as_pointer(a[10], &bad);
    int groups = as_int(a[11], &bad);
    int rows = as_int(a[12], &bad);
    int F = as_int(a[13], &bad);
    int K = as_int(a[14], &bad);
    int fmt_a = as_int(a[15], &bad);
    int fmt_b = as_int(a[16], &bad);
    int fmt_h = as_int(a[17], &bad);
    float alpha = as_float(a[18], &bad);
    void *workspace = as_pointer(a[19], &bad);
    size_t workspace_bytes = as_size(a[20], &bad);
    void *stream = as_stream(so, &bad);
    if (bad)
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = mxfp8_grouped_swiglu_at(H, ldh, SH, A, lda, SA, B, ldb, stride_b, SB, offsets,
        groups, rows, F, K, fmt_a, fmt_b, fmt_h, alpha, workspace, workspace_bytes, stream);
    Py_END_ALLOW_THREADS
    return finish(status, "mxfp8_grouped_swiglu");
}

static int (*mxfp4_moe_combine_at)(void *, int64_t, void *, int64_t, void *, int64_t, int, void *,
    void *, int, void *, int64_t, void *, void *, float, float, float, int, int, void *);

static PyObject *call_mxfp4_moe_combine(PyObject *self, PyObject *const *a, Py_ssize_t n, PyObject *kw)
{
    (void)self;
    PyObject *so;
    int bad = 0;
    if (!stream_argument("mxfp4_moe_combine", 19, a, n, kw, &so))
        return NULL;
    void *H = as_pointer(a[0], &bad);
    int64_t ldh = as_int64(a[1], &bad);
    void *Nrm = as_pointer(a[2], &bad);
    int64_t ldn = as_int64(a[3], &bad);
    void *Y = as_pointer(a[4], &bad);
    int64_t ldy = as_int64(a[5], &bad);
    int rows = as_int(a[6], &bad);
    void *slot_row = as_pointer(a[7], &bad);
    void *gates = as_pointer(a[8], &bad);
    int k = as_int(a[9], &bad);
    void *resid = as_pointer(a[10], &bad);
    int64_t ldr = as_int64(a[11], &bad);
    void *w_post = as_pointer(a[12], &bad);
    void *w_pre = as_pointer(a[13], &bad);
    float res_scale = as_float(a[14], &bad);
    float out_scale = as_float(a[15], &bad);
    float eps = as_float(a[16], &bad);
    int T = as_int(a[17], &bad);
    int N = as_int(a[18], &bad);
    void *stream = as_stream(so, &bad);
    if (bad)
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = mxfp4_moe_combine_at(H, ldh, Nrm, ldn, Y, ldy, rows, slot_row, gates, k, resid,
        ldr, w_post, w_pre, res_scale, out_scale, eps, T, N, stream);
    Py_END_ALLOW_THREADS
    return finish(status, "mxfp4_moe_combine");
}

static int (*mxfp4_moe_ffn_at)(void *, int64_t, void *, int64_t, void *, int64_t, void *, void *,
    void *, void *, int, int, int, int, int, void *, int64_t, void *, void *, int64_t, void *, void *,
    int64_t, void *, void *, float, float, float, void *, size_t, void *);

static PyObject *call_mxfp4_moe_ffn(PyObject *self, PyObject *const *a, Py_ssize_t n, PyObject *kw)
{
    (void)self;
    PyObject *so;
    int bad = 0;
    if (!stream_argument("mxfp4_moe_ffn", 30, a, n, kw, &so))
        return NULL;
    void *H = as_pointer(a[0], &bad);
    int64_t ldh = as_int64(a[1], &bad);
    void *Nrm = as_pointer(a[2], &bad);
    int64_t ldn = as_int64(a[3], &bad);
    void *X = as_pointer(a[4], &bad);
    int64_t ldx = as_int64(a[5], &bad);
    void *ids = as_pointer(a[6], &bad);
    void *gates = as_pointer(a[7], &bad);
    void *offsets = as_pointer(a[8], &bad);
    void *slot_row = as_pointer(a[9], &bad);
    int T = as_int(a[10], &bad);
    int E = as_int(a[11], &bad);
    int k = as_int(a[12], &bad);
    int K = as_int(a[13], &bad);
    int F = as_int(a[14], &bad);
    void *B1 = as_pointer(a[15], &bad);
    int64_t ldb1 = as_int64(a[16], &bad);
    void *SB1 = as_pointer(a[17], &bad);
    void *B2 = as_pointer(a[18], &bad);
    int64_t ldb2 = as_int64(a[19], &bad);
    void *SB2 = as_pointer(a[20], &bad);
    void *resid = as_pointer(a[21], &bad);
    int64_t ldr = as_int64(a[22], &bad);
    void *w_post = as_pointer(a[23], &bad);
    void *w_pre = as_pointer(a[24], &bad);
    float res_scale = as_float(a[25], &bad);
    float out_scale = as_float(a[26], &bad);
    float eps = as_float(a[27], &bad);
    void *workspace = as_pointer(a[28], &bad);
    size_t workspace_bytes = as_size(a[29], &bad);
    void *stream = as_stream(so, &bad);
    if (bad)
        return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = mxfp4_moe_ffn_at(H, ldh, Nrm, ldn, X, ldx, ids, gates, offsets, slot_row, T, E, k,
        K, F, B1, ldb1, SB1, B2, ldb2, SB2, resid, ldr, w_post, w_pre, res_scale, out_scale, eps,
        workspace, workspace_bytes, stream);
    Py_END_ALLOW_THREADS
    return finish(status, "mxfp4_moe_ffn");
}

static struct {
    const char *name;
    void **at;
} g_entries[] = {
    {"mxfp4_moe_route", (void **)&mxfp4_moe_route_at},
    {"mxfp4_group_quantize", (void **)&mxfp4_group_quantize_at},
    {"mxfp8_group_quantize", (void **)&mxfp8_group_quantize_at},
    {"mxfp4_grouped_gemm", (void **)&mxfp4_grouped_gemm_at},
    {"mxfp8_grouped_gemm", (void **)&mxfp8_grouped_gemm_at},
    {"mxfp4_grouped_swiglu", (void **)&mxfp4_grouped_swiglu_at},
    {"mxfp8_grouped_swiglu", (void **)&mxfp8_grouped_swiglu_at},
    {"mxfp4_moe_combine", (void **)&mxfp4_moe_combine_at},
    {"mxfp4_moe_ffn", (void **)&mxfp4_moe_ffn_at},
};

// bind(addresses: dict, pointer, current_stream, raise_error)
static PyObject *bind(PyObject *self, PyObject *args)
{
    (void)self;
    PyObject *addresses, *pointer, *stream, *raise;
    if (!PyArg_ParseTuple(args, "O!OOO", &PyDict_Type, &addresses, &pointer, &stream, &raise))
        return NULL;
    for (size_t i = 0; i < sizeof(g_entries) / sizeof(g_entries[0]); ++i) {
        PyObject *v = PyDict_GetItemString(addresses, g_entries[i].name);
        if (!v) {
            PyErr_SetString(PyExc_KeyError, g_entries[i].name);
            return NULL;
        }
        *g_entries[i].at = PyLong_AsVoidPtr(v);
        if (!*g_entries[i].at)
            return NULL;
    }
    Py_XSETREF(g_pointer, Py_NewRef(pointer));
    Py_XSETREF(g_current_stream, Py_NewRef(stream));
    Py_XSETREF(g_raise, Py_NewRef(raise));
    Py_RETURN_NONE;
}

#define METHOD(NAME) {#NAME, (PyCFunction)(void (*)(void))call_##NAME, METH_FASTCALL | METH_KEYWORDS, NULL}
static PyMethodDef g_methods[] = {
    METHOD(mxfp4_moe_route),
    METHOD(mxfp4_group_quantize),
    METHOD(mxfp8_group_quantize),
    METHOD(mxfp4_grouped_gemm),
    METHOD(mxfp8_grouped_gemm),
    METHOD(mxfp4_grouped_swiglu),
    METHOD(mxfp8_grouped_swiglu),
    METHOD(mxfp4_moe_combine),
    METHOD(mxfp4_moe_ffn),
    {"bind", bind, METH_VARARGS, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_entry", NULL, -1, g_methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__entry(void)
{
    g_data_ptr = PyUnicode_InternFromString("data_ptr");
    g_stream_attr = PyUnicode_InternFromString("cuda_stream");
    if (!g_data_ptr || !g_stream_attr)
        return NULL;
    return PyModule_Create(&g_module);
}
