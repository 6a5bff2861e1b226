// Fast path of the Python binding for the calls of a decoding step, where the
// time to marshal a call's arguments in Python (3 us on the host of a GB300)
// is a good part of the call.  The module holds no arithmetic and links
// nothing: each function takes the arguments of the C entry of its name (device
// pointers as tensors, integers or None; an optional stream), by place or by
// name like the package's Python function that it stands in for, calls the entry
// at the address that bind() was given, and raises through the package's own
// error.  An entry is one list of its arguments' kinds and names.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

static PyObject *g_data_ptr;        // "data_ptr"
static PyObject *g_stream_attr;     // "cuda_stream"
static PyObject *g_pointer;         // the package's pointer conversion, for other objects
static PyObject *g_current_stream;  // -> the current stream's handle
static PyObject *g_raise;           // (status, name): raises

typedef void *ptr;
typedef int64_t i64;
typedef int i32;
typedef float f32;
typedef size_t size;

static ptr as_ptr(PyObject *o, int *bad)
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

static i64 as_i64(PyObject *o, int *bad)
{
    if (*bad)
        return 0;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        *bad = 1;
    return v;
}

static i32 as_i32(PyObject *o, int *bad)
{
    const i64 v = as_i64(o, bad);
    if (!*bad && (v < INT32_MIN || v > INT32_MAX)) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit a C int");
        *bad = 1;
    }
    return (int)v;
}

static size as_size(PyObject *o, int *bad)
{
    const i64 v = as_i64(o, bad);
    if (!*bad && v < 0) {
        PyErr_SetString(PyExc_OverflowError, "a size is negative");
        *bad = 1;
    }
    return (size)v;
}

static f32 as_f32(PyObject *o, int *bad)
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

// The arguments in the order of `names`, whose last is the optional stream: `a`
// itself where all are given by place, else `v` (NULL for no stream), else NULL
// with an error.
static PyObject *const *arrange(const char *entry, const char *const *names, Py_ssize_t count, PyObject *const *a,
                                Py_ssize_t n, PyObject *kw, PyObject **v)
{
    const Py_ssize_t named = kw ? PyTuple_GET_SIZE(kw) : 0;
    if (named == 0 && (n == count - 1 || n == count))
        return a;
    if (n > count) {
        PyErr_Format(PyExc_TypeError, "%s() takes at most %zd arguments (%zd given)", entry, count, n);
        return NULL;
    }
    for (Py_ssize_t i = 0; i < count; ++i)
        v[i] = i < n ? a[i] : NULL;
    for (Py_ssize_t j = 0; j < named; ++j) {
        PyObject *name = PyTuple_GET_ITEM(kw, j);
        Py_ssize_t i = count - 1;                          // the stream first: the usual one
        while (i >= 0 && PyUnicode_CompareWithASCIIString(name, names[i]) != 0)
            --i;
        if (i < 0 || v[i]) {
            PyErr_Format(PyExc_TypeError, i < 0 ? "%s() got an unexpected keyword argument '%U'"
                                                : "%s() got multiple values for argument '%U'", entry, name);
            return NULL;
        }
        v[i] = a[n + j];
    }
    for (Py_ssize_t i = 0; i < count - 1; ++i)
        if (!v[i]) {
            PyErr_Format(PyExc_TypeError, "%s() missing required argument '%s'", entry, names[i]);
            return NULL;
        }
    return v;
}

static PyObject *finish(int status, const char *name)
{
    if (status == 0)
        return PyLong_FromLong(0);
    return PyObject_CallFunction(g_raise, "is", status, name);
}

#define ARGS_mxfp4_moe_route(ARG) \
    ARG(ptr, ids) ARG(ptr, gates) ARG(ptr, offsets) ARG(ptr, row_token) ARG(ptr, slot_row) ARG(ptr, logits) ARG(i64, ldl) \
    ARG(i32, logits_type) ARG(ptr, token_mask) ARG(i32, T) ARG(i32, E) ARG(i32, k) ARG(i32, gate_mode) ARG(f32, gate_scale) \
    ARG(ptr, workspace) ARG(size, workspace_bytes)
#define DOC_mxfp4_moe_route \
    "The k largest logits per token, their gates, and the rows' grouping by expert."

#define ARGS_mxfp4_group_quantize(ARG) \
    ARG(ptr, Q) ARG(i64, ldq) ARG(ptr, S) ARG(ptr, X) ARG(i64, ldx) ARG(i32, T) ARG(i32, K) ARG(ptr, slot_row) ARG(ptr, ids) \
    ARG(i32, k) ARG(ptr, offsets) ARG(i32, groups) ARG(i32, rows)
#define DOC_mxfp4_group_quantize \
    "bf16 rows -> packed E2M1 rows at their places in the grouping, grouped scales."

#define ARGS_mxfp8_group_quantize(ARG) \
    ARG(ptr, Q) ARG(i64, ldq) ARG(ptr, S) ARG(ptr, X) ARG(i64, ldx) ARG(i32, T) ARG(i32, K) ARG(ptr, slot_row) ARG(ptr, ids) \
    ARG(i32, k) ARG(ptr, offsets) ARG(i32, groups) ARG(i32, rows) ARG(i32, fmt)
#define DOC_mxfp8_group_quantize \
    "mxfp4_group_quantize into E4M3 / E5M2 codes, one per byte."

#define ARGS_mxfp4_grouped_gemm(ARG) \
    ARG(ptr, D) ARG(i64, ldd) ARG(ptr, A) ARG(i64, lda) ARG(ptr, SA) ARG(ptr, B) ARG(i64, ldb) ARG(i64, stride_b) ARG(ptr, SB) \
    ARG(ptr, offsets) ARG(i32, groups) ARG(i32, rows) ARG(i32, N) ARG(i32, K) ARG(f32, alpha) ARG(ptr, workspace) \
    ARG(size, workspace_bytes)
#define DOC_mxfp4_grouped_gemm \
    "D[r] = alpha * A[r] . B[e]^T for every row r of group e (bf16 out)."

#define ARGS_mxfp8_grouped_gemm(ARG) \
    ARG(ptr, D) ARG(i64, ldd) ARG(ptr, A) ARG(i64, lda) ARG(ptr, SA) ARG(ptr, B) ARG(i64, ldb) ARG(i64, stride_b) ARG(ptr, SB) \
    ARG(ptr, offsets) ARG(i32, groups) ARG(i32, rows) ARG(i32, N) ARG(i32, K) ARG(i32, fmt_a) ARG(i32, fmt_b) ARG(f32, alpha) \
    ARG(ptr, workspace) ARG(size, workspace_bytes)
#define DOC_mxfp8_grouped_gemm \
    "mxfp4_grouped_gemm on the byte formats of mxfp8_gemm."

#define ARGS_mxfp4_grouped_swiglu(ARG) \
    ARG(ptr, H) ARG(i64, ldh) ARG(ptr, SH) ARG(ptr, A) ARG(i64, lda) ARG(ptr, SA) ARG(ptr, B) ARG(i64, ldb) ARG(i64, stride_b) \
    ARG(ptr, SB) ARG(ptr, offsets) ARG(i32, groups) ARG(i32, rows) ARG(i32, F) ARG(i32, K) ARG(f32, alpha) ARG(ptr, workspace) \
    ARG(size, workspace_bytes)
#define DOC_mxfp4_grouped_swiglu \
    "H = quantise(silu(A . Bgate^T) * (A . Bup^T)) per group, packed E2M1."

#define ARGS_mxfp8_grouped_swiglu(ARG) \
    ARG(ptr, H) ARG(i64, ldh) ARG(ptr, SH) ARG(ptr, A) ARG(i64, lda) ARG(ptr, SA) ARG(ptr, B) ARG(i64, ldb) ARG(i64, stride_b) \
    ARG(ptr, SB) ARG(ptr, offsets) ARG(i32, groups) ARG(i32, rows) ARG(i32, F) ARG(i32, K) ARG(i32, fmt_a) ARG(i32, fmt_b) \
    ARG(i32, fmt_h) ARG(f32, alpha) ARG(ptr, workspace) ARG(size, workspace_bytes)
#define DOC_mxfp8_grouped_swiglu \
    "mxfp4_grouped_swiglu on byte formats, into E4M3 / E5M2 codes."

#define ARGS_mxfp4_moe_combine(ARG) \
    ARG(ptr, H) ARG(i64, ldh) ARG(ptr, Nrm) ARG(i64, ldn) ARG(ptr, Y) ARG(i64, ldy) ARG(i32, rows) ARG(ptr, slot_row) \
    ARG(ptr, gates) ARG(i32, k) ARG(ptr, resid) ARG(i64, ldr) ARG(ptr, w_post) ARG(ptr, w_pre) ARG(f32, res_scale) \
    ARG(f32, out_scale) ARG(f32, eps) ARG(i32, T) ARG(i32, N)
#define DOC_mxfp4_moe_combine \
    "Gated sum of a token's rows, its norm, the residual stream and the next block's norm."

#define ARGS_mxfp4_moe_ffn(ARG) \
    ARG(ptr, H) ARG(i64, ldh) ARG(ptr, Nrm) ARG(i64, ldn) ARG(ptr, X) ARG(i64, ldx) ARG(ptr, ids) ARG(ptr, gates) \
    ARG(ptr, offsets) ARG(ptr, slot_row) ARG(i32, T) ARG(i32, E) ARG(i32, k) ARG(i32, K) ARG(i32, F) ARG(ptr, B1) ARG(i64, ldb1) \
    ARG(ptr, SB1) ARG(ptr, B2) ARG(i64, ldb2) ARG(ptr, SB2) ARG(ptr, resid) ARG(i64, ldr) ARG(ptr, w_post) ARG(ptr, w_pre) \
    ARG(f32, res_scale) ARG(f32, out_scale) ARG(f32, eps) ARG(ptr, workspace) ARG(size, workspace_bytes)
#define DOC_mxfp4_moe_ffn \
    "A routed feed-forward block on MXFP4 weights: quantise, both products, join."

#define KIND_OF(kind, name) kind,
#define NAME_OF(kind, name) #name,
#define SHOWN(kind, name) #name ", "
#define CONVERT(kind, name) kind name = as_##kind(v_[at_++], &bad_);
#define PASS(kind, name) name,

#define DEFINE(NAME)                                                                                              \
    static int (*NAME##_at)(ARGS_##NAME(KIND_OF) void *);                                                          \
    static PyObject *call_##NAME(PyObject *self_, PyObject *const *a_, Py_ssize_t n_, PyObject *kw_)               \
    {                                                                                                              \
        (void)self_;                                                                                               \
        static const char *const names[] = {ARGS_##NAME(NAME_OF) "stream"};                                        \
        enum { COUNT = sizeof(names) / sizeof(names[0]) };                                                         \
        PyObject *arranged_[COUNT];                                                                                \
        PyObject *const *v_ = arrange(#NAME, names, COUNT, a_, n_, kw_, arranged_);                                \
        int bad_ = 0, at_ = 0;                                                                                     \
        if (!v_)                                                                                                   \
            return NULL;                                                                                           \
        ARGS_##NAME(CONVERT)                                                                                       \
        void *stream_ = as_stream(v_ == a_ && n_ < COUNT ? NULL : v_[at_], &bad_);                                 \
        if (bad_)                                                                                                  \
            return NULL;                                                                                           \
        int status_;                                                                                               \
        Py_BEGIN_ALLOW_THREADS                                                                                     \
        status_ = NAME##_at(ARGS_##NAME(PASS) stream_);                                                            \
        Py_END_ALLOW_THREADS                                                                                       \
        return finish(status_, #NAME);                                                                             \
    }

#define ENTRIES(DO)                                                                                               \
    DO(mxfp4_moe_route)                                                                                            \
    DO(mxfp4_group_quantize)                                                                                       \
    DO(mxfp8_group_quantize)                                                                                       \
    DO(mxfp4_grouped_gemm)                                                                                         \
    DO(mxfp8_grouped_gemm)                                                                                         \
    DO(mxfp4_grouped_swiglu)                                                                                       \
    DO(mxfp8_grouped_swiglu)                                                                                       \
    DO(mxfp4_moe_combine)                                                                                          \
    DO(mxfp4_moe_ffn)

ENTRIES(DEFINE)

#define ADDRESS(NAME) {#NAME, (void **)&NAME##_at},
static struct {
    const char *name;
    void **at;
} g_entries[] = {ENTRIES(ADDRESS)};

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

#define METHOD(NAME)                                                              \
    {#NAME, (PyCFunction)(void (*)(void))call_##NAME, METH_FASTCALL | METH_KEYWORDS, \
     #NAME "($module, " ARGS_##NAME(SHOWN) "stream=None)\n--\n\n" DOC_##NAME},
static PyMethodDef g_methods[] = {
    ENTRIES(METHOD){"bind", bind, METH_VARARGS, NULL},
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
