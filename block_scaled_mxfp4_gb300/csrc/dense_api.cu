// C ABI of the dense layer's operators besides its products: argument checks and
// launches.  Declared in include/mxfp4_gemm.h.
#include <cstring>

#include "../../include/mxfp4_gemm.h"
#include "dense.h"
#include "expert.h"

using namespace mxfp4;

namespace {

constexpr size_t kAlign = 256;
// Sizes that the kernels' 32-bit steps past the last row or column cannot carry over the end.
constexpr int kMaxCount = 0x7FFFFFFF - (1 << 16);
constexpr int kMaxNorm = 32768;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t up32(int n) { return (static_cast<int64_t>(n) + 31) / 32 * 32; }
int status_of(cudaError_t e) { return e == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA; }
bool byte_fmt(int f) { return f == MXFP8_E4M3 || f == MXFP8_E5M2; }

// Codes [.., n] that are read or written: null, or rows of whole blocks on 16-byte boundaries with their scales.
int check_codes(const void *q, int64_t ldq, const void *s, int64_t lds, int n, int fmt)
{
    if (!q)
        return s ? MXFP4_ERR_INVALID_ARG : MXFP4_OK;
    if (!s || ldq < up32(n) || lds < up32(n) / 32 || !byte_fmt(fmt))
        return MXFP4_ERR_INVALID_ARG;
    return !aligned(q, 16) || (ldq % 16) != 0 ? MXFP4_ERR_MISALIGNED : MXFP4_OK;
}

CodesOut codes_out(void *q, int64_t ldq, void *s, int64_t lds, int fmt)
{
    return CodesOut{static_cast<uint8_t *>(q), ldq, static_cast<uint8_t *>(s), lds, fmt == MXFP8_E5M2 ? 1 : 0};
}

size_t partial_bytes(int64_t strips, int64_t cols)
{
    return strips > 1 ? align_up(static_cast<size_t>(strips) * static_cast<size_t>(cols) * sizeof(float)) : 0;
}

int check_workspace(size_t need, const void *workspace, size_t bytes)
{
    if (need == 0)
        return MXFP4_OK;
    if (!workspace || bytes < need)
        return MXFP4_ERR_WORKSPACE;
    return aligned(workspace, kAlign) ? MXFP4_OK : MXFP4_ERR_MISALIGNED;
}

// Rows of `size`-byte elements in boxes of `wide` columns x `tall` rows, zeros past the last ones.
bool encode(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t rows, int64_t cols, int64_t ld, int size, int wide, int tall,
            CUtensorMapSwizzle swizzle)
{
    auto enc = tensor_map_encode_fn();
    if (!enc)
        return false;
    if (rows == 1)
        ld = (cols + 15) / 16 * 16;                      // a lone row's stride can be anything
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * static_cast<cuuint64_t>(size)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(wide), static_cast<cuuint32_t>(tall)}, ones[2] = {1, 1};
    return enc(map, type, 2, const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same of an output's codes [rows, cols], whole blocks of 32 in each row; true too where it is not wanted.
bool encode_codes(CUtensorMap *map, const CodesOut &o, int64_t rows, int64_t cols, int wide, int tall, CUtensorMapSwizzle swizzle)
{
    return !o.q || encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.q, rows, (cols + 31) / 32 * 32, o.ldq, 1, wide, tall, swizzle);
}

int run_checkpoint(CheckpointArgs &a, bool backward, const void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    checkpoint_shape(a, backward);
    if (a.strips * a.across > 0x7FFFFFFF)
        return MXFP4_ERR_UNSUPPORTED_SHAPE;              // more blocks than a grid has
    int st = check_workspace(a.sums ? partial_bytes(a.strips, a.cols) : 0, workspace, workspace_bytes);
    if (st != MXFP4_OK)
        return st;
    int sms = 0;
    st = check_current_device(&sms);
    if (st != MXFP4_OK)
        return st;
    a.partials = static_cast<float *>(const_cast<void *>(workspace));
    a.wait_limit = current_wait_limit();
    BackwardMaps m;
    std::memset(&m, 0, sizeof(m));
    if (!encode(&m.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.rows, a.cols, a.ldx, 2, 64, backward ? 64 : 128, CU_TENSOR_MAP_SWIZZLE_128B))
        return MXFP4_ERR_CUDA;
    if (!backward)
        return status_of(launch_checkpoint(a, m.x, stream));
    if (!encode(&m.z, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.z, a.rows, a.cols, a.ldz, 1, 64, 64, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_codes(&m.by_row, a.by_row, a.rows, a.cols, 64, 64, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_codes(&m.by_col, a.by_col, a.cols, a.rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_codes(&m.act_by_col, a.act_by_col, a.cols, a.rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_64B))
        return MXFP4_ERR_CUDA;
    return status_of(launch_act_backward(a, m, stream));
}

// Rows of 16-bit values as the checkpoint kernels read them.
int check_rows(const void *x, int64_t ldx, int rows, int cols)
{
    if (!x || rows < 1 || cols < 1 || ldx < cols)
        return MXFP4_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ldx % 8) != 0)
        return MXFP4_ERR_MISALIGNED;
    return rows > kMaxCount || cols > kMaxCount ? MXFP4_ERR_UNSUPPORTED_SHAPE : MXFP4_OK;
}

// The widest access, in elements, that 16-bit rows at p allow.
void allow_rows(int &width, const void *p, int64_t ld)
{
    while (p && width > 1 && (!aligned(p, 2 * static_cast<size_t>(width)) || (ld % width) != 0))
        width /= 2;
}

void allow_param(int &width, const void *p, bool fp32)
{
    while (p && width > 1 && !aligned(p, fp32 ? (width >= 4 ? 16 : 4) : 2 * static_cast<size_t>(width)))
        width /= 2;
}

int check_norm(int T, int N, const void *w, const void *b, int param_type)
{
    if (T < 0 || N < 1 || (param_type != MXFP4_PARAM_BF16 && param_type != MXFP4_PARAM_FP32))
        return MXFP4_ERR_INVALID_ARG;
    const size_t size = param_type == MXFP4_PARAM_FP32 ? 4 : 2;
    if (!aligned(w, size) || !aligned(b, size))
        return MXFP4_ERR_MISALIGNED;
    return T > kMaxCount || N > kMaxNorm ? MXFP4_ERR_UNSUPPORTED_SHAPE : MXFP4_OK;
}

}  // namespace

extern "C" {

size_t mxfp8_checkpoint_workspace_size(int rows, int cols)
{
    if (rows < 1 || cols < 1 || rows > kMaxCount || cols > kMaxCount)
        return 0;
    size_t need = 0;
    for (const bool backward : {false, true}) {
        CheckpointArgs a{};
        a.rows = rows;
        a.cols = cols;
        checkpoint_shape(a, backward);
        const size_t bytes = partial_bytes(a.strips, cols);
        need = need > bytes ? need : bytes;
    }
    return need;
}

int mxfp8_checkpoint(void *Q, int64_t ldq, void *S, int64_t lds, void *QT, int64_t ldqt, void *ST, int64_t ldst, float *col_sums,
                     const void *X, int64_t ldx, int rows, int cols, int fmt, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!Q && !QT && !col_sums)
        return MXFP4_ERR_INVALID_ARG;
    if (!byte_fmt(fmt))
        return MXFP4_ERR_INVALID_ARG;
    int st = check_rows(X, ldx, rows, cols);
    if (st == MXFP4_OK)
        st = check_codes(Q, ldq, S, lds, cols, fmt);
    if (st == MXFP4_OK)
        st = check_codes(QT, ldqt, ST, ldst, rows, fmt);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(col_sums, 4))
        return MXFP4_ERR_MISALIGNED;
    CheckpointArgs a;
    std::memset(&a, 0, sizeof(a));
    a.by_row = codes_out(Q, ldq, S, lds, fmt);
    a.by_col = codes_out(QT, ldqt, ST, ldst, fmt);
    a.sums = col_sums;
    a.x = static_cast<const uint16_t *>(X);
    a.ldx = ldx;
    a.rows = rows;
    a.cols = cols;
    return run_checkpoint(a, false, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int mxfp8_act_backward(void *dZ, int64_t lddz, void *Q, int64_t ldq, void *S, int64_t lds, void *QT, int64_t ldqt, void *ST, int64_t ldst,
                       void *HT, int64_t ldht, void *SHT, int64_t ld_sht, float *dbias, const void *dH, int64_t lddh, const void *Z,
                       int64_t ldz, const void *SZ, int64_t ld_sz, int fmt_z, int act, int rows, int cols, int fmt, int fmt_h,
                       void *workspace, size_t workspace_bytes, void *stream)
{
    if (!dZ && !Q && !QT && !HT && !dbias)
        return MXFP4_ERR_INVALID_ARG;
    if (!byte_fmt(fmt) || !byte_fmt(fmt_h) || act < MXFP4_ACT_NONE || act > MXFP4_ACT_SILU || !Z || (dZ && lddz < cols))
        return MXFP4_ERR_INVALID_ARG;
    int st = check_rows(dH, lddh, rows, cols);
    if (st == MXFP4_OK)
        st = check_codes(Z, ldz, SZ, ld_sz, cols, fmt_z);
    if (st == MXFP4_OK)
        st = check_codes(Q, ldq, S, lds, cols, fmt);
    if (st == MXFP4_OK)
        st = check_codes(QT, ldqt, ST, ldst, rows, fmt);
    if (st == MXFP4_OK)
        st = check_codes(HT, ldht, SHT, ld_sht, rows, fmt_h);
    if (st != MXFP4_OK)
        return st;
    if (!aligned(dbias, 4) || !aligned(dZ, 2))
        return MXFP4_ERR_MISALIGNED;
    CheckpointArgs a;
    std::memset(&a, 0, sizeof(a));
    a.by_row = codes_out(Q, ldq, S, lds, fmt);
    a.by_col = codes_out(QT, ldqt, ST, ldst, fmt);
    a.act_by_col = codes_out(HT, ldht, SHT, ld_sht, fmt_h);
    a.dz = static_cast<uint16_t *>(dZ);
    a.lddz = lddz;
    a.vec_dz = aligned(dZ, 16) && (lddz % 8) == 0;
    a.sums = dbias;
    a.x = static_cast<const uint16_t *>(dH);
    a.ldx = lddh;
    a.z = static_cast<const uint8_t *>(Z);
    a.ldz = ldz;
    a.sz = static_cast<const uint8_t *>(SZ);
    a.ld_sz = ld_sz;
    a.fmt_z = fmt_z == MXFP8_E5M2 ? 1 : 0;
    a.act = act;
    a.rows = rows;
    a.cols = cols;
    return run_checkpoint(a, true, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int mxfp4_layer_norm(void *Y, int64_t ldy, float *mean, float *rstd, const void *X, int64_t ldx, const void *w, const void *b,
                     int param_type, float eps, int T, int N, void *stream)
{
    int st = check_norm(T, N, w, b, param_type);
    if (st == MXFP4_ERR_INVALID_ARG || !(eps >= 0.0f) || (T > 0 && (!Y || !X || ldy < N || ldx < N)))
        return MXFP4_ERR_INVALID_ARG;
    if (!aligned(Y, 2) || !aligned(X, 2) || !aligned(mean, 4) || !aligned(rstd, 4))
        return MXFP4_ERR_MISALIGNED;
    if (st != MXFP4_OK)
        return st;
    int sms = 0;
    st = check_current_device(&sms);
    if (st != MXFP4_OK || T == 0)
        return st;
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = static_cast<const uint16_t *>(X);
    a.ldx = ldx;
    a.w = w;
    a.b = b;
    a.fp32 = param_type == MXFP4_PARAM_FP32 ? 1 : 0;
    a.y = static_cast<uint16_t *>(Y);
    a.ldy = ldy;
    a.mean = mean;
    a.rstd = rstd;
    a.eps = eps;
    a.wait_limit = current_wait_limit();
    a.T = T;
    a.N = N;
    a.width = 8;
    allow_rows(a.width, X, T > 1 ? ldx : 0);
    allow_rows(a.width, Y, T > 1 ? ldy : 0);
    allow_param(a.width, w, a.fp32 != 0);
    allow_param(a.width, b, a.fp32 != 0);
    while (N % a.width != 0)
        a.width /= 2;
    return status_of(launch_layer_norm(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t mxfp4_layer_norm_workspace_size(int T, int N)
{
    if (T < 0 || N < 1 || T > kMaxCount || N > kMaxNorm)
        return 0;
    return partial_bytes(norm_backward_blocks(T, N), 2 * static_cast<int64_t>(N));
}

int mxfp4_layer_norm_backward(void *dX, int64_t lddx, float *dw, float *db, const void *dY, int64_t lddy, const void *X, int64_t ldx,
                              const float *mean, const float *rstd, const void *w, int param_type, const void *dres, int64_t ldr, int T,
                              int N, void *workspace, size_t workspace_bytes, void *stream)
{
    int st = check_norm(T, N, w, nullptr, param_type);
    if (st == MXFP4_ERR_INVALID_ARG ||
        (T > 0 && (!dX || !dY || !X || !mean || !rstd || lddx < N || lddy < N || ldx < N || (dres && ldr < N))))
        return MXFP4_ERR_INVALID_ARG;
    if (!aligned(dX, 2) || !aligned(dY, 2) || !aligned(X, 2) || !aligned(dres, 2) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        !aligned(dw, 4) || !aligned(db, 4))
        return MXFP4_ERR_MISALIGNED;
    if (st != MXFP4_OK)
        return st;
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.blocks = norm_backward_blocks(T, N);
    st = check_workspace(dw || db ? partial_bytes(a.blocks, 2 * static_cast<int64_t>(N)) : 0, workspace, workspace_bytes);
    if (st != MXFP4_OK)
        return st;
    int sms = 0;
    st = check_current_device(&sms);
    if (st != MXFP4_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0)                                          // sums of nothing
        return dw || db ? status_of(launch_sum_partials(dw, N, db, N, nullptr, 0, s)) : MXFP4_OK;
    a.x = static_cast<const uint16_t *>(X);
    a.ldx = ldx;
    a.w = w;
    a.fp32 = param_type == MXFP4_PARAM_FP32 ? 1 : 0;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dy = static_cast<const uint16_t *>(dY);
    a.lddy = lddy;
    a.dres = static_cast<const uint16_t *>(dres);
    a.ldr = ldr;
    a.dx = static_cast<uint16_t *>(dX);
    a.lddx = lddx;
    a.dw = dw;
    a.db = db;
    a.partials = static_cast<float *>(workspace);
    a.wait_limit = current_wait_limit();
    a.T = T;
    a.N = N;
    a.width = 8;
    allow_rows(a.width, X, T > 1 ? ldx : 0);
    allow_rows(a.width, dY, T > 1 ? lddy : 0);
    allow_rows(a.width, dX, T > 1 ? lddx : 0);
    allow_rows(a.width, dres, T > 1 ? ldr : 0);
    while (N % a.width != 0)
        a.width /= 2;
    // (w changes how it is read, and not the order of the sums)
    int width = a.width;
    allow_param(width, w, a.fp32 != 0);
    a.single_w = width < a.width ? 1 : 0;
    return status_of(launch_layer_norm_backward(a, s));
}

}  // extern "C"
