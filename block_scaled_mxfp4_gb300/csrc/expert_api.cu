// C ABI of the expert-layer operators: argument checks, tensor maps, launch
// sequences.  Declared in include/mxfp4_gemm.h.
#include <cstring>

#include "../../include/mxfp4_gemm.h"
#include "expert.h"
#include "ptx.cuh"

using namespace mxfp4;

namespace {

constexpr size_t kAlign = 256;
// Row and token counts that the kernels' 32-bit indexes can step over: a tile's
// rows (256) or a grid's tokens (a few thousand) past the last one.
constexpr int kMaxRows = 0x7FFFFFFF - (1 << 16);

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool bad_groups(int groups) { return groups < 1 || groups > kMaxGroups; }
bool bad_k(int K) { return K < 32 || (K % 32) != 0; }
bool known_fmt(int f) { return f == MXFP8_E4M3 || f == MXFP8_E5M2 || (f >= MXFP6_E2M3 && f <= MXFP4_E2M1_PADDED); }
int status_of(cudaError_t e) { return e == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA; }

bool encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle)
{
    auto enc = tensor_map_encode_fn();
    if (!enc)
        return false;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return enc(map, type, static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One grouped product.  Strides of A, B and of a quantised output in elements.
// out: -1 bf16 into D, else the QuantFmt of the codes written to D.
struct Product {
    void *D;
    int64_t ldd;
    void *SH;
    const void *A;
    int64_t lda;
    const void *SA;
    const void *B;
    int64_t ldb, stride_b;
    const void *SB;
    const int *offsets;
    int groups, rows, N, K;
    float alpha;
    bool bytes8;
    int fmt_a, fmt_b;
    int out;
    bool early;             // GroupedArgs::early
};

int check_product(const Product &p)
{
    const bool gated = p.out >= 0;
    const int64_t halves = gated ? 2 : 1;
    if (bad_groups(p.groups) || p.rows < 0 || p.N < 1 || bad_k(p.K) || (gated && (p.N % 32) != 0))
        return MXFP4_ERR_INVALID_ARG;
    if (p.rows == 0)
        return MXFP4_OK;                             // no array is touched
    if (!p.D || !p.A || !p.SA || !p.B || !p.SB || !p.offsets || (gated && !p.SH))
        return MXFP4_ERR_INVALID_ARG;
    if (p.lda < p.K || p.ldb < p.K || p.ldd < p.N || p.stride_b < halves * p.N * p.ldb)
        return MXFP4_ERR_INVALID_ARG;
    if (p.bytes8 && (!known_fmt(p.fmt_a) || !known_fmt(p.fmt_b)))
        return MXFP4_ERR_INVALID_ARG;
    const int unit = p.bytes8 ? 16 : 32;             // elements of 16 bytes
    if (!aligned(p.offsets, 4) || (p.lda % unit) != 0 || (p.ldb % unit) != 0 || (p.stride_b % unit) != 0 || !aligned(p.A, 16) ||
        !aligned(p.B, 16) || !aligned(p.SA, 16) || !aligned(p.SB, 16))
        return MXFP4_ERR_MISALIGNED;
    if (gated && ((p.ldd % unit) != 0 || !aligned(p.D, 16) || !aligned(p.SH, 16)))
        return MXFP4_ERR_MISALIGNED;
    if (!gated && !aligned(p.D, 2))
        return MXFP4_ERR_MISALIGNED;
    if (p.rows > kMaxRows)
        return MXFP4_ERR_UNSUPPORTED_SHAPE;
    const int64_t row_tiles = p.rows / 256 + (p.groups < p.rows ? p.groups : p.rows);
    const int64_t nt = (static_cast<int64_t>(p.N) + (gated ? 127 : 255)) / (gated ? 128 : 256);
    if (row_tiles * nt > 0x3FFFFFFF || group_sf_blocks(p.rows, p.groups) > 0x7FFFFFFF)
        return MXFP4_ERR_UNSUPPORTED_SHAPE;
    return MXFP4_OK;
}

int run_product(const Product &p, cudaStream_t stream)
{
    if (p.rows == 0)
        return MXFP4_OK;
    const bool gated = p.out >= 0;
    const int64_t den = p.bytes8 ? 1 : 2;            // elements per byte
    const int64_t atoms = sf_groups(p.K);
    const int per_stage = p.bytes8 ? 1 : 2;
    const int64_t rb = sf_row_blocks(p.N);
    GroupedMaps m;
    std::memset(&m, 0, sizeof(m));
    {
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.K / den), static_cast<cuuint64_t>(p.rows)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.lda / den)};
        const cuuint32_t box[2] = {128, 128}, box32[2] = {128, 32};
        if (!encode(&m.A, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.A, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode(&m.A32, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.A, dims, strides, box32, CU_TENSOR_MAP_SWIZZLE_128B))
            return MXFP4_ERR_CUDA;
    }
    {
        const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(atoms),
                                    static_cast<cuuint64_t>(group_sf_blocks(p.rows, p.groups))};
        const cuuint64_t strides[2] = {kSfAtomBytes, static_cast<cuuint64_t>(atoms * kSfAtomBytes)};
        const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(per_stage), 1};
        if (!encode(&m.SA, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, p.SA, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE))
            return MXFP4_ERR_CUDA;
    }
    {
        const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.K / den), static_cast<cuuint64_t>(p.N),
                                    gated ? 2ull : 1ull, static_cast<cuuint64_t>(p.groups)};
        const cuuint64_t row = static_cast<cuuint64_t>(p.ldb / den);
        const cuuint64_t strides[3] = {row, row * static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.stride_b / den)};
        const cuuint32_t box[4] = {128, gated ? 64u : 128u, gated ? 2u : 1u, 1};
        if (!encode(&m.B, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.B, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return MXFP4_ERR_CUDA;
    }
    {
        const cuuint64_t dims[4] = {128, static_cast<cuuint64_t>(atoms), static_cast<cuuint64_t>(rb),
                                    static_cast<cuuint64_t>(p.groups) * (gated ? 2 : 1)};
        const cuuint64_t strides[3] = {kSfAtomBytes, static_cast<cuuint64_t>(atoms * kSfAtomBytes),
                                       static_cast<cuuint64_t>(rb * atoms * kSfAtomBytes)};
        const cuuint32_t box[4] = {128, static_cast<cuuint32_t>(per_stage), gated ? 1u : 2u, gated ? 2u : 1u};
        if (!encode(&m.SB, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, p.SB, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE))
            return MXFP4_ERR_CUDA;
    }
    GroupedArgs a;
    std::memset(&a, 0, sizeof(a));
    a.offsets = p.offsets;
    a.groups = p.groups;
    a.rows = p.rows;
    a.N = p.N;
    a.K = p.K;
    const int stage = p.bytes8 ? 128 : 256;
    a.kt = (p.K + stage - 1) / stage;
    a.nt = gated ? (p.N + 127) / 128 : (p.N + 255) / 256;
    a.alpha = p.alpha;
    a.early = p.early ? 1 : 0;
    if (gated) {
        a.H = static_cast<uint8_t *>(p.D);
        a.ldh = p.out == 0 ? p.ldd / 2 : p.ldd;
        a.SH = static_cast<uint8_t *>(p.SH);
        a.vec32_ok = aligned(p.D, 32) && (a.ldh % 32) == 0;
    } else {
        a.D = static_cast<uint16_t *>(p.D);
        a.ldd = p.ldd;
        a.vec_ok = aligned(p.D, 16) && (p.ldd % 8) == 0;
        a.vec32_ok = aligned(p.D, 32) && (p.ldd % 16) == 0;
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.rows)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.ldd) * 2};
        const cuuint32_t box[2] = {32, 32};
        if (a.vec_ok && !encode(&m.D, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.D, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B))
            return MXFP4_ERR_CUDA;
    }
    if (p.bytes8) {
        a.idesc8 = idesc_mxf8(256, 256, static_cast<uint32_t>(p.fmt_a), static_cast<uint32_t>(p.fmt_b));
        a.idesc8_solo = idesc_mxf8(128, 256, static_cast<uint32_t>(p.fmt_a), static_cast<uint32_t>(p.fmt_b));
        a.idesc8_half = idesc_mxf8(128, 128, static_cast<uint32_t>(p.fmt_a), static_cast<uint32_t>(p.fmt_b));
    }
    a.wait_limit = current_wait_limit();
    return status_of(launch_grouped(a, m, p.bytes8, p.out, stream));
}

int product_entry(const Product &p, void *stream)
{
    int st = check_product(p);
    if (st != MXFP4_OK)
        return st;
    int sms = 0;
    st = check_current_device(&sms);
    if (st != MXFP4_OK)
        return st;
    return run_product(p, static_cast<cudaStream_t>(stream));
}

int quantize_entry(void *Q, int64_t ldq, void *S, const void *X, int64_t ldx, int T, int K, const int *slot_row,
                   const int *ids, int k, const int *offsets, int groups, int rows, int fmt, void *stream)
{
    if (T < 0 || bad_k(K) || bad_groups(groups) || rows < 0 ||
        (T > 0 && rows > 0 && (!Q || !S || !X || !offsets || ldx < K || ldq < K)))
        return MXFP4_ERR_INVALID_ARG;
    if ((slot_row == nullptr) != (ids == nullptr) || (slot_row ? k < 1 || k > kMaxTopK : k != 1 || rows != T))
        return MXFP4_ERR_INVALID_ARG;
    if (T > 0 && rows > 0 &&
        (!aligned(X, 16) || (ldx % 8) != 0 || !aligned(Q, 16) || (ldq % (fmt ? 16 : 32)) != 0 || !aligned(S, 16)))
        return MXFP4_ERR_MISALIGNED;
    if (!aligned(slot_row, 4) || !aligned(ids, 4) || !aligned(offsets, 4))
        return MXFP4_ERR_MISALIGNED;
    int sms = 0;
    const int st = check_current_device(&sms);
    if (st != MXFP4_OK)
        return st;
    if (T == 0 || rows == 0)
        return MXFP4_OK;
    GroupQuantArgs a;
    a.Q = static_cast<uint8_t *>(Q);
    a.ldq_bytes = fmt ? ldq : ldq / 2;
    a.S = static_cast<uint8_t *>(S);
    a.X = static_cast<const uint16_t *>(X);
    a.ldx = ldx;
    a.T = T;
    a.K = K;
    a.k = k;
    a.slot_row = slot_row;
    a.ids = ids;
    a.offsets = offsets;
    a.groups = groups;
    a.rows = rows;
    a.fmt = fmt;
    return status_of(launch_group_quantize(a, sms, static_cast<cudaStream_t>(stream)));
}

int run_combine(void *H, int64_t ldh, void *Nrm, int64_t ldn, const void *Y, int64_t ldy, int rows, const int *slot_row,
                const float *gates, int k, const void *resid, int64_t ldr, const void *w_post, const void *w_pre,
                float res_scale, float out_scale, float eps, int T, int N, bool early, int sms, void *stream)
{
    CombineArgs a;
    a.H = static_cast<uint16_t *>(H);
    a.ldh = ldh;
    a.Nrm = static_cast<uint16_t *>(Nrm);
    a.ldn = ldn;
    a.Y = static_cast<const uint16_t *>(Y);
    a.ldy = ldy;
    a.rows = rows;
    a.slot_row = slot_row;
    a.gates = gates;
    a.k = k;
    a.resid = static_cast<const uint16_t *>(resid);
    a.ldr = ldr;
    a.w_post = static_cast<const uint16_t *>(w_post);
    a.w_pre = static_cast<const uint16_t *>(w_pre);
    a.res_scale = res_scale;
    a.out_scale = out_scale;
    a.eps = eps;
    a.T = T;
    a.N = N;
    a.early = early ? 1 : 0;
    a.wait_limit = current_wait_limit();
    a.width = 8;
    auto allow = [&a](const void *p, int64_t ld) {
        while (p && a.width > 1 && (!aligned(p, 2 * static_cast<size_t>(a.width)) || (ld % a.width) != 0))
            a.width /= 2;
    };
    allow(H, ldh);
    allow(Nrm, ldn);
    allow(Y, ldy);
    allow(resid, ldr);
    allow(w_post, N);
    allow(w_pre, N);
    while (N % a.width != 0)
        a.width /= 2;
    return status_of(launch_combine(a, sms, static_cast<cudaStream_t>(stream)));
}

// Workspace of mxfp4_moe_ffn: what each step leaves for the next.
struct FfnLayout {
    size_t q, sq, h, sh, y, total;
};

FfnLayout ffn_layout(int T, int E, int k, int K, int F)
{
    const int rows = T * k;
    FfnLayout l;
    size_t at = 0;
    auto take = [&at](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes);
        return here;
    };
    l.q = take(static_cast<size_t>(rows) * (K / 2));
    l.sq = take(static_cast<size_t>(group_sf_blocks(rows, E) * sf_groups(K) * kSfAtomBytes));
    l.h = take(static_cast<size_t>(rows) * (F / 2));
    l.sh = take(static_cast<size_t>(group_sf_blocks(rows, E) * sf_groups(F) * kSfAtomBytes));
    l.y = take(static_cast<size_t>(rows) * K * 2);
    l.total = at;
    return l;
}

bool bad_ffn_sizes(int T, int E, int k, int K, int F)
{
    return T < 0 || bad_groups(E) || k < 1 || k > kMaxTopK || k > E || bad_k(K) || bad_k(F) ||
           static_cast<int64_t>(T) * k > 0x7FFFFFFF;
}

}  // namespace

extern "C" {

size_t mxfp4_moe_route_workspace_size(int T, int E)
{
    if (T < 0 || bad_groups(E))
        return 0;
    int chunk = 0;
    const int blocks = route_blocks(T, &chunk);
    return blocks > 1 ? align_up(static_cast<size_t>(blocks) * ((E + 7) / 8 * 8) * 2) : 0;
}

int mxfp4_moe_route(int *ids, float *gates, int *offsets, int *row_token, int *slot_row, const void *logits,
                    int64_t ldl, int logits_type, const void *token_mask, int T, int E, int k, int gate_mode,
                    float gate_scale, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!offsets || T < 0 || bad_groups(E) || k < 1 || k > kMaxTopK || k > E ||
        (T > 0 && (!ids || !gates || !row_token || !slot_row || !logits || ldl < E)) ||
        (logits_type != MXFP4_LOGITS_BF16 && logits_type != MXFP4_LOGITS_FP32) || gate_mode < MXFP4_GATE_TOPK ||
        gate_mode > MXFP4_GATE_SIGMOID)
        return MXFP4_ERR_INVALID_ARG;
    if (!aligned(logits, logits_type == MXFP4_LOGITS_FP32 ? 4 : 2))
        return MXFP4_ERR_MISALIGNED;
    if (!aligned(ids, 4) || !aligned(gates, 4) || !aligned(offsets, 4) || !aligned(row_token, 4) || !aligned(slot_row, 4))
        return MXFP4_ERR_MISALIGNED;
    RouteArgs a;
    a.blocks = route_blocks(T, &a.chunk);
    if (static_cast<int64_t>(T) * k > 0x7FFFFFFF || a.chunk > 65504)
        return MXFP4_ERR_UNSUPPORTED_SHAPE;
    if (a.blocks > 1) {
        if (!workspace || workspace_bytes < mxfp4_moe_route_workspace_size(T, E))
            return MXFP4_ERR_WORKSPACE;
        if (!aligned(workspace, kAlign))
            return MXFP4_ERR_MISALIGNED;
    }
    int sms = 0;
    const int st = check_current_device(&sms);
    if (st != MXFP4_OK)
        return st;
    a.logits = logits;
    a.ldl = ldl;
    a.fp32 = logits_type == MXFP4_LOGITS_FP32;
    a.vec = aligned(logits, a.fp32 ? 16 : 8) && (ldl % 4) == 0;
    a.mask = static_cast<const uint8_t *>(token_mask);
    a.T = T;
    a.E = E;
    a.k = k;
    a.mode = gate_mode;
    a.gate_scale = gate_scale;
    a.ids = ids;
    a.gates = gates;
    a.offsets = offsets;
    a.row_token = row_token;
    a.slot_row = slot_row;
    a.counts = static_cast<uint16_t *>(workspace);
    return status_of(launch_route(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t mxfp4_group_scale_size(int rows, int groups, int K)
{
    if (rows < 0 || bad_groups(groups) || bad_k(K))
        return 0;
    return static_cast<size_t>(group_sf_blocks(rows, groups) * sf_groups(K) * kSfAtomBytes);
}

int mxfp4_group_quantize(void *Q, int64_t ldq, void *S, const void *X, int64_t ldx, int T, int K, const int *slot_row,
                         const int *ids, int k, const int *offsets, int groups, int rows, void *stream)
{
    return quantize_entry(Q, ldq, S, X, ldx, T, K, slot_row, ids, k, offsets, groups, rows, 0, stream);
}

int mxfp8_group_quantize(void *Q, int64_t ldq, void *S, const void *X, int64_t ldx, int T, int K, const int *slot_row,
                         const int *ids, int k, const int *offsets, int groups, int rows, int fmt, void *stream)
{
    if (fmt != MXFP8_E4M3 && fmt != MXFP8_E5M2)
        return MXFP4_ERR_INVALID_ARG;
    return quantize_entry(Q, ldq, S, X, ldx, T, K, slot_row, ids, k, offsets, groups, rows, 1 + fmt, stream);
}

// The present kernels keep everything on chip.
size_t mxfp4_grouped_workspace_size(int, int, int, int) { return 0; }

int mxfp4_grouped_gemm(void *D, int64_t ldd, const void *A, int64_t lda, const void *SA, const void *B, int64_t ldb,
                       int64_t stride_b, const void *SB, const int *offsets, int groups, int rows, int N, int K,
                       float alpha, void *, size_t, void *stream)
{
    const Product p{D, ldd, nullptr, A, lda, SA, B, ldb, stride_b, SB, offsets, groups, rows, N, K, alpha,
                    false, 0, 0, -1, false};
    return product_entry(p, stream);
}

int mxfp8_grouped_gemm(void *D, int64_t ldd, const void *A, int64_t lda, const void *SA, const void *B, int64_t ldb,
                       int64_t stride_b, const void *SB, const int *offsets, int groups, int rows, int N, int K,
                       int fmt_a, int fmt_b, float alpha, void *, size_t, void *stream)
{
    const Product p{D, ldd, nullptr, A, lda, SA, B, ldb, stride_b, SB, offsets, groups, rows, N, K, alpha,
                    true, fmt_a, fmt_b, -1, false};
    return product_entry(p, stream);
}

int mxfp4_grouped_swiglu(void *H, int64_t ldh, void *SH, const void *A, int64_t lda, const void *SA, const void *B,
                         int64_t ldb, int64_t stride_b, const void *SB, const int *offsets, int groups, int rows,
                         int F, int K, float alpha, void *, size_t, void *stream)
{
    const Product p{H, ldh, SH, A, lda, SA, B, ldb, stride_b, SB, offsets, groups, rows, F, K, alpha,
                    false, 0, 0, 0, false};
    return product_entry(p, stream);
}

int mxfp8_grouped_swiglu(void *H, int64_t ldh, void *SH, const void *A, int64_t lda, const void *SA, const void *B,
                         int64_t ldb, int64_t stride_b, const void *SB, const int *offsets, int groups, int rows,
                         int F, int K, int fmt_a, int fmt_b, int fmt_h, float alpha, void *, size_t, void *stream)
{
    if (fmt_h != MXFP8_E4M3 && fmt_h != MXFP8_E5M2)
        return MXFP4_ERR_INVALID_ARG;
    const Product p{H, ldh, SH, A, lda, SA, B, ldb, stride_b, SB, offsets, groups, rows, F, K, alpha,
                    true, fmt_a, fmt_b, 1 + fmt_h, false};
    return product_entry(p, stream);
}

int mxfp4_moe_combine(void *H, int64_t ldh, void *Nrm, int64_t ldn, const void *Y, int64_t ldy, int rows,
                      const int *slot_row, const float *gates, int k, const void *resid, int64_t ldr,
                      const void *w_post, const void *w_pre, float res_scale, float out_scale, float eps, int T, int N,
                      void *stream)
{
    if (T < 0 || N < 1 || rows < 0 || k < 1 || k > kMaxTopK || (!slot_row && (k != 1 || rows < T)) || !(eps >= 0.0f))
        return MXFP4_ERR_INVALID_ARG;
    if (T > 0 && ((!H && !Nrm) || (rows > 0 && (!Y || ldy < N)) || (H && ldh < N) || (Nrm && ldn < N) || (resid && ldr < N)))
        return MXFP4_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(H), static_cast<const void *>(Nrm), Y, resid, w_post, w_pre})
        if (!aligned(p, 2))
            return MXFP4_ERR_MISALIGNED;
    if (!aligned(slot_row, 4) || !aligned(gates, 4))
        return MXFP4_ERR_MISALIGNED;
    if (N > 32768 || T > kMaxRows)
        return MXFP4_ERR_UNSUPPORTED_SHAPE;
    int sms = 0;
    const int st = check_current_device(&sms);
    if (st != MXFP4_OK)
        return st;
    if (T == 0)
        return MXFP4_OK;
    return run_combine(H, ldh, Nrm, ldn, Y, ldy, rows, slot_row, gates, k, resid, ldr, w_post, w_pre, res_scale,
                       out_scale, eps, T, N, false, sms, stream);
}

size_t mxfp4_moe_ffn_workspace_size(int T, int E, int k, int K, int F)
{
    if (bad_ffn_sizes(T, E, k, K, F))
        return 0;
    return ffn_layout(T, E, k, K, F).total;
}

int mxfp4_moe_ffn(void *H, int64_t ldh, void *Nrm, int64_t ldn, const void *X, int64_t ldx, const int *ids,
                  const float *gates, const int *offsets, const int *slot_row, int T, int E, int k, int K, int F,
                  const void *B1, int64_t ldb1, const void *SB1, const void *B2, int64_t ldb2, const void *SB2,
                  const void *resid, int64_t ldr, const void *w_post, const void *w_pre, float res_scale,
                  float out_scale, float eps, void *workspace, size_t workspace_bytes, void *stream)
{
    if (bad_ffn_sizes(T, E, k, K, F) || !(eps >= 0.0f))
        return MXFP4_ERR_INVALID_ARG;
    if (T > 0 && (!ids || !gates || !slot_row || !X || ldx < K || (!H && !Nrm) || (H && ldh < K) ||
                  (Nrm && ldn < K) || (resid && ldr < K)))
        return MXFP4_ERR_INVALID_ARG;
    if (K > 32768 || static_cast<int64_t>(T) * k > kMaxRows)
        return MXFP4_ERR_UNSUPPORTED_SHAPE;
    if (T > 0 && (!aligned(H, 2) || !aligned(Nrm, 2) || !aligned(resid, 2) || !aligned(w_post, 2) ||
                  !aligned(w_pre, 2) || !aligned(X, 16) || (ldx % 8) != 0 || !aligned(ids, 4) || !aligned(gates, 4) ||
                  !aligned(slot_row, 4) || !aligned(workspace, kAlign)))
        return MXFP4_ERR_MISALIGNED;
    const FfnLayout l = ffn_layout(T, E, k, K, F);
    if (T > 0 && (!workspace || workspace_bytes < l.total))
        return MXFP4_ERR_WORKSPACE;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    const int rows = T * k;
    // Every step's arguments are checked before the first one is enqueued.
    const Product up{w + l.h, F, w + l.sh, w + l.q, K, w + l.sq, B1, ldb1, 2 * static_cast<int64_t>(F) * ldb1, SB1,
                     offsets, E, rows, F, K, 1.0f, false, 0, 0, 0, true};
    const Product down{w + l.y, K, nullptr, w + l.h, F, w + l.sh, B2, ldb2, static_cast<int64_t>(K) * ldb2, SB2,
                       offsets, E, rows, K, F, 1.0f, false, 0, 0, -1, true};
    int st = check_product(up);
    if (st == MXFP4_OK)
        st = check_product(down);
    if (st != MXFP4_OK)
        return st;
    int sms = 0;
    st = check_current_device(&sms);
    if (st != MXFP4_OK || T == 0)
        return st;
    // The quantiser waits for the work before the call, so that the steps after
    // it may read the call's own inputs before their predecessor has ended.
    st = mxfp4_group_quantize(w + l.q, K, w + l.sq, X, ldx, T, K, slot_row, ids, k, offsets, E, rows, stream);
    if (st == MXFP4_OK)
        st = run_product(up, static_cast<cudaStream_t>(stream));
    if (st == MXFP4_OK)
        st = run_product(down, static_cast<cudaStream_t>(stream));
    if (st == MXFP4_OK)
        st = run_combine(H, ldh, Nrm, ldn, w + l.y, K, rows, slot_row, gates, k, resid, ldr, w_post, w_pre, res_scale,
                         out_scale, eps, T, K, true, sms, stream);
    return st;
}

}  // extern "C"
