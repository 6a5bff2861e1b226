// Layer norm of bf16 rows and its gradients.
#include <cuda_bf16.h>

#include "dense.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace mxfp4 {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kRowWarps = 8;                     // rows of a block where a warp takes one

// ------------------------------------------------------------------- norm --
//
//   mean = sum x / N,  rstd = 1 / sqrt(sum (x - mean)^2 / N + eps)
//   y = (x - mean) rstd w + b                       one rounding, at the end
//
// A row lies in registers between the sums, so it is read once; the second
// sum is of the differences, not of squares, so that a large mean costs no
// precision.  Sums and statistics are fp32.  Short rows take a warp each, long
// ones a block.

// W elements as they lie in memory.
template <int W>
struct UnitOf;
template <>
struct UnitOf<8> { using T = uint4; };
template <>
struct UnitOf<4> { using T = uint2; };
template <>
struct UnitOf<2> { using T = uint32_t; };
template <>
struct UnitOf<1> { using T = uint16_t; };

template <int W>
__device__ __forceinline__ typename UnitOf<W>::T zero_unit()
{
    if constexpr (W == 8)
        return make_uint4(0u, 0u, 0u, 0u);
    else if constexpr (W == 4)
        return make_uint2(0u, 0u);
    else
        return 0;
}

template <int W>
__device__ __forceinline__ float pick(const typename UnitOf<W>::T &v, int i)
{
    uint32_t w;
    if constexpr (W == 8)
        w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    else if constexpr (W == 4)
        w = i < 2 ? v.x : v.y;
    else
        w = v;
    return i & 1 ? bf16_hi(w) : bf16_lo(w);
}

template <int W>
__device__ __forceinline__ typename UnitOf<W>::T load_unit(const uint16_t *p)
{
    return __ldcs(reinterpret_cast<const typename UnitOf<W>::T *>(p));
}

template <int W>
__device__ __forceinline__ void store_unit(uint16_t *p, const float (&x)[W])
{
    if constexpr (W == 1) {
        const __nv_bfloat16 v = __float2bfloat16_rn(x[0]);
        *p = *reinterpret_cast<const uint16_t *>(&v);
    } else {
        uint32_t w[W / 2];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        if constexpr (W == 8)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (W == 4)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(p) = w[0];
    }
}

// W parameters from element n on, `missing` where there is no array.
template <int W>
__device__ __forceinline__ void load_param(const void *p, int fp32, int n, float missing, float (&x)[W])
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            x[i] = missing;
    } else if (fp32) {
        const float *f = static_cast<const float *>(p) + n;
        if constexpr (W >= 4) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(f + i));
                x[i] = v.x;
                x[i + 1] = v.y;
                x[i + 2] = v.z;
                x[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
                x[i] = __ldg(f + i);
        }
    } else {
        const auto v = __ldg(reinterpret_cast<const typename UnitOf<W>::T *>(static_cast<const uint16_t *>(p) + n));
#pragma unroll
        for (int i = 0; i < W; ++i)
            x[i] = pick<W>(v, i);
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// Sums over the row's threads; every one of them gets them.  slots: one float2 per
// warp; callers alternate slots, so that the next call's writes do not meet this
// one's reads.
template <bool WARP>
__device__ __forceinline__ float2 row_sum(float2 v, float2 *slots)
{
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if constexpr (!WARP) {
        const int lane = threadIdx.x & 31, warps = static_cast<int>(blockDim.x) >> 5;
        if (lane == 0)
            slots[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? slots[lane] : make_float2(0.0f, 0.0f);
        v.x = warp_sum(v.x);
        v.y = warp_sum(v.y);
    }
    return v;
}

// EPT elements of a row per thread, in units of W.
template <int W, int EPT, bool WARP>
__global__ void __launch_bounds__(WARP ? kRowWarps * 32 : 1024) norm_kernel(const __grid_constant__ NormArgs a)
{
    constexpr int VPT = EPT / W;
    __shared__ float2 slots[2][32];
    const int tpr = WARP ? 32 : static_cast<int>(blockDim.x);
    const int at = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int rows = WARP ? kRowWarps : 1;
    const float inv_n = 1.0f / static_cast<float>(a.N);
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * rows + (WARP ? threadIdx.x >> 5 : 0); t < a.T;
         t += static_cast<int64_t>(gridDim.x) * rows) {
        typename UnitOf<W>::T x[VPT];
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = (v * tpr + at) * W;
            x[v] = n < a.N ? load_unit<W>(a.x + t * a.ldx + n) : zero_unit<W>();
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int i = 0; i < W; ++i)
                s.x += pick<W>(x[v], i);
        const float mean = row_sum<WARP>(s, slots[0]).x * inv_n;
        s.x = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if ((v * tpr + at) * W < a.N) {
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float d = pick<W>(x[v], i) - mean;
                    s.x = fmaf(d, d, s.x);
                }
            }
        const float rstd = rsqrtf(row_sum<WARP>(s, slots[1]).x * inv_n + a.eps);
        if (at == 0) {
            if (a.mean)
                a.mean[t] = mean;
            if (a.rstd)
                a.rstd[t] = rstd;
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = (v * tpr + at) * W;
            if (n < a.N) {
                float w[W], b[W], y[W];
                load_param<W>(a.w, a.fp32, n, 1.0f, w);
                load_param<W>(a.b, a.fp32, n, 0.0f, b);
#pragma unroll
                for (int i = 0; i < W; ++i)
                    y[i] = fmaf((pick<W>(x[v], i) - mean) * rstd, w[i], b[i]);
                store_unit<W>(a.y + t * a.ldy + n, y);
            }
        }
    }
}

// -------------------------------------------------------------- gradients --
//
// With xhat = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum g / N - xhat sum (g xhat) / N) + dres
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
// all in fp32; dx is rounded once.  x and dy are read once: a block takes rows
// gridDim apart, keeps its share of dw and db in registers and leaves it in
// partials, which a second kernel adds in a fixed order.
template <int W, int EPT, bool WARP, bool PARAMS>
__global__ void __launch_bounds__(WARP ? kRowWarps * 32 : PARAMS ? 512 : 1024) norm_backward_kernel(const __grid_constant__ NormArgs a)
{
    constexpr int VPT = EPT / W;
    __shared__ float2 slots[2][32];
    __shared__ float joint[WARP && PARAMS ? kRowWarps : 1][WARP && PARAMS ? 32 * EPT : 1];
    const int tpr = WARP ? 32 : static_cast<int>(blockDim.x);
    const int at = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int rows = WARP ? kRowWarps : 1;
    const float inv_n = 1.0f / static_cast<float>(a.N);
    float dw[PARAMS ? EPT : 1], db[PARAMS ? EPT : 1];
    if constexpr (PARAMS) {
#pragma unroll
        for (int i = 0; i < EPT; ++i)
            dw[i] = db[i] = 0.0f;
    }
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    int parity = 0;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * rows + (WARP ? threadIdx.x >> 5 : 0); t < a.T;
         t += static_cast<int64_t>(gridDim.x) * rows, parity ^= 1) {
        typename UnitOf<W>::T x[VPT], dy[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = (v * tpr + at) * W;
            x[v] = n < a.N ? load_unit<W>(a.x + t * a.ldx + n) : zero_unit<W>();
            dy[v] = n < a.N ? load_unit<W>(a.dy + t * a.lddy + n) : zero_unit<W>();
        }
        const float mean = a.mean[t], rstd = a.rstd[t];
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = (v * tpr + at) * W;
            if (n < a.N) {
                float w[W];
                load_param<W>(a.w, a.fp32, n, 1.0f, w);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float xhat = (pick<W>(x[v], i) - mean) * rstd, d = pick<W>(dy[v], i), g = d * w[i];
                    s.x += g;
                    s.y = fmaf(g, xhat, s.y);
                    if constexpr (PARAMS) {
                        dw[v * W + i] = fmaf(d, xhat, dw[v * W + i]);
                        db[v * W + i] += d;
                    }
                }
            }
        }
        s = row_sum<WARP>(s, slots[parity]);
        s.x *= inv_n;
        s.y *= inv_n;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = (v * tpr + at) * W;
            if (n < a.N) {
                float w[W], y[W];
                load_param<W>(a.w, a.fp32, n, 1.0f, w);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    const float xhat = (pick<W>(x[v], i) - mean) * rstd;
                    y[i] = rstd * (fmaf(pick<W>(dy[v], i), w[i], -s.x) - xhat * s.y);
                }
                if (a.dres) {
                    const auto r = load_unit<W>(a.dres + t * a.ldr + n);
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        y[i] += pick<W>(r, i);
                }
                store_unit<W>(a.dx + t * a.lddx + n, y);
            }
        }
    }
    if constexpr (PARAMS) {
        float *out[2] = {a.dw, a.db};
        if (gridDim.x > 1) {
            out[0] = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.N;
            out[1] = out[0] + a.N;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float *mine = k ? db : dw;
            if constexpr (WARP) {
                if (k)
                    __syncthreads();
#pragma unroll
                for (int v = 0; v < VPT; ++v)
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        joint[threadIdx.x >> 5][(v * 32 + at) * W + i] = mine[v * W + i];
                __syncthreads();
                for (int n = threadIdx.x; n < a.N; n += kRowWarps * 32) {
                    float s = 0.0f;
#pragma unroll
                    for (int r = 0; r < kRowWarps; ++r)
                        s += joint[r][n];
                    if (out[k])
                        out[k][n] = s;
                }
            } else if (out[k]) {
#pragma unroll
                for (int v = 0; v < VPT; ++v)
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        if ((v * tpr + at) * W < a.N)
                            out[k][(v * tpr + at) * W + i] = mine[v * W + i];
            }
        }
    }
}

// The gradients of many aligned rows: the same sums, with the rows streamed through
// shared memory.  A ring of stages, each the x, dy and dres of as many rows as
// 512 threads with 16 elements each hold, is filled by bulk copies; the
// threads take a stage into registers, add to dw and db and reduce, and the
// reduction's barrier is also what frees the stage for the next copy.  One block
// to an SM, 150 KB of reads in flight in each: bound by HBM.
constexpr int kRing = 8;                         // most stages
constexpr int kRingBytes = 200 << 10;
constexpr int kStreamThreads = 512;
constexpr int kStreamRow = 8192;                 // longest row: 16 elements a thread

struct StreamShape {
    int tpr;                    // threads of a row, whole warps
    int rows;                   // rows of a stage
    int row_bytes;
    int arrays;                 // 2, or 3 with dres
    int depth;                  // stages
};

__device__ int g_status = 0;                     // bounded waits that ran out

__global__ void __launch_bounds__(kStreamThreads, 1) norm_backward_stream_kernel(const __grid_constant__ NormArgs a, const StreamShape sh)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kRing];
    __shared__ float2 slots[2][kStreamThreads / 32];
    __shared__ int abort_flag;
    const int stage_bytes = sh.rows * sh.arrays * sh.row_bytes;
    const int mine = static_cast<int>(threadIdx.x) / sh.tpr;         // the thread's row of a stage
    const int at = static_cast<int>(threadIdx.x) - mine * sh.tpr;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool works = mine < sh.rows;
    const float inv_n = 1.0f / static_cast<float>(a.N);
    const int64_t groups = (static_cast<int64_t>(a.T) + sh.rows - 1) / sh.rows;
    const int64_t mygroups = groups > blockIdx.x ? (groups - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < sh.depth; ++s)
            mbar_init(&full[s], static_cast<uint32_t>(sh.rows));
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    // The first thread of each row copies that row of group k to stage s; rows past the last arrive empty.
    auto fill = [&](int64_t k, int s) {
        if (at != 0 || !works || k >= mygroups)
            return;
        const int64_t t = (blockIdx.x + k * gridDim.x) * sh.rows + mine;
        if (t >= a.T) {
            mbar_arrive(&full[s]);
            return;
        }
        const uint64_t policy = l2_policy_evict_first();
        uint8_t *dst = ring + s * stage_bytes + mine * sh.arrays * sh.row_bytes;
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(sh.arrays * sh.row_bytes));
        bulk_load(dst, a.x + t * a.ldx, static_cast<uint32_t>(sh.row_bytes), &full[s], policy);
        bulk_load(dst + sh.row_bytes, a.dy + t * a.lddy, static_cast<uint32_t>(sh.row_bytes), &full[s], policy);
        if (a.dres)
            bulk_load(dst + 2 * sh.row_bytes, a.dres + t * a.ldr, static_cast<uint32_t>(sh.row_bytes), &full[s], policy);
    };
    for (int k = 0; k < sh.depth; ++k)
        fill(k, k);
    const int n0 = at * 8, n1 = (sh.tpr + at) * 8;       // the thread's two units of a row
    const bool on0 = works && n0 < a.N, on1 = works && n1 < a.N;
    float w[16], dw[16], db[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        w[i] = dw[i] = db[i] = 0.0f;
    {
        float u[8];
        if (on0) {
            load_param<8>(a.w, a.fp32, n0, 1.0f, u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = u[i];
        }
        if (on1) {
            load_param<8>(a.w, a.fp32, n1, 1.0f, u);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[8 + i] = u[i];
        }
    }
    float mean = 0.0f, rstd = 0.0f;
    auto statistics = [&](int64_t k) {
        const int64_t t = (blockIdx.x + k * gridDim.x) * sh.rows + mine;
        if (works && k < mygroups && t < a.T) {
            mean = a.mean[t];
            rstd = a.rstd[t];
        }
    };
    statistics(0);
    int s = 0;
    uint32_t phase = 0;
    for (int64_t k = 0; k < mygroups; ++k) {
        const bool ok = mbar_wait(&full[s], phase, &abort_flag, a.wait_limit, &g_status);
        const int64_t t = (blockIdx.x + k * gridDim.x) * sh.rows + mine;
        const bool row = ok && t < a.T;
        const uint8_t *src = ring + s * stage_bytes + mine * sh.arrays * sh.row_bytes;
        uint4 x[2], dy[2], res[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            x[v] = dy[v] = res[v] = make_uint4(0u, 0u, 0u, 0u);
            if (row && (v ? on1 : on0)) {
                const uint8_t *p = src + 2 * (v ? n1 : n0);
                x[v] = *reinterpret_cast<const uint4 *>(p);
                dy[v] = *reinterpret_cast<const uint4 *>(p + sh.row_bytes);
                if (a.dres)
                    res[v] = *reinterpret_cast<const uint4 *>(p + 2 * sh.row_bytes);
            }
        }
        const float mu = mean, r = row ? rstd : 0.0f;
        statistics(k + 1);
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xhat = (pick<8>(x[v], i) - mu) * r, d = pick<8>(dy[v], i), g = d * w[8 * v + i];
                sum.x += g;
                sum.y = fmaf(g, xhat, sum.y);
                dw[8 * v + i] = fmaf(d, xhat, dw[8 * v + i]);
                db[8 * v + i] += d;
            }
        sum.x = warp_sum(sum.x);
        sum.y = warp_sum(sum.y);
        if (lane == 0)
            slots[k & 1][warp] = sum;
        // Every thread has taken the stage into registers: it fills again.
        if (__syncthreads_or(!ok)) {
            if (threadIdx.x == 0)                        // copies land before the block leaves
                for (int64_t j = k; j < k + sh.depth && j < mygroups; ++j) {
                    mbar_wait_drain(&full[s], phase, a.wait_limit);
                    if (++s == sh.depth) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            return;
        }
        fill(k + sh.depth, s);
        if (++s == sh.depth) {
            s = 0;
            phase ^= 1u;
        }
        const int first = mine * sh.tpr / 32, warps = sh.tpr / 32;
        sum = lane < warps && works ? slots[k & 1][first + lane] : make_float2(0.0f, 0.0f);
        sum.x = warp_sum(sum.x) * inv_n;
        sum.y = warp_sum(sum.y) * inv_n;
#pragma unroll
        for (int v = 0; v < 2; ++v)
            if (row && (v ? on1 : on0)) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xhat = (pick<8>(x[v], i) - mu) * r;
                    y[i] = r * (fmaf(pick<8>(dy[v], i), w[8 * v + i], -sum.x) - xhat * sum.y) + pick<8>(res[v], i);
                }
                store_unit<8>(a.dx + t * a.lddx + (v ? n1 : n0), y);
            }
    }
    if (!a.dw && !a.db)
        return;
    // The stage's rows of a block add up in the ring's memory, in their order.
    float *joint = reinterpret_cast<float *>(ring);
    float *out[2] = {a.dw, a.db};
    if (gridDim.x > 1) {
        out[0] = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.N;
        out[1] = out[0] + a.N;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < 2; ++v)
            if (v ? on1 : on0) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    joint[mine * a.N + (v ? n1 : n0) + i] = q ? db[8 * v + i] : dw[8 * v + i];
            }
        __syncthreads();
        for (int n = threadIdx.x; n < a.N; n += kStreamThreads) {
            float s = 0.0f;
            for (int g = 0; g < sh.rows; ++g)
                s += joint[g * a.N + n];
            if (out[q])
                out[q][n] = s;
        }
    }
}

// dw and db of rows too long for a block's registers: a block takes 32 W columns
// and rows gridDim.y apart, a warp every eighth of them.
template <int W>
__global__ void __launch_bounds__(256) norm_params_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float joint[8][2][32 * W];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int n = (static_cast<int>(blockIdx.x) * 32 + lane) * W;
    float dw[W], db[W];
#pragma unroll
    for (int i = 0; i < W; ++i)
        dw[i] = db[i] = 0.0f;
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    if (n < a.N)
        for (int64_t t = static_cast<int64_t>(blockIdx.y) * 8 + warp; t < a.T; t += static_cast<int64_t>(gridDim.y) * 8) {
            const auto x = load_unit<W>(a.x + t * a.ldx + n), dy = load_unit<W>(a.dy + t * a.lddy + n);
            const float mean = a.mean[t], rstd = a.rstd[t];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float d = pick<W>(dy, i);
                dw[i] = fmaf(d, (pick<W>(x, i) - mean) * rstd, dw[i]);
                db[i] += d;
            }
        }
#pragma unroll
    for (int i = 0; i < W; ++i) {
        joint[warp][0][lane * W + i] = dw[i];
        joint[warp][1][lane * W + i] = db[i];
    }
    __syncthreads();
    float *out[2] = {a.dw, a.db};
    if (gridDim.y > 1) {
        out[0] = a.partials + static_cast<int64_t>(blockIdx.y) * 2 * a.N;
        out[1] = out[0] + a.N;
    }
    for (int i = threadIdx.x; i < 2 * 32 * W; i += 256) {
        const int k = i / (32 * W), m = i % (32 * W), col = static_cast<int>(blockIdx.x) * 32 * W + m;
        if (col >= a.N || !out[k])
            continue;
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            s += joint[r][k][m];
        out[k][col] = s;
    }
}

constexpr int kWarpRow = 1024;                   // longest row of one warp: 32 elements a lane
constexpr int kStreamBlocks = 152;               // one to each SM of a GB300
constexpr int kBlockRow = 16384;                 // longest row whose dw and db fit a block's registers

// Elements a thread and threads a row, in whole warps.
int threads_for(int N, int ept) { return ((N + ept - 1) / ept + 31) / 32 * 32; }

template <int W, int EPT, bool WARP>
cudaError_t start_norm(const NormArgs &a, int sms, cudaStream_t stream)
{
    const int threads = WARP ? kRowWarps * 32 : threads_for(a.N, EPT);
    const int64_t blocks = WARP ? (static_cast<int64_t>(a.T) + kRowWarps - 1) / kRowWarps : a.T;
    const int64_t most = static_cast<int64_t>(sms) * (2048 / threads);
    return launch_dependent(norm_kernel<W, EPT, WARP>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                            dim3(static_cast<unsigned>(threads)), 0, stream, a);
}

template <int W>
cudaError_t start_norm_width(const NormArgs &a, int sms, cudaStream_t stream)
{
    // Many rows: 32 elements a thread, so that many rows are in flight on an SM.  Few: eight, the shortest
    // time for one row.
    const bool many = a.T > 2 * sms;
    if (a.N <= kWarpRow && many)
        return a.N <= 256 ? start_norm<W, 8, true>(a, sms, stream) : start_norm<W, 32, true>(a, sms, stream);
    if (a.N <= 8192 && !many)
        return start_norm<W, 8, false>(a, sms, stream);
    return start_norm<W, 32, false>(a, sms, stream);
}

template <int W, int EPT, bool WARP, bool PARAMS>
cudaError_t start_backward(const NormArgs &a, cudaStream_t stream)
{
    const int threads = WARP ? kRowWarps * 32 : threads_for(a.N, EPT);
    return launch_dependent(norm_backward_kernel<W, EPT, WARP, PARAMS>, dim3(static_cast<unsigned>(a.blocks)),
                            dim3(static_cast<unsigned>(threads)), 0, stream, a);
}

// Whether a call's rows are streamed: 16-byte rows of a fair length, enough of them to fill the ring.
bool streams(const NormArgs &a)
{
    return a.width == 8 && a.N > kWarpRow && a.N <= kStreamRow && a.T >= 8 * kStreamBlocks;
}

cudaError_t start_stream(const NormArgs &a, cudaStream_t stream)
{
    StreamShape sh;
    sh.tpr = threads_for(a.N, 16);
    sh.rows = kStreamThreads / sh.tpr;
    sh.row_bytes = 2 * a.N;
    sh.arrays = a.dres ? 3 : 2;
    const int stage = sh.rows * sh.arrays * sh.row_bytes;
    sh.depth = kRingBytes / stage < kRing ? kRingBytes / stage : kRing;
    const int bytes = sh.depth * stage;
    const cudaError_t e = opt_in<norm_backward_stream_kernel>(bytes);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(norm_backward_stream_kernel, dim3(static_cast<unsigned>(a.blocks)), dim3(kStreamThreads),
                            static_cast<size_t>(bytes), stream, a, sh);
}

template <int W>
cudaError_t start_backward_width(const NormArgs &a, cudaStream_t stream)
{
    if (a.N <= 256)
        return start_backward<W, 8, true, true>(a, stream);
    if (a.N <= kWarpRow)
        return start_backward<W, 32, true, true>(a, stream);
    if (a.N <= 8192)
        return start_backward<W, 16, false, true>(a, stream);
    if (a.N <= kBlockRow)
        return start_backward<W, 32, false, true>(a, stream);
    // First the sums: dx may take the place of what they read.
    const int cols = 32 * W;
    const cudaError_t e = !a.dw && !a.db ? cudaSuccess
                                         : launch_dependent(norm_params_kernel<W>, dim3(static_cast<unsigned>((a.N + cols - 1) / cols),
                                                                                        static_cast<unsigned>(a.blocks)),
                                                            dim3(256), 0, stream, a);
    return e == cudaSuccess ? start_backward<W, 32, false, false>(a, stream) : e;
}

}  // namespace

cudaError_t launch_layer_norm(const NormArgs &a, int sms, cudaStream_t stream)
{
    switch (a.width) {
    case 8: return start_norm_width<8>(a, sms, stream);
    case 4: return start_norm_width<4>(a, sms, stream);
    case 2: return start_norm_width<2>(a, sms, stream);
    default: return start_norm_width<1>(a, sms, stream);
    }
}

int norm_backward_blocks(int T, int N)
{
    const int64_t rows = N <= kWarpRow ? kRowWarps : 1;
    const int64_t need = (static_cast<int64_t>(T) + rows - 1) / rows;
    const int64_t most = 2 * 152;
    return static_cast<int>(need < 1 ? 1 : need < most ? need : most);
}

cudaError_t launch_layer_norm_backward(NormArgs &a, cudaStream_t stream)
{
    cudaError_t e;
    const bool stream_rows = streams(a);
    if (stream_rows)
        a.blocks = kStreamBlocks;                        // (fewer than norm_backward_blocks)
    switch (a.width) {
    case 8: e = stream_rows ? start_stream(a, stream) : start_backward_width<8>(a, stream); break;
    case 4: e = start_backward_width<4>(a, stream); break;
    case 2: e = start_backward_width<2>(a, stream); break;
    default: e = start_backward_width<1>(a, stream); break;
    }
    if (e == cudaSuccess && a.blocks > 1 && (a.dw || a.db))
        e = launch_sum_partials(a.dw, a.N, a.db, a.N, a.partials, a.blocks, stream);
    return e;
}

cudaError_t read_norm_status(int *status, int reset)
{
    const cudaError_t e = cudaMemcpyFromSymbol(status, g_status, sizeof(int));
    if (e != cudaSuccess || !reset)
        return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
}

}  // namespace mxfp4
