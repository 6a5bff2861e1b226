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

// ------------------------------------------------------------ many rows --
//
// The same sums with the rows streamed through shared memory.  A ring of stages,
// each the arrays' rows of as many row numbers as 512 threads with 16 elements
// each hold, is filled by bulk copies; the threads take a stage into registers and
// reduce, and the reduction's barrier is also what frees the stage for the next
// copy.  Bound by HBM.
//
// Bulk copies want 16-byte boundaries.  Rows off them are copied from the boundary
// before to the one after, which lie in the array except at its two ends: the
// first and the last row are read straight from memory instead.

constexpr int kRing = 8;                         // most stages
constexpr int kStreamThreads = 512;
constexpr int kStreamRow = 8192;                 // longest row: 16 elements a thread

struct StreamShape {
    int tpr;                    // threads of a row, whole warps
    int rows;                   // rows of a stage
    int slot;                   // bytes of a row in the ring
    int arrays;
    int depth;                  // stages
};

__device__ int g_status = 0;                     // bounded waits that ran out

// Element i of a thread's 16: whole units of eight, or (W = 1) neighbours to neighbouring lanes.
template <int W>
__device__ __forceinline__ int element(int tpr, int at, int i)
{
    return W == 8 ? (i / 8 * tpr + at) * 8 + i % 8 : i * tpr + at;
}

// Two elements, as they lie in a word.
__device__ __forceinline__ F2 pair_of(uint32_t w) { return f2(bf16_lo(w), bf16_hi(w)); }

// A thread's 16 elements of a row at p (shared or global memory), zeros past the end.
template <int W>
__device__ __forceinline__ void take(const uint16_t *p, int tpr, int at, int N, bool row, uint32_t (&w)[8])
{
    if constexpr (W == 8) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            uint4 q = make_uint4(0u, 0u, 0u, 0u);
            if (row && element<8>(tpr, at, 8 * v) < N)
                q = *reinterpret_cast<const uint4 *>(p + element<8>(tpr, at, 8 * v));
            w[4 * v] = q.x;
            w[4 * v + 1] = q.y;
            w[4 * v + 2] = q.z;
            w[4 * v + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int lo = element<1>(tpr, at, 2 * i), hi = element<1>(tpr, at, 2 * i + 1);
            w[i] = (row && lo < N ? static_cast<uint32_t>(p[lo]) : 0u) | (row && hi < N ? static_cast<uint32_t>(p[hi]) << 16 : 0u);
        }
    }
}

template <int W>
__device__ __forceinline__ void give(uint16_t *p, int tpr, int at, int N, const F2 (&y)[8])
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 v = parts(y[i]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    if constexpr (W == 8) {
#pragma unroll
        for (int v = 0; v < 2; ++v)
            if (element<8>(tpr, at, 8 * v) < N)
                *reinterpret_cast<uint4 *>(p + element<8>(tpr, at, 8 * v)) = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (element<1>(tpr, at, i) < N)
                p[element<1>(tpr, at, i)] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
    }
}

// A thread's 16 parameters, zeros past the end.
template <int W>
__device__ __forceinline__ void take_params(const void *p, int fp32, float missing, int tpr, int at, int N, F2 (&w)[8])
{
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; i += W) {
        float u[W];
#pragma unroll
        for (int j = 0; j < W; ++j)
            u[j] = 0.0f;
        if (element<W>(tpr, at, i) < N)
            load_param<W>(p, fp32, element<W>(tpr, at, i), missing, u);
#pragma unroll
        for (int j = 0; j < W; ++j)
            v[i + j] = u[j];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = f2(v[2 * i], v[2 * i + 1]);
}

// x - m of two elements, zero past the row's end (where x is 0 and m need not be a number).
template <int W>
__device__ __forceinline__ F2 centred(uint32_t word, F2 minus_m, int tpr, int at, int N, int i)
{
    const F2 d = pair_of(word) + minus_m;
    if (W == 8)
        return element<8>(tpr, at, 2 * i) < N ? d : f2(0.0f);
    const float2 v = parts(d);
    return f2(element<1>(tpr, at, 2 * i) < N ? v.x : 0.0f, element<1>(tpr, at, 2 * i + 1) < N ? v.y : 0.0f);
}

// The ring of one block.  Group k of the block is its rows first + k * step .. + rows - 1; stage
// k % depth holds it.  (Row numbers past the last stay below 2^31: T does by more than a step.)
template <int W, int ARRAYS>
struct Ring {
    const uint16_t *array[ARRAYS];
    int64_t ld[ARRAYS];
    uint8_t *memory;            // of the thread's row in stage 0
    uint64_t *full;
    StreamShape sh;
    int T, bytes;               // bytes of a row
    int t;                      // the row that is filled next: the thread's
    int step, last;             // last: no group starts behind it
    int mine;
    int s = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ int stage_bytes() const { return sh.rows * sh.arrays * sh.slot; }
    // Rows that are not copied: W = 1, the arrays' ends.
    __device__ __forceinline__ bool direct(int row) const { return W == 1 && (row == 0 || row == T - 1); }
    __device__ __forceinline__ static uint32_t ahead(const uint16_t *p) { return W == 1 ? reinterpret_cast<uintptr_t>(p) & 15u : 0u; }

    // By the first thread of each row: copy that row of the next group to stage `stage`; rows past the
    // last, and those that are read from memory, arrive empty.
    __device__ __forceinline__ void fill(int stage)
    {
        const int row = t;
        if (row - mine > last)
            return;
        t += step;
        if (row >= T || direct(row)) {
            mbar_arrive(&full[stage]);
            return;
        }
        const uint64_t policy = l2_policy_evict_first();
        const uint16_t *p[ARRAYS];
        uint32_t size[ARRAYS], total = 0;
#pragma unroll
        for (int i = 0; i < ARRAYS; ++i)
            if (i < sh.arrays) {
                p[i] = array[i] + row * ld[i];
                size[i] = W == 8 ? bytes : (ahead(p[i]) + bytes + 15u) / 16u * 16u;
                total += size[i];
            }
        mbar_arrive_expect_tx(&full[stage], total);
#pragma unroll
        for (int i = 0; i < ARRAYS; ++i)
            if (i < sh.arrays)
                bulk_load(memory + stage * stage_bytes() + i * sh.slot, reinterpret_cast<const uint8_t *>(p[i]) - ahead(p[i]), size[i],
                          &full[stage], policy);
    }
    // Array i's row `row` of the present stage.
    __device__ __forceinline__ const uint16_t *at_row(int row, int i) const
    {
        const uint8_t *here = memory + s * stage_bytes() + i * sh.slot;
        if (W == 8)
            return reinterpret_cast<const uint16_t *>(here);
        const uint16_t *p = array[i] + row * ld[i];
        return direct(row) ? p : reinterpret_cast<const uint16_t *>(here + ahead(p));
    }
    __device__ __forceinline__ void next()
    {
        if (++s == sh.depth) {
            s = 0;
            phase ^= 1u;
        }
    }
    // After a wait that ran out: the copies of the stages from this one on land before the block leaves.
    __device__ __forceinline__ void drain(int first, long long limit)
    {
        for (int j = 0; j < sh.depth && first <= last; ++j, first += step) {
            mbar_wait_drain(&full[s], phase, limit);
            next();
        }
    }
};

// One block to an SM.
template <int W>
__global__ void __launch_bounds__(kStreamThreads, 1) norm_backward_stream_kernel(const __grid_constant__ NormArgs a, const StreamShape sh)
{
    extern __shared__ __align__(128) uint8_t memory[];
    __shared__ uint64_t full[kRing];
    __shared__ float2 slots[2][kStreamThreads / 32];
    __shared__ int abort_flag;
    const int mine = static_cast<int>(threadIdx.x) / sh.tpr;         // the thread's row of a stage
    const int at = static_cast<int>(threadIdx.x) - mine * sh.tpr;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool works = mine < sh.rows, fills = works && at == 0;
    const float inv_n = 1.0f / static_cast<float>(a.N);
    const int first = static_cast<int>(blockIdx.x) * sh.rows, step = static_cast<int>(gridDim.x) * sh.rows;
    Ring<W, 3> ring{{a.x, a.dy, a.dres}, {a.ldx, a.lddy, a.ldr}, memory + mine * sh.arrays * sh.slot, full, sh, a.T, 2 * a.N, first + mine, step,
                    a.T - 1, mine};
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
    if (fills)
        for (int k = 0; k < sh.depth; ++k)
            ring.fill(k);
    F2 w[8], dw[8], db[8];
    take_params<W>(a.w, a.fp32, 1.0f, sh.tpr, at, a.N, w);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        dw[i] = db[i] = f2(0.0f);
    const int warp0 = mine * sh.tpr / 32, warps = sh.tpr / 32;
    float mean = 0.0f, rstd = 0.0f;
    if (works && first + mine < a.T) {
        mean = a.mean[first + mine];
        rstd = a.rstd[first + mine];
    }
    uint16_t *out = a.dx + (first + mine) * a.lddx;
    int parity = 0;
    for (int t0 = first; t0 < a.T; t0 += step, parity ^= 1, out += step * a.lddx) {
        const bool ok = mbar_wait(&full[ring.s], ring.phase, &abort_flag, a.wait_limit, &g_status);
        const int t = t0 + mine;
        const bool row = ok && works && t < a.T;
        uint32_t x[8], dy[8], res[8];
        take<W>(ring.at_row(t, 0), sh.tpr, at, a.N, row, x);
        take<W>(ring.at_row(t, 1), sh.tpr, at, a.N, row, dy);
        if (a.dres)
            take<W>(ring.at_row(t, 2), sh.tpr, at, a.N, row, res);
        const F2 minus_m = f2(row ? -mean : 0.0f), r = f2(row ? rstd : 0.0f);
        if (works && t + step < a.T) {
            mean = a.mean[t + step];
            rstd = a.rstd[t + step];
        }
        F2 s1 = f2(0.0f), s2 = f2(0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const F2 xhat = centred<W>(x[i], minus_m, sh.tpr, at, a.N, i) * r, d = pair_of(dy[i]), g = d * w[i];
            s1 = s1 + g;
            s2 = fma2(g, xhat, s2);
            dw[i] = fma2(d, xhat, dw[i]);
            db[i] = db[i] + d;
        }
        const float2 p1 = parts(s1), p2 = parts(s2);
        float2 sum = make_float2(warp_sum(p1.x + p1.y), warp_sum(p2.x + p2.y));
        if (lane == 0)
            slots[parity][warp] = sum;
        // Every thread has taken the stage into registers: it fills again.
        if (__syncthreads_or(!ok)) {
            if (threadIdx.x == 0)
                ring.drain(t0, a.wait_limit);
            return;
        }
        if (fills)
            ring.fill(ring.s);
        ring.next();
        sum = lane < warps && works ? slots[parity][warp0 + lane] : make_float2(0.0f, 0.0f);
        const F2 m1 = f2(-warp_sum(sum.x) * inv_n), m2 = f2(-warp_sum(sum.y) * inv_n);
        if (row) {
            F2 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const F2 xhat = (pair_of(x[i]) + minus_m) * r;
                y[i] = r * fma2(xhat, m2, fma2(pair_of(dy[i]), w[i], m1));
                if (a.dres)
                    y[i] = y[i] + pair_of(res[i]);
            }
            give<W>(out, sh.tpr, at, a.N, y);
        }
    }
    if (!a.dw && !a.db)
        return;
    // The stage's rows of a block add up in the ring's memory, in their order.
    float *joint = reinterpret_cast<float *>(memory);
    float *sums[2] = {a.dw, a.db};
    if (gridDim.x > 1) {
        sums[0] = a.partials + static_cast<int64_t>(blockIdx.x) * 2 * a.N;
        sums[1] = sums[0] + a.N;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        __syncthreads();
        if (works) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 v = parts(q ? db[i / 2] : dw[i / 2]);
                if (element<W>(sh.tpr, at, i) < a.N)
                    joint[mine * a.N + element<W>(sh.tpr, at, i)] = i & 1 ? v.y : v.x;
            }
        }
        __syncthreads();
        for (int n = threadIdx.x; n < a.N; n += kStreamThreads) {
            float s = 0.0f;
            for (int g = 0; g < sh.rows; ++g)
                s += joint[g * a.N + n];
            if (sums[q])
                sums[q][n] = s;
        }
    }
}

// The norm itself: two blocks to an SM, half of the ring each.  One barrier a
// stage: a warp takes the mean of its elements and the squares of their
// differences from that, and the row's follow from the warps' as
//   m = sum n_i m_i / N,  sum (x - m)^2 = sum [q_i + n_i (m_i - m)^2],
// sums of positive terms throughout.
template <int W>
__global__ void __launch_bounds__(kStreamThreads, 2) norm_stream_kernel(const __grid_constant__ NormArgs a, const StreamShape sh)
{
    extern __shared__ __align__(128) uint8_t memory[];
    __shared__ uint64_t full[kRing];
    __shared__ float2 slots[2][kStreamThreads / 32];
    __shared__ int abort_flag;
    const int mine = static_cast<int>(threadIdx.x) / sh.tpr;
    const int at = static_cast<int>(threadIdx.x) - mine * sh.tpr;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool works = mine < sh.rows, fills = works && at == 0;
    const float inv_n = 1.0f / static_cast<float>(a.N);
    const int first = static_cast<int>(blockIdx.x) * sh.rows, step = static_cast<int>(gridDim.x) * sh.rows;
    Ring<W, 1> ring{{a.x}, {a.ldx}, memory + mine * sh.slot, full, sh, a.T, 2 * a.N, first + mine, step, a.T - 1, mine};
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
    if (fills)
        for (int k = 0; k < sh.depth; ++k)
            ring.fill(k);
    F2 w[8], b[8];
    take_params<W>(a.w, a.fp32, 1.0f, sh.tpr, at, a.N, w);
    take_params<W>(a.b, a.fp32, 0.0f, sh.tpr, at, a.N, b);
    // Elements of the row's warp number i.
    auto count = [&](int i) {
        int n = 0;
        for (int j = 0; j < 16; j += W)
            n += max(0, min(32 * W, a.N - element<W>(sh.tpr, 32 * i, j)));
        return static_cast<float>(n);
    };
    const int warp0 = mine * sh.tpr / 32, warps = sh.tpr / 32;
    const float own = count(warp - warp0), theirs = lane < warps ? count(lane) : 0.0f;
    const float inv_own = own > 0.0f ? 1.0f / own : 0.0f;
    uint16_t *out = a.y + (first + mine) * a.ldy;
    int parity = 0;
    for (int t0 = first; t0 < a.T; t0 += step, parity ^= 1, out += step * a.ldy) {
        const bool ok = mbar_wait(&full[ring.s], ring.phase, &abort_flag, a.wait_limit, &g_status);
        const int t = t0 + mine;
        const bool row = ok && works && t < a.T;
        uint32_t x[8];
        take<W>(ring.at_row(t, 0), sh.tpr, at, a.N, row, x);
        F2 total = pair_of(x[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i)
            total = total + pair_of(x[i]);
        const float2 p = parts(total);
        const float m = warp_sum(p.x + p.y) * inv_own;
        F2 squares = f2(0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const F2 d = centred<W>(x[i], f2(-m), sh.tpr, at, a.N, i);
            squares = fma2(d, d, squares);
        }
        const float2 q = parts(squares);
        const float q_warp = warp_sum(q.x + q.y);
        if (lane == 0)
            slots[parity][warp] = make_float2(m, q_warp);
        // Every thread has taken the stage into registers: it fills again.
        if (__syncthreads_or(!ok)) {
            if (threadIdx.x == 0)
                ring.drain(t0, a.wait_limit);
            return;
        }
        if (fills)
            ring.fill(ring.s);
        ring.next();
        const float2 part = lane < warps && works ? slots[parity][warp0 + lane] : make_float2(0.0f, 0.0f);
        const float mean = warp_sum(theirs * part.x) * inv_n;
        const float d = part.x - mean;
        const float rstd = rsqrtf(warp_sum(theirs > 0.0f ? fmaf(theirs * d, d, part.y) : 0.0f) * inv_n + a.eps);
        if (row) {
            if (at == 0) {
                if (a.mean)
                    a.mean[t] = mean;
                if (a.rstd)
                    a.rstd[t] = rstd;
            }
            F2 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = fma2((pair_of(x[i]) + f2(-mean)) * f2(rstd), w[i], b[i]);
            give<W>(out, sh.tpr, at, a.N, y);
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
constexpr int kRingBytes = 200 << 10;            // of an SM
constexpr int kStreamLeast = 256;                // shorter rows are a warp's
constexpr int kBlockRow = 16384;                 // longest row whose dw and db fit a block's registers

// Elements a thread and threads a row, in whole warps.
int threads_for(int N, int ept) { return ((N + ept - 1) / ept + 31) / 32 * 32; }

// The ring of a call, if its rows are streamed: of a fair length, and enough of them for every block.
bool stream_shape(const NormArgs &a, int arrays, int blocks, int ring_bytes, StreamShape &sh)
{
    if (a.N <= kStreamLeast || a.N > kStreamRow)
        return false;
    sh.tpr = threads_for(a.N, 16);
    sh.rows = kStreamThreads / sh.tpr;
    sh.slot = a.width == 8 ? 2 * a.N : (2 * a.N + 14 + 15) / 16 * 16;
    sh.arrays = arrays;
    const int stage = sh.rows * arrays * sh.slot;
    sh.depth = ring_bytes / stage < kRing ? ring_bytes / stage : kRing;
    return sh.depth >= 2 && a.T >= sh.rows * blocks;
}

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
    StreamShape sh;
    if (stream_shape(a, 1, 2 * kStreamBlocks, kRingBytes / 2, sh)) {
        const int bytes = sh.depth * sh.rows * sh.slot;
        auto kernel = norm_stream_kernel<W == 8 ? 8 : 1>;
        const cudaError_t e = opt_in<norm_stream_kernel<W == 8 ? 8 : 1>>(bytes);
        if (e != cudaSuccess)
            return e;
        return launch_dependent(kernel, dim3(2 * kStreamBlocks), dim3(kStreamThreads), static_cast<size_t>(bytes),
                                stream, a, sh);
    }
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

template <int W>
cudaError_t start_backward_width(NormArgs &a, cudaStream_t stream)
{
    StreamShape sh;
    if (stream_shape(a, a.dres ? 3 : 2, kStreamBlocks, kRingBytes, sh)) {
        a.blocks = kStreamBlocks;                        // (never more than norm_backward_blocks)
        const int ring = sh.depth * sh.rows * sh.arrays * sh.slot, joint = sh.rows * a.N * 4;
        const int bytes = ring > joint ? ring : joint;
        auto kernel = norm_backward_stream_kernel<W == 8 ? 8 : 1>;
        const cudaError_t e = opt_in<norm_backward_stream_kernel<W == 8 ? 8 : 1>>(bytes);
        if (e != cudaSuccess)
            return e;
        return launch_dependent(kernel, dim3(kStreamBlocks), dim3(kStreamThreads),
                                static_cast<size_t>(bytes), stream, a, sh);
    }
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
    switch (a.width) {
    case 8: e = start_backward_width<8>(a, stream); break;
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
