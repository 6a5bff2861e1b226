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

// W parameters from element n on, `missing` where there is no array.  SINGLE: the array does not allow
// accesses of W elements.
template <int W, bool SINGLE = false>
__device__ __forceinline__ void load_param(const void *p, int fp32, int n, float missing, float (&x)[W])
{
    if constexpr (SINGLE) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float one[1];
            load_param<1>(p, fp32, n + i, missing, one);
            x[i] = one[0];
        }
        return;
    }
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
template <int W, int EPT, bool WARP, bool PARAMS, bool SINGLE>
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
                load_param<W, SINGLE>(a.w, a.fp32, n, 1.0f, w);
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
                load_param<W, SINGLE>(a.w, a.fp32, n, 1.0f, w);
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
        if (!a.dw && !a.db)
            return;                                      // (and perhaps no workspace)
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
// The same sums with the rows streamed through shared memory: rings of stages that
// bulk copies fill, as far ahead as shared memory reaches; a row's threads take
// a stage into registers and reduce, and the reduction's barrier is also what frees
// the stage for the next copy.  Bound by HBM.
//
// A thread holds units of eight elements, a warp's side by side (a lane's next
// unit is 32 on), so that accesses are of 16 bytes.  Bulk copies want 16-byte
// boundaries too.  Rows off them (ALIGNED false) are copied from the boundary before to
// the one after, which lie in the array except at its two ends: the first and the
// last row are read straight from memory instead.  A unit is then cut out of two
// neighbouring 16-byte words in shared memory, and stores take the end of the
// lane before's unit and the start of the own, so that they lie on boundaries again.

constexpr int kRing = 8;                         // most stages
constexpr int kStreamThreads = 512;
constexpr int kStreamRow = 8192;                 // longest row

struct StreamShape {
    int tpr;                    // threads of a row, whole warps
    int rows;                   // rows of a stage
    int slot;                   // bytes of a row in the ring
    int arrays;
    int depth;                  // stages
};

__device__ int g_status = 0;                     // bounded waits that ran out

// First element of a thread's unit v of UNITS.
template <int UNITS>
__device__ __forceinline__ int unit_at(int at, int v)
{
    return ((at >> 5) * UNITS * 32 + v * 32 + (at & 31)) * 8;
}

// Two elements, as they lie in a word.
__device__ __forceinline__ F2 pair_of(uint32_t w) { return f2(bf16_lo(w), bf16_hi(w)); }

__device__ __forceinline__ uint32_t word_of(F2 v)
{
    const float2 p = parts(v);
    const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// Words k .. k + 3 of eight, half a word on if shift is 16.
__device__ __forceinline__ void cut(const uint32_t (&w)[8], int k, uint32_t shift, uint32_t (&out)[4])
{
    switch (k) {                                         // uniform
    case 0:
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[i] = __funnelshift_r(w[i], w[i + 1], shift);
        break;
    case 1:
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[i] = __funnelshift_r(w[i + 1], w[i + 2], shift);
        break;
    case 2:
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[i] = __funnelshift_r(w[i + 2], w[i + 3], shift);
        break;
    default:
#pragma unroll
        for (int i = 0; i < 4; ++i)
            out[i] = __funnelshift_r(w[i + 3], w[i + 4], shift);
        break;
    }
}

// A thread's units of a row, zeros past its end.  The row's first element is number `ahead` of the
// 16-byte word at p in shared memory, or the row is at `direct` in memory.
template <bool ALIGNED, int UNITS>
__device__ __forceinline__ void take(const uint8_t *p, uint32_t ahead, const uint16_t *direct, int at, int N, uint32_t (&w)[4 * UNITS])
{
#pragma unroll
    for (int v = 0; v < UNITS; ++v) {
        const int n = unit_at<UNITS>(at, v);
        uint32_t out[4] = {0u, 0u, 0u, 0u};
        if (n < N) {
            if (!ALIGNED && direct) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (n + i < N)
                        out[i / 2] |= static_cast<uint32_t>(direct[n + i]) << (16 * (i & 1));
            } else {
                const uint4 lo = *reinterpret_cast<const uint4 *>(p + 2 * n);
                if (ALIGNED || ahead == 0u) {
                    out[0] = lo.x;
                    out[1] = lo.y;
                    out[2] = lo.z;
                    out[3] = lo.w;
                } else {
                    const uint4 hi = *reinterpret_cast<const uint4 *>(p + 2 * n + 16);
                    const uint32_t both[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    cut(both, static_cast<int>(ahead >> 1), 16u * (ahead & 1u), out);
                }
                if (!ALIGNED && n + 8 > N) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        out[i] = n + 2 * i >= N ? 0u : n + 2 * i + 1 >= N ? out[i] & 0xFFFFu : out[i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[4 * v + i] = out[i];
    }
}

// A thread's units to a row off 16-byte boundaries, or one that ends inside a unit.
template <int UNITS>
__device__ __forceinline__ void give_anywhere(uint16_t *p, int at, int N, const uint32_t (&w)[4 * UNITS])
{
    const int lane = at & 31;
    const uint32_t ahead = (reinterpret_cast<uintptr_t>(p) & 15u) / 2u;
    // The lane's 16-byte word of memory starts `ahead` elements before its unit: in the unit before,
    // which is the lane before's, or for the first lane the last one's of the v before.
#pragma unroll
    for (int v = 0; v < UNITS; ++v) {
        const int n = unit_at<UNITS>(at, v), e0 = n - static_cast<int>(ahead);
        uint32_t both[8], out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            both[4 + i] = w[4 * v + i];
            const uint32_t sent = v > 0 && lane == 31 ? w[v > 0 ? 4 * v - 4 + i : 0] : w[4 * v + i];
            both[i] = __shfl_sync(kFull, sent, (lane + 31) & 31);
        }
        if (ahead == 0u) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                out[i] = both[4 + i];
        } else {
            cut(both, static_cast<int>((8u - ahead) >> 1), 16u * (ahead & 1u), out);
        }
        const int begin = v == 0 && lane == 0 ? n : e0;  // what comes before a warp's first unit is the warp before's
        if (begin == e0 && e0 + 8 <= N) {
            *reinterpret_cast<uint4 *>(p + e0) = make_uint4(out[0], out[1], out[2], out[3]);
        } else if (begin < N) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e0 + i >= begin && e0 + i < N)
                    p[e0 + i] = static_cast<uint16_t>(out[i / 2] >> (16 * (i & 1)));
        }
    }
    // And the end of its last unit, behind the last lane's word.
    const int n = unit_at<UNITS>(at, UNITS - 1);
    if (lane == 31 && n + 8 - static_cast<int>(ahead) < N) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= 8 - static_cast<int>(ahead) && n + i < N)
                p[n + i] = static_cast<uint16_t>(w[4 * (UNITS - 1) + i / 2] >> (16 * (i & 1)));
    }
}

// A thread's units to a row; all lanes of a warp call it.
template <bool ALIGNED, int UNITS>
__device__ __forceinline__ void give(uint16_t *p, int at, int N, const uint32_t (&w)[4 * UNITS])
{
    if constexpr (ALIGNED) {
#pragma unroll
        for (int v = 0; v < UNITS; ++v) {
            const int n = unit_at<UNITS>(at, v);
            if (n < N)
                *reinterpret_cast<uint4 *>(p + n) = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
        }
    } else {
        give_anywhere<UNITS>(p, at, N, w);
    }
}

// The ring of one block, or of one team of it.  Group k is the rows first + k * step .. + rows - 1;
// stage k % depth holds it.  (Row numbers past the last stay below 2^31: T does by more than a step.)
template <bool ALIGNED, int ARRAYS>
struct Ring {
    const uint16_t *array[ARRAYS];
    int64_t ld[ARRAYS];
    uint8_t *memory;            // of the thread's row in stage 0
    uint64_t *full;
    StreamShape sh;
    int T, bytes;               // bytes of a row
    int t;                      // the row that is filled next: the thread's
    int step, last;             // last: no group starts behind it
    int mine;                   // the thread's row of a stage
    int s = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ int stage_bytes() const { return sh.rows * sh.arrays * sh.slot; }
    __device__ __forceinline__ bool direct(int row) const { return !ALIGNED && (row == 0 || row == T - 1); }
    __device__ __forceinline__ static uint32_t ahead(const uint16_t *p) { return ALIGNED ? 0u : reinterpret_cast<uintptr_t>(p) & 15u; }

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
                size[i] = ALIGNED ? bytes : (ahead(p[i]) + bytes + 15u) / 16u * 16u;
                total += size[i];
            }
        mbar_arrive_expect_tx(&full[stage], total);
#pragma unroll
        for (int i = 0; i < ARRAYS; ++i)
            if (i < sh.arrays)
                bulk_load(memory + stage * stage_bytes() + i * sh.slot, reinterpret_cast<const uint8_t *>(p[i]) - ahead(p[i]), size[i],
                          &full[stage], policy);
    }
    // The thread's units of array i's row `row`, which the present stage holds.
    template <int UNITS>
    __device__ __forceinline__ void read(int row, int i, int at, int N, uint32_t (&w)[4 * UNITS]) const
    {
        const uint16_t *p = array[i] + row * ld[i];
        take<ALIGNED, UNITS>(memory + s * stage_bytes() + i * sh.slot, ahead(p) / 2u, direct(row) ? p : nullptr, at, N, w);
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

// The gradients: one block of 512 threads to an SM, as many rows a stage as they
// hold with two units each, all of a block's in step.
template <bool ALIGNED>
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
    Ring<ALIGNED, 3> ring{{a.x, a.dy, a.dres}, {a.ldx, a.lddy, a.ldr}, memory + mine * sh.arrays * sh.slot, full, sh, a.T, 2 * a.N,
                          first + mine, step, a.T - 1, mine};
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
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = unit_at<2>(at, i / 4) + 2 * (i % 4);
        float lo[1] = {0.0f}, hi[1] = {0.0f};
        if (n < a.N)
            load_param<1>(a.w, a.fp32, n, 1.0f, lo);
        if (n + 1 < a.N)
            load_param<1>(a.w, a.fp32, n + 1, 1.0f, hi);
        w[i] = f2(lo[0], hi[0]);
        dw[i] = db[i] = f2(0.0f);
    }
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
        const bool row = works && t < a.T;               // (of whole warps)
        uint32_t x[8], dy[8], res[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = dy[i] = res[i] = 0u;
        if (row) {
            ring.template read<2>(t, 0, at, a.N, x);
            ring.template read<2>(t, 1, at, a.N, dy);
            if (a.dres)
                ring.template read<2>(t, 2, at, a.N, res);
        }
        const F2 minus_m = f2(row ? -mean : 0.0f), r = f2(row ? rstd : 0.0f);
        if (works && t + step < a.T) {
            mean = a.mean[t + step];
            rstd = a.rstd[t + step];
        }
        // (Past the row's end dy is 0.)
        F2 s1 = f2(0.0f), s2 = f2(0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const F2 xhat = (pair_of(x[i]) + minus_m) * r, d = pair_of(dy[i]), g = d * w[i];
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
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const F2 xhat = (pair_of(x[i]) + minus_m) * r;
                F2 v = r * fma2(xhat, m2, fma2(pair_of(dy[i]), w[i], m1));
                if (a.dres)
                    v = v + pair_of(res[i]);
                y[i] = word_of(v);
            }
            give<ALIGNED, 2>(out, at, a.N, y);
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
                const int n = unit_at<2>(at, i / 8) + i % 8;
                if (n < a.N)
                    joint[mine * a.N + n] = i & 1 ? v.y : v.x;
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

// The norm itself: four units a thread, teams of a row's threads that go round
// rings of their own and meet at barriers of their own; the parameters are in shared
// memory as fp32.  One barrier a row: a warp takes the mean of its elements and
// the squares of their differences from that, and the row's follow from the warps' as
//   m = sum n_i m_i / N,  sum (x - m)^2 = sum [q_i + n_i (m_i - m)^2],
// sums of positive terms throughout.
constexpr int kNormThreads = 768;
constexpr int kTeams = kNormThreads / 32;

// Whether any of a team's threads says so, and a barrier for them.
__device__ __forceinline__ bool team_any(bool yes, int team, int threads)
{
    int any;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.s32 p, %1, 0;\n\t"
                 "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
                 "selp.s32 %0, 1, 0, q;\n\t}"
                 : "=r"(any)
                 : "r"(static_cast<int>(yes)), "r"(team + 1), "r"(threads)
                 : "memory");
    return any != 0;
}

template <bool ALIGNED>
__global__ void __launch_bounds__(kNormThreads, 1) norm_stream_kernel(const __grid_constant__ NormArgs a, const StreamShape sh)
{
    extern __shared__ __align__(128) uint8_t memory[];
    __shared__ uint64_t full[kTeams][kRing];
    __shared__ float2 slots[kTeams][2][8];
    __shared__ int abort_flag[kTeams];
    const int teams = sh.rows;
    const int team = static_cast<int>(threadIdx.x) / sh.tpr;
    const int at = static_cast<int>(threadIdx.x) - team * sh.tpr;
    const int lane = threadIdx.x & 31, warp = at >> 5, warps = sh.tpr >> 5;
    const int units = (a.N + 7) / 8;
    // w, then b: the first four of every unit, then the other four, so that neighbouring lanes' reads are neighbours.
    float *params = reinterpret_cast<float *>(memory);
    const float inv_n = 1.0f / static_cast<float>(a.N);
    if (team < teams && at == 0) {
        for (int s = 0; s < sh.depth; ++s)
            mbar_init(&full[team][s], 1);
        abort_flag[team] = 0;
        fence_mbar_init();
    }
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    for (int n = threadIdx.x; n < 8 * units; n += kNormThreads) {
        float w[1] = {0.0f}, b[1] = {0.0f};
        if (n < a.N) {
            load_param<1>(a.w, a.fp32, n, 1.0f, w);
            load_param<1>(a.b, a.fp32, n, 0.0f, b);
        }
        const int to = ((n >> 2 & 1) * units + (n >> 3)) * 4 + (n & 3);
        params[to] = w[0];
        params[8 * units + to] = b[0];
    }
    __syncthreads();
    if (team >= teams)
        return;
    // A team is a block of its own in the ring's terms: one row a stage.
    StreamShape mine = sh;
    mine.rows = 1;
    const int step = static_cast<int>(gridDim.x) * teams, first = static_cast<int>(blockIdx.x) * teams + team;
    Ring<ALIGNED, 1> ring{{a.x}, {a.ldx}, memory + 64 * units + team * sh.depth * sh.slot, full[team], mine, a.T, 2 * a.N, first, step,
                          a.T - 1, 0};
    if (at == 0)
        for (int k = 0; k < sh.depth; ++k)
            ring.fill(k);
    // Elements of the row's warp number i.
    auto count = [&](int i) { return static_cast<float>(max(0, min(1024, a.N - 1024 * i))); };
    const float own = count(warp), theirs = (lane & 7) < warps ? count(lane & 7) : 0.0f;
    const float inv_own = own > 0.0f ? 1.0f / own : 0.0f;
    uint16_t *out = a.y + first * a.ldy;
    int parity = 0;
    for (int t = first; t < a.T; t += step, parity ^= 1, out += step * a.ldy) {
        const bool ok = mbar_wait(&full[team][ring.s], ring.phase, &abort_flag[team], a.wait_limit, &g_status);
        F2 x[16];
        {
            uint32_t words[16];
            ring.template read<4>(t, 0, at, a.N, words);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[i] = pair_of(words[i]);
        }
        F2 total = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i)
            total = total + x[i];
        const float2 p = parts(total);
        const float m = warp_sum(p.x + p.y) * inv_own;
        const F2 minus_m = f2(-m);
        F2 squares = f2(0.0f);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int n = unit_at<4>(at, v);
            if (n + 8 <= a.N) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const F2 d = x[4 * v + i] + minus_m;
                    squares = fma2(d, d, squares);
                }
            } else if (!ALIGNED && n < a.N) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 d = parts(x[4 * v + i] + minus_m);
                    const F2 e = f2(n + 2 * i < a.N ? d.x : 0.0f, n + 2 * i + 1 < a.N ? d.y : 0.0f);
                    squares = fma2(e, e, squares);
                }
            }
        }
        const float2 q = parts(squares);
        float2 part = make_float2(m, warp_sum(q.x + q.y));
        if (warps > 1) {
            if (lane == 0)
                slots[team][parity][warp] = part;
            // Every thread has taken the stage into registers: it fills again.
            if (team_any(!ok, team, sh.tpr)) {
                if (at == 0)
                    ring.drain(t, a.wait_limit);
                return;
            }
            part = (lane & 7) < warps ? slots[team][parity][lane & 7] : make_float2(0.0f, 0.0f);
        } else if (__any_sync(kFull, !ok)) {
            if (at == 0)
                ring.drain(t, a.wait_limit);
            return;
        }
        if (at == 0)
            ring.fill(ring.s);
        ring.next();
        float mean = part.x, var = part.y * inv_n;
        if (warps > 1) {
            mean = theirs * part.x;
#pragma unroll
            for (int d = 1; d < 8; d <<= 1)
                mean += __shfl_xor_sync(kFull, mean, d);
            mean *= inv_n;
            const float d = part.x - mean;
            var = theirs > 0.0f ? fmaf(theirs * d, d, part.y) : 0.0f;
#pragma unroll
            for (int d = 1; d < 8; d <<= 1)
                var += __shfl_xor_sync(kFull, var, d);
            var *= inv_n;
        }
        const float rstd = rsqrtf(var + a.eps);
        if (at == 0) {
            if (a.mean)
                a.mean[t] = mean;
            if (a.rstd)
                a.rstd[t] = rstd;
        }
        const F2 centre = f2(-mean), r = f2(rstd);
        uint32_t y[16];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int unit = unit_at<4>(at, v) / 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = w;
                if (unit < units) {
                    w = *reinterpret_cast<const float4 *>(params + (h * units + unit) * 4);
                    b = *reinterpret_cast<const float4 *>(params + 8 * units + (h * units + unit) * 4);
                }
                y[4 * v + 2 * h] = word_of(fma2((x[4 * v + 2 * h] + centre) * r, f2(w.x, w.y), f2(b.x, b.y)));
                y[4 * v + 2 * h + 1] = word_of(fma2((x[4 * v + 2 * h + 1] + centre) * r, f2(w.z, w.w), f2(b.z, b.w)));
            }
        }
        give<ALIGNED, 4>(out, at, a.N, y);
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
constexpr int kRingBytes = 216 << 10;            // of an SM: the most dynamic shared memory of a streamed launch
constexpr int kStreamLeast = 256;                // shorter rows are a warp's
constexpr int kBlockRow = 16384;                 // longest row whose dw and db fit a block's registers

// Elements a thread and threads a row, in whole warps.
int threads_for(int N, int ept) { return ((N + ept - 1) / ept + 31) / 32 * 32; }

// The ring of a call, if its rows are streamed: of a fair length, and enough of them for every block.
bool stream_shape(const NormArgs &a, bool backward, StreamShape &sh)
{
    if (a.N <= kStreamLeast || a.N > kStreamRow)
        return false;
    sh.tpr = threads_for(a.N, backward ? 16 : 32);
    sh.rows = (backward ? kStreamThreads : kNormThreads) / sh.tpr;
    sh.slot = a.width == 8 ? 2 * a.N : (2 * a.N + 14 + 15) / 16 * 16 + 16;   // (the last unit's second word)
    sh.arrays = !backward ? 1 : a.dres ? 3 : 2;
    const int stage = sh.rows * sh.arrays * sh.slot;
    const int room = kRingBytes - (backward ? 0 : (a.N + 7) / 8 * 64);
    sh.depth = room / stage < kRing ? room / stage : kRing;
    // Against the kernels above: aligned rows of the norm gain from four full rounds of stages on (2432 x 2048:
    // 6.2 us there, 7.8 here); others, which those take element by element, soon (608 x 1501: 10.1 there,
    // 6.4 here); its gradients of more than 1024 soon too, as each of its blocks writes one partial
    // sum for all its rows (304 x 2048: 14.2 there, 9.7 here; 1216 x 701: 10.7 and 10.5).
    const int full = sh.rows * kStreamBlocks;            // every block's first stage
    const int least = backward ? (a.N > kWarpRow ? full / 4 : full) : a.width == 8 ? 4 * full : full / 4;
    return sh.depth >= 2 && a.T >= least;
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
    // time for one row; with narrow accesses up to more rows, whose code for 32 is long (608 x 701: 8.1 us
    // with 32, 4.8 with eight).
    const bool many = a.T > (W < 8 ? 8 : 2) * sms;
    StreamShape sh;
    if (a.T > 2 * sms && stream_shape(a, false, sh)) {
        const int bytes = sh.depth * sh.rows * sh.slot + (a.N + 7) / 8 * 64;
        auto kernel = norm_stream_kernel<W == 8>;
        const cudaError_t e = opt_in<norm_stream_kernel<W == 8>, kRingBytes>();
        if (e != cudaSuccess)
            return e;
        return launch_dependent(kernel, dim3(kStreamBlocks), dim3(kNormThreads), static_cast<size_t>(bytes), stream, a,
                                sh);
    }
    if (a.N <= kWarpRow && many)
        return a.N <= 256 ? start_norm<W, 8, true>(a, sms, stream) : start_norm<W, 32, true>(a, sms, stream);
    if (a.N <= 8192 && !many)
        return start_norm<W, 8, false>(a, sms, stream);
    return start_norm<W, 32, false>(a, sms, stream);
}

// Blocks that share T rows, so many at a time each.
int backward_blocks(int T, int rows)
{
    const int64_t need = (static_cast<int64_t>(T) + rows - 1) / rows, most = 2 * 152;
    return static_cast<int>(need < 1 ? 1 : need < most ? need : most);
}

template <int W, int EPT, bool WARP, bool PARAMS>
cudaError_t start_backward(const NormArgs &a, cudaStream_t stream)
{
    const int threads = WARP ? kRowWarps * 32 : threads_for(a.N, EPT);
    // (a kernel of its own for each way to read w: both in one take up to 38 registers more, and from the
    // blocks of an SM)
    auto start = [&](auto kernel) {
        return launch_dependent(kernel, dim3(static_cast<unsigned>(a.blocks)), dim3(static_cast<unsigned>(threads)), 0, stream, a);
    };
    if constexpr (W > 1)
        if (a.single_w)
            return start(norm_backward_kernel<W, EPT, WARP, PARAMS, true>);
    return start(norm_backward_kernel<W, EPT, WARP, PARAMS, false>);
}

template <int W>
cudaError_t start_backward_width(NormArgs &a, cudaStream_t stream)
{
    StreamShape sh;
    // A few rows of middling length: eight elements a thread, a block each, while their partial sums are
    // small (152 x 2048: 8.6 us, streamed 10.0; 304 x 2048: 11.9 and 9.8).
    const bool few_long = a.N > kWarpRow && a.N <= 4096 && static_cast<int64_t>(a.T) * a.N <= 3 << 17;
    if (!few_long && stream_shape(a, true, sh)) {
        const int stages = (a.T + sh.rows - 1) / sh.rows;
        a.blocks = stages < kStreamBlocks ? stages : kStreamBlocks;      // (never more than norm_backward_blocks)
        const int ring = sh.depth * sh.rows * sh.arrays * sh.slot, joint = sh.rows * a.N * 4;
        const int bytes = ring > joint ? ring : joint;
        auto kernel = norm_backward_stream_kernel<W == 8>;
        const cudaError_t e = opt_in<norm_backward_stream_kernel<W == 8>, kRingBytes>();
        if (e != cudaSuccess)
            return e;
        return launch_dependent(kernel, dim3(static_cast<unsigned>(a.blocks)), dim3(kStreamThreads),
                                static_cast<size_t>(bytes), stream, a, sh);
    }
    // A row of up to 1024 is a warp's where there are many: fewer partial sums.  Few are a block's each,
    // eight elements a thread: a lane's 32 elements in accesses of two bytes are long code, which
    // comes cold to every call.  Rows of 1001: 7.4 us against 13.6 for 300, 13.5 against 14.4 for 1200;
    // of 1024: 4.3 against 5.5 for 20, 6.0 against 5.7 for 100, 8.7 against 6.1 for 300.
    const bool few = a.T <= (W < 4 ? 8 * 152 : 76);
    if (a.N <= kWarpRow && a.N > 256 && few)
        return start_backward<W, 8, false, true>(a, stream);
    if (a.N <= kWarpRow) {
        a.blocks = backward_blocks(a.T, kRowWarps);
        return a.N <= 256 ? start_backward<W, 8, true, true>(a, stream) : start_backward<W, 32, true, true>(a, stream);
    }
    if (few_long)
        return start_backward<W, 8, false, true>(a, stream);
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

int norm_backward_blocks(int T, int N) { return backward_blocks(T, N <= 256 ? kRowWarps : 1); }

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
