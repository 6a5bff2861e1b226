// Gated join of a token's expert rows with the norms around the residual stream.
#include <cuda_bf16.h>

#include "expert.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace mxfp4 {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ int g_status = 0;                     // bounded waits that ran out

// ------------------------------------------------------------------- join --
//
//   b = sum_j gates[t, j] Y[slot_row[t, j]]          (fp32, slots in order)
//   b = b rsqrt(mean b^2 + eps) w_post               with w_post
//   h = res_scale resid[t] + out_scale b             -> H, one rounding
//   n = h rsqrt(mean h^2 + eps) w_pre                -> Nrm, one rounding, from the fp32 h
//
// One block per token (grid-stride), the row in registers between the two
// sums, so that every input is read once.  b, the sums and h are fp32; the sum
// over slots keeps their order, so a result does not depend on the launch.
//
// Three forms.  Few tokens: as many threads per token as have eight elements
// each, four rows in flight; the latency of two dependent loads and of the sums
// bounds it (8 tokens x 8 rows of 7168: 3.8 us a call, an empty one's 2.9).  Rows off 16-byte boundaries: narrower units.  Many tokens with long
// rows: a ring that streams rows ahead, bound by HBM.

constexpr int kCombineThreads = 512;
constexpr int kCombineMaxVec = 8;                // 8-element vectors of one thread

__device__ __forceinline__ uint4 raw8(const uint16_t *p, int n) { return *reinterpret_cast<const uint4 *>(p + n); }

__device__ __forceinline__ void store8(uint16_t *p, int n, const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    *reinterpret_cast<uint4 *>(p + n) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int W>
__device__ __forceinline__ void store_unit(uint16_t *p, const float (&x)[W])
{
    if constexpr (W == 8) {
        store8(p, 0, x);
    } else if constexpr (W == 1) {
        const __nv_bfloat16 v = __float2bfloat16_rn(x[0]);
        *p = *reinterpret_cast<const uint16_t *>(&v);
    } else {
        uint32_t w[W / 2];
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        if constexpr (W == 4)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(p) = w[0];
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// Sum over the block; every thread gets it.  slot: one float per warp.  The
// callers alternate slots so that the next call's writes do not meet this one's
// reads.
__device__ __forceinline__ float block_sum(float v, float *slot)
{
    const int lane = threadIdx.x & 31, warps = static_cast<int>(blockDim.x) >> 5;
    v = warp_sum(v);
    if (lane == 0)
        slot[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? slot[lane] : 0.0f);
}

// 1 / sqrt(mean + eps) from the sum of squares.
__device__ __forceinline__ float inverse_rms(const CombineArgs &a, float ss)
{
    return rsqrtf(ss / static_cast<float>(a.N) + a.eps);
}

__device__ __forceinline__ float pick8(const uint4 &v, int i)
{
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return i & 1 ? bf16_hi(w) : bf16_lo(w);
}

// W elements as they lie in memory, and element i of them.
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
__device__ __forceinline__ float pick(const typename UnitOf<W>::T &v, int i)
{
    if constexpr (W == 8)
        return pick8(v, i);
    else if constexpr (W == 4)
        return i & 1 ? bf16_hi(i < 2 ? v.x : v.y) : bf16_lo(i < 2 ? v.x : v.y);
    else
        return i & 1 ? bf16_hi(v) : bf16_lo(v);
}

template <int W>
__device__ __forceinline__ void load_unit(const uint16_t *p, float (&x)[W])
{
    const typename UnitOf<W>::T v = *reinterpret_cast<const typename UnitOf<W>::T *>(p);
#pragma unroll
    for (int i = 0; i < W; ++i)
        x[i] = pick<W>(v, i);
}

// VPT 8-element vectors per thread, JC slots' rows in flight together.  8192
// tokens x 4 rows of 1024, below the ring's sizes: 26 us, 118 MB, 4.5 TB/s.
// Few tokens run on up to MAXT = 1024 threads each, the shortest time for one.
template <int VPT, int JC, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == kCombineThreads && VPT <= 2 ? 2 : 1) combine_kernel(const __grid_constant__ CombineArgs a)
{
    __shared__ float slots[4][MAXT / 32];
    if (!a.early)
        pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    bool waited = !a.early;
    int parity = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 2) {
        float b[VPT][8];
        uint4 res[VPT];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = (v * blockDim.x + threadIdx.x) * 8;
            res[v] = make_uint4(0u, 0u, 0u, 0u);
            if (VPT < 8 && a.resid && n < a.N)             // early, where registers allow
                res[v] = raw8(a.resid + static_cast<int64_t>(t) * a.ldr, n);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                b[v][i] = 0.0f;
        }
        for (int j0 = 0; j0 < a.k; j0 += JC) {
            int row[JC];
            float g[JC];
            uint4 y[JC][VPT];
#pragma unroll
            for (int j = 0; j < JC; ++j) {
                const int64_t at = static_cast<int64_t>(t) * a.k + j0 + j;
                row[j] = j0 + j < a.k ? (a.slot_row ? a.slot_row[at] : t) : -1;
                g[j] = j0 + j < a.k && a.gates ? a.gates[at] : 1.0f;
            }
            if (!waited) {
                pdl_wait_prerequisites();
                waited = true;
            }
#pragma unroll
            for (int j = 0; j < JC; ++j)
#pragma unroll
                for (int v = 0; v < VPT; ++v) {
                    const int n = (v * blockDim.x + threadIdx.x) * 8;
                    if (row[j] >= 0 && row[j] < a.rows && n < a.N)
                        y[j][v] = raw8(a.Y + static_cast<int64_t>(row[j]) * a.ldy, n);
                }
#pragma unroll
            for (int j = 0; j < JC; ++j) {
                if (row[j] < 0 || row[j] >= a.rows)
                    continue;                              // block-uniform
#pragma unroll
                for (int v = 0; v < VPT; ++v)
                    if ((v * blockDim.x + threadIdx.x) * 8 < a.N) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            b[v][i] = fmaf(g[j], pick8(y[j][v], i), b[v][i]);
                    }
            }
        }
        if (a.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ss = fmaf(b[v][i], b[v][i], ss);
            ss = block_sum(ss, slots[parity]);
            const float r = inverse_rms(a, ss);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int n = (v * blockDim.x + threadIdx.x) * 8;
                if (n < a.N) {
                    const uint4 w = raw8(a.w_post, n);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        b[v][i] = b[v][i] * r * pick8(w, i);
                }
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = (v * blockDim.x + threadIdx.x) * 8;
            if (n < a.N) {
                if (VPT == 8 && a.resid)
                    res[v] = raw8(a.resid + static_cast<int64_t>(t) * a.ldr, n);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    b[v][i] = a.resid ? fmaf(a.out_scale, b[v][i], a.res_scale * pick8(res[v], i)) : a.out_scale * b[v][i];
                    ss = fmaf(b[v][i], b[v][i], ss);
                }
                if (a.H)
                    store8(a.H + static_cast<int64_t>(t) * a.ldh, n, b[v]);
            }
        }
        if (a.Nrm) {
            ss = block_sum(ss, slots[parity + 1]);
            const float r = inverse_rms(a, ss);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int n = (v * blockDim.x + threadIdx.x) * 8;
                if (n < a.N) {
                    float y[8];
                    if (a.w_pre) {
                        const uint4 w = raw8(a.w_pre, n);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            y[i] = b[v][i] * r * pick8(w, i);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            y[i] = b[v][i] * r;
                    }
                    store8(a.Nrm + static_cast<int64_t>(t) * a.ldn, n, y);
                }
            }
        }
    }
}

// Rows that do not allow 16-byte accesses (an odd length, stride or start): the
// threads take units of W elements in turn, so that a warp's accesses are
// contiguous whatever W is.  THREADS threads with E elements each (both fixed, so
// that a row's units are one pointer and constants); JC rows in flight together.
// 6437 tokens x 3 rows of 1196: 22 to 25 us, 92 MB, bound by instructions.
template <int W, int E, int JC, int THREADS, int MINB>
__global__ void __launch_bounds__(THREADS, MINB) combine_narrow_kernel(const __grid_constant__ CombineArgs a)
{
    constexpr int PER = E / W;
    __shared__ float slots[4][THREADS / 32];
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    int parity = 0;
    constexpr int step = THREADS * W;
    const int n0 = static_cast<int>(threadIdx.x) * W;
    // Lane j holds slot j of the token at hand, and already of the next one.
    const int lane = static_cast<int>(threadIdx.x) & 31;
    auto look_up = [&](int t, int &row, float &g) {
        row = -1;
        g = 1.0f;
        if (t < a.T && lane < a.k) {
            const int64_t at = static_cast<int64_t>(t) * a.k + lane;
            row = a.slot_row ? a.slot_row[at] : t;
            if (row >= a.rows)
                row = -1;
            if (a.gates)
                g = a.gates[at];
        }
    };
    int next_row;
    float next_g;
    look_up(blockIdx.x, next_row, next_g);
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 2) {
        const int slot_row = next_row;
        const float slot_g = next_g;
        look_up(t + static_cast<int>(gridDim.x), next_row, next_g);
        float b[PER][W];
#pragma unroll
        for (int u = 0; u < PER; ++u)
#pragma unroll
            for (int i = 0; i < W; ++i)
                b[u][i] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += JC) {
            int row[JC];
            float g[JC];
            float x[JC][PER][W];
#pragma unroll
            for (int j = 0; j < JC; ++j) {
                row[j] = __shfl_sync(kFull, slot_row, j0 + j);
                g[j] = __shfl_sync(kFull, slot_g, j0 + j);
            }
#pragma unroll
            for (int j = 0; j < JC; ++j) {
                if (row[j] < 0)
                    continue;                              // block-uniform
                const uint16_t *y = a.Y + static_cast<int64_t>(row[j]) * a.ldy + n0;
#pragma unroll
                for (int u = 0; u < PER; ++u)
                    if (n0 + u * step < a.N)
                        load_unit<W>(y + u * step, x[j][u]);
            }
#pragma unroll
            for (int j = 0; j < JC; ++j) {
                if (row[j] < 0)
                    continue;
#pragma unroll
                for (int u = 0; u < PER; ++u)
                    if (n0 + u * step < a.N) {
#pragma unroll
                        for (int i = 0; i < W; ++i)
                            b[u][i] = fmaf(g[j], x[j][u][i], b[u][i]);
                    }
            }
        }
        if (a.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int u = 0; u < PER; ++u)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    ss = fmaf(b[u][i], b[u][i], ss);
            ss = block_sum(ss, slots[parity]);
            const float r = inverse_rms(a, ss);
#pragma unroll
            for (int u = 0; u < PER; ++u)
                if (n0 + u * step < a.N) {
                    float w[W];
                    load_unit<W>(a.w_post + n0 + u * step, w);
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        b[u][i] = b[u][i] * r * w[i];
                }
        }
        float ss = 0.0f;
#pragma unroll
        for (int u = 0; u < PER; ++u)
            if (n0 + u * step < a.N) {
                float x[W];
                if (a.resid)
                    load_unit<W>(a.resid + static_cast<int64_t>(t) * a.ldr + n0 + u * step, x);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    b[u][i] = a.resid ? fmaf(a.out_scale, b[u][i], a.res_scale * x[i]) : a.out_scale * b[u][i];
                    ss = fmaf(b[u][i], b[u][i], ss);
                }
                if (a.H)
                    store_unit<W>(a.H + static_cast<int64_t>(t) * a.ldh + n0 + u * step, b[u]);
            }
        if (a.Nrm) {
            ss = block_sum(ss, slots[parity + 1]);
            const float r = inverse_rms(a, ss);
#pragma unroll
            for (int u = 0; u < PER; ++u)
                if (n0 + u * step < a.N) {
                    float y[W];
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        y[i] = b[u][i] * r;
                    if (a.w_pre) {
                        float w[W];
                        load_unit<W>(a.w_pre + n0 + u * step, w);
#pragma unroll
                        for (int i = 0; i < W; ++i)
                            y[i] *= w[i];
                    }
                    store_unit<W>(a.Nrm + static_cast<int64_t>(t) * a.ldn + n0 + u * step, y);
                }
        }
    }
}

// The same for long prefills, where the sums' barriers must not leave HBM
// idle: persistent blocks, whose last warps stream the tokens' rows (the taken
// rows of Y, then the residual row) into a ring of whole rows in shared memory
// with bulk copies, as far ahead as the ring holds, while the others work on the
// token at hand.  Bound by HBM: 8192 tokens x 4 rows of 8192 move 940 MB in
// 144 us, 98 % of a plain copy's rate.
//
// W < 8 is for rows off 16-byte boundaries.  Such a row is copied with the rest
// of its first and last 16 bytes, which belong to the tensor's other rows; the
// entry notes where the row begins.  Only the tensor's first and last row may
// have no such neighbours: there the warp sets down the elements beside the
// whole 16-byte parts itself, so nothing outside the tensor is read.
constexpr int kRingMaxRows = 32;
constexpr int kRingBytes = 200 * 1024;           // of an SM's blocks together

struct RingMeta {
    uint64_t full[kRingMaxRows];
    uint64_t empty[kRingMaxRows];
    float gate[kRingMaxRows];
    int last[kRingMaxRows];                      // 1: the token's last entry (its residual row, or nothing)
    int shift[kRingMaxRows];                     // the row's first byte
    float slots[4][16];
    int abort_flag;
};

__host__ __device__ constexpr uint32_t ring_pitch(int N, int W)
{
    return (static_cast<uint32_t>(N) * 2 + (W < 8 ? 14u : 0u) + 127u) / 128u * 128u;
}

template <int THREADS>
__device__ __forceinline__ float ring_sum(float v, float *slot)
{
    const int lane = threadIdx.x & 31;
    v = warp_sum(v);
    if (lane == 0)
        slot[threadIdx.x >> 5] = v;
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
    return warp_sum(lane < THREADS / 32 ? slot[lane] : 0.0f);
}

// PER units of W elements per thread, unit u at element (u * THREADS + thread) * W.
template <int W, int PER, int THREADS, int BLOCKS, int LOADERS>
__global__ void __launch_bounds__(THREADS + 32 * LOADERS, BLOCKS) combine_ring_kernel(const __grid_constant__ CombineArgs a, int depth)
{
    using Unit = typename UnitOf<W>::T;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ RingMeta m;
    const uint32_t row_bytes = static_cast<uint32_t>(a.N) * 2;
    const uint32_t pitch = ring_pitch(a.N, W);
    volatile int *abort_flag = &m.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < depth; ++s) {
            mbar_init(&m.full[s], 1);
            mbar_init(&m.empty[s], THREADS / 32);
        }
        m.abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    if (warp >= THREADS / 32) {
        const int loader = warp - THREADS / 32;
        const uint64_t once = l2_policy_evict_first();
        int entry = 0;                                     // of this block's, in order
        bool ok = true;
        auto look_up = [&](int t, int &row, float &g) {
            row = -1;
            g = 1.0f;
            if (t < a.T && lane < a.k) {
                const int64_t at = static_cast<int64_t>(t) * a.k + lane;
                row = a.slot_row ? a.slot_row[at] : t;
                if (row >= a.rows)
                    row = -1;
                if (a.gates)
                    g = a.gates[at];
            }
        };
        int row, next_row;
        float g, next_g;
        look_up(blockIdx.x, next_row, next_g);
        for (int t = blockIdx.x; t < a.T && ok; t += gridDim.x) {
            row = next_row;
            g = next_g;
            look_up(t + gridDim.x, next_row, next_g);      // a token ahead
            const uint32_t taken = __ballot_sync(kFull, row >= 0);
            const int entries = __popc(taken) + 1;
            uint32_t left = taken;
            for (int i = 0; i < entries; ++i, ++entry) {
                const bool last = left == 0u;
                const int j = last ? 0 : __ffs(left) - 1;
                left &= left - 1u;
                if (entry % LOADERS != loader)
                    continue;
                const int s = entry % depth;
                const uint32_t phase = static_cast<uint32_t>(entry / depth) & 1u;
                const int r = __shfl_sync(kFull, row, j);
                const float gate = __shfl_sync(kFull, g, j);
                const uint16_t *src = !last      ? a.Y + static_cast<int64_t>(r) * a.ldy
                                      : a.resid ? a.resid + static_cast<int64_t>(t) * a.ldr
                                                : nullptr;
                // The 16-byte parts to copy: [from, to), the row at `shift`.
                const uint8_t *from = reinterpret_cast<const uint8_t *>(src), *to = from + row_bytes;
                uint32_t shift = 0, at = 0;                // at: where `from` goes
                bool edge = false;
                if constexpr (W < 8) {
                    if (src) {
                        const uint8_t *row_end = to;
                        shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(from) & 15u);
                        from -= shift;
                        to += (16u - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to) & 15u)) & 15u;
                        const int64_t rows = last ? a.T : a.rows, ld = last ? a.ldr : a.ldy;
                        const uint8_t *low = reinterpret_cast<const uint8_t *>(last ? a.resid : a.Y);
                        const uint8_t *high = low + ((rows - 1) * ld + a.N) * 2;
                        if (from < low) {
                            from += 16;
                            at = 16;
                            edge = true;
                        }
                        if (to > high) {
                            to -= 16;
                            edge = true;
                        }
                        if (edge) {
                            // Lane q has the row's elements q of the first and
                            // of the last partly covered 16 bytes.
                            if (lane == 0)
                                ok = mbar_wait(&m.empty[s], phase ^ 1u, abort_flag, a.wait_limit, &g_status);
                            ok = __shfl_sync(kFull, ok, 0);
                            if (ok) {
                                uint8_t *to_ring = ring + static_cast<size_t>(s) * pitch + shift;
                                const uint8_t *row0 = reinterpret_cast<const uint8_t *>(src);
                                const uint8_t *head = row0 + 2 * lane, *tail = to + 2 * lane;
                                if (head < from)
                                    *reinterpret_cast<uint16_t *>(to_ring + 2 * lane) = *reinterpret_cast<const uint16_t *>(head);
                                if (tail < row_end)
                                    *reinterpret_cast<uint16_t *>(to_ring + (tail - row0)) = *reinterpret_cast<const uint16_t *>(tail);
                            }
                            __syncwarp();
                        }
                    }
                }
                if (lane == 0) {
                    ok = ok && (edge || mbar_wait(&m.empty[s], phase ^ 1u, abort_flag, a.wait_limit, &g_status));
                    if (ok) {
                        const uint32_t bytes = src ? static_cast<uint32_t>(to - from) : 0u;
                        m.gate[s] = gate;
                        m.last[s] = last ? 1 : 0;
                        m.shift[s] = static_cast<int>(shift);
                        mbar_arrive_expect_tx(&m.full[s], bytes);
                        if (src)
                            bulk_load(ring + static_cast<size_t>(s) * pitch + at, from, bytes, &m.full[s], once);
                    }
                }
                ok = __shfl_sync(kFull, ok, 0);
                if (!ok)
                    break;
            }
        }
        if (lane == 0 && *abort_flag)
            // Let the copies already issued land before the block exits.
            for (int i = max(0, entry - depth); i < entry; ++i)
                if (i % LOADERS == loader)
                    mbar_wait_drain(&m.full[i % depth], (i / depth) & 1u, a.wait_limit);
        return;
    }
    const int n0 = static_cast<int>(threadIdx.x) * W;
    constexpr int step = THREADS * W;
    auto fetch = [&](const uint16_t *w, int u) {
        return w && n0 + u * step < a.N ? *reinterpret_cast<const Unit *>(w + n0 + u * step) : Unit{};
    };
    constexpr bool KEEP = W * PER <= 16 && THREADS * BLOCKS <= 768;        // the norms' weights stay in registers
    Unit post[KEEP ? PER : 1], pre[KEEP ? PER : 1];
    if constexpr (KEEP) {
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            post[u] = fetch(a.w_post, u);
            pre[u] = fetch(a.w_pre, u);
        }
    }
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;                              // after a wait that ran out: no data, but every barrier
    auto release = [&]() {
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&m.empty[s]);
        if (++s == depth) {
            s = 0;
            phase ^= 1u;
        }
    };
    auto entry = [&]() { return ring + static_cast<size_t>(s) * pitch + (W < 8 ? m.shift[s] : 0) + 2 * n0; };
    int parity = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 2) {
        float b[PER][W];
#pragma unroll
        for (int u = 0; u < PER; ++u)
#pragma unroll
            for (int i = 0; i < W; ++i)
                b[u][i] = 0.0f;
        for (;;) {
            ok = __all_sync(kFull, mbar_wait(&m.full[s], phase, abort_flag, a.wait_limit, &g_status));
            if (!ok || m.last[s])
                break;
            const float g = m.gate[s];
            const uint8_t *y = entry();
#pragma unroll
            for (int u = 0; u < PER; ++u)
                if (n0 + u * step < a.N) {
                    const Unit x = *reinterpret_cast<const Unit *>(y + 2 * u * step);
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        b[u][i] = fmaf(g, pick<W>(x, i), b[u][i]);
                }
            release();
        }
        if (a.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int u = 0; u < PER; ++u)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    ss = fmaf(b[u][i], b[u][i], ss);
            ss = ring_sum<THREADS>(ss, m.slots[parity]);
            const float r = inverse_rms(a, ss);
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const Unit w = KEEP ? post[KEEP ? u : 0] : fetch(a.w_post, u);
#pragma unroll
                for (int i = 0; i < W; ++i)
                    b[u][i] = b[u][i] * r * pick<W>(w, i);
            }
        }
        float ss = 0.0f;
        const uint8_t *res = entry();
#pragma unroll
        for (int u = 0; u < PER; ++u)
            if (n0 + u * step < a.N) {
                Unit x{};
                if (a.resid && ok)
                    x = *reinterpret_cast<const Unit *>(res + 2 * u * step);
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    b[u][i] = a.resid ? fmaf(a.out_scale, b[u][i], a.res_scale * pick<W>(x, i)) : a.out_scale * b[u][i];
                    ss = fmaf(b[u][i], b[u][i], ss);
                }
            }
        release();
#pragma unroll
        for (int u = 0; u < PER; ++u)
            if (n0 + u * step < a.N && a.H && ok)
                store_unit<W>(a.H + static_cast<int64_t>(t) * a.ldh + n0 + u * step, b[u]);
        if (a.Nrm) {
            ss = ring_sum<THREADS>(ss, m.slots[parity + 1]);
            const float r = inverse_rms(a, ss);
#pragma unroll
            for (int u = 0; u < PER; ++u)
                if (n0 + u * step < a.N && ok) {
                    const Unit w = KEEP ? pre[KEEP ? u : 0] : fetch(a.w_pre, u);
                    float y[W];
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        y[i] = b[u][i] * r * (a.w_pre ? pick<W>(w, i) : 1.0f);
                    store_unit<W>(a.Nrm + static_cast<int64_t>(t) * a.ldn + n0 + u * step, y);
                }
        }
    }
}

template <int W, int E, int JC, int THREADS, int BLOCKS>
cudaError_t launch_narrow_as(const CombineArgs &a, int sms, cudaStream_t stream)
{
    const int most = sms * BLOCKS;
    return launch_dependent(combine_narrow_kernel<W, E, JC, THREADS, BLOCKS>, dim3(a.T < most ? a.T : most), dim3(THREADS),
                            0, stream, a);
}

// Few tokens: eight elements per thread and two rows in flight, the shortest
// time for one (3 tokens of 2858: 3.7 against 6.0 us).  Many: sixteen elements,
// so that the sums' share is small and more tokens fit an SM (6437 tokens of
// 1196: 23 against 38 us).
template <int W>
cudaError_t launch_narrow(const CombineArgs &a, int sms, cudaStream_t stream)
{
    if (a.T < 2 * sms && a.N <= 8192)
        return a.N <= 512    ? launch_narrow_as<W, 8, 2, 64, 16>(a, sms, stream)
               : a.N <= 1024 ? launch_narrow_as<W, 8, 2, 128, 8>(a, sms, stream)
               : a.N <= 2048 ? launch_narrow_as<W, 8, 2, 256, 4>(a, sms, stream)
               : a.N <= 4096 ? launch_narrow_as<W, 8, 2, 512, 2>(a, sms, stream)
                             : launch_narrow_as<W, 8, 2, 1024, 1>(a, sms, stream);
    const int threads = (a.N + 15) / 16;
    return threads <= 32    ? launch_narrow_as<W, 16, 1, 32, 32>(a, sms, stream)
           : threads <= 64  ? launch_narrow_as<W, 16, 1, 64, 16>(a, sms, stream)
           : threads <= 96  ? launch_narrow_as<W, 16, 1, 96, 12>(a, sms, stream)
           : threads <= 128 ? launch_narrow_as<W, 16, 1, 128, 8>(a, sms, stream)
           : threads <= 192 ? launch_narrow_as<W, 16, 1, 192, 6>(a, sms, stream)
           : threads <= 256 ? launch_narrow_as<W, 16, 1, 256, 4>(a, sms, stream)
           : threads <= 384 ? launch_narrow_as<W, 16, 1, 384, 3>(a, sms, stream)
           : threads <= 512 ? launch_narrow_as<W, 16, 1, 512, 2>(a, sms, stream)
                            : launch_narrow_as<W, 32, 1, 1024, 1>(a, sms, stream);
}

template <int W, int E, int THREADS, int BLOCKS, int LOADERS>
cudaError_t launch_ring_as(const CombineArgs &a, int sms, cudaStream_t stream)
{
    constexpr auto kern = combine_ring_kernel<W, E / W, THREADS, BLOCKS, LOADERS>;
    const cudaError_t e = opt_in<kern, kRingBytes / BLOCKS>();
    if (e != cudaSuccess)
        return e;
    const int pitch = static_cast<int>(ring_pitch(a.N, W));
    const int fit = kRingBytes / BLOCKS / pitch;
    const int depth = fit < kRingMaxRows ? fit : kRingMaxRows;
    const int most = sms * BLOCKS;
    return launch_dependent(kern, dim3(a.T < most ? a.T : most), dim3(THREADS + 32 * LOADERS),
                            static_cast<size_t>(depth) * pitch, stream, a, depth);
}

// Enough tokens for every SM to have several, and rows long enough that a ring
// entry's hand-over (some 600 cycles for a block) is short beside them.
bool ring_pays(const CombineArgs &a, int sms)
{
    return a.T >= 4 * sms && a.N <= 16384 && (a.N > 1280 || (a.width == 1 && a.N > 1024));
}

// Sixteen elements per thread, so that few threads share a token and an SM has
// several tokens at hand: one's hand-overs, sums and stores hide behind another's.
// 8192 tokens x 4 rows, both norms: N = 2048: 39 us (one block of 512 threads per
// SM 128, no ring 50), 4096: 78 (118, 101), 8184: 148 (one loading warp 165, no
// ring 183).
template <int W>
cudaError_t launch_ring(const CombineArgs &a, int sms, cudaStream_t stream)
{
    if (a.N <= 2048)
        return launch_ring_as<W, 16, 128, 5, 1>(a, sms, stream);
    if (a.N <= 4096)
        return launch_ring_as<W, 16, 256, 3, 1>(a, sms, stream);
    if (a.N <= 6144)
        // Single elements take so many instructions that the weights, which only
        // one block's threads have registers for, count more than a second block
        // (1000 tokens x 2 rows of 5001: 20 against 28 us).
        return launch_ring_as<W, 16, 384, W == 1 ? 1 : 2, W == 1 ? 2 : 1>(a, sms, stream);
    if (a.N <= 8192)
        return launch_ring_as<W, 16, 512, 1, 2>(a, sms, stream);
    return launch_ring_as<W, 32, 512, 1, 2>(a, sms, stream);
}

}  // namespace

cudaError_t launch_combine(const CombineArgs &a, int sms, cudaStream_t stream)
{
    if (ring_pays(a, sms))
        return a.width == 8   ? launch_ring<8>(a, sms, stream)
               : a.width == 4 ? launch_ring<4>(a, sms, stream)
               : a.width == 2 ? launch_ring<2>(a, sms, stream)
                              : launch_ring<1>(a, sms, stream);
    if (a.width < 8)
        return a.width == 4   ? launch_narrow<4>(a, sms, stream)
               : a.width == 2 ? launch_narrow<2>(a, sms, stream)
                              : launch_narrow<1>(a, sms, stream);
    const int vecs = (a.N + 7) / 8;
    // Fewer tokens than SMs: up to 1024 threads each (8 tokens x 8 rows of 7168:
    // 3.8 us, with 512 threads 5.1).
    const bool few = a.T < sms && vecs <= 2048;
    const int most_threads = few ? 1024 : kCombineThreads;
    const int threads = vecs < most_threads ? (vecs + 31) / 32 * 32 : most_threads;
    const int per = (vecs + threads - 1) / threads;
    const int most = sms * (2048 / threads);
    const dim3 grid(static_cast<unsigned>(a.T < most ? a.T : most)), block(static_cast<unsigned>(threads));
    if (few && per <= 1)
        return launch_dependent(combine_kernel<1, 4, 1024>, grid, block, 0, stream, a);
    if (few)
        return launch_dependent(combine_kernel<2, 2, 1024>, grid, block, 0, stream, a);
    if (per <= 1)
        return launch_dependent(combine_kernel<1, 4, kCombineThreads>, grid, block, 0, stream, a);
    if (per <= 2)
        return launch_dependent(combine_kernel<2, 4, kCombineThreads>, grid, block, 0, stream, a);
    if (per <= 4)
        return launch_dependent(combine_kernel<4, 2, kCombineThreads>, grid, block, 0, stream, a);
    if (per <= kCombineMaxVec)
        return launch_dependent(combine_kernel<8, 1, kCombineThreads>, grid, block, 0, stream, a);
    return cudaErrorInvalidValue;
}

cudaError_t read_expert_status(int *status, int reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(status, g_status, sizeof(int));
    if (e != cudaSuccess || !reset)
        return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
}

}  // namespace mxfp4
