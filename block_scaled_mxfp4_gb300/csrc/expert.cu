// Expert-layer operators around the grouped products: routing, the grouped
// quantiser and the gated join with its norms.  All three are bound by HBM
// traffic at prefill sizes and by latency at decoding sizes; every kernel is a
// programmatic dependent of the work before it on the stream and waits for that
// work before it reads anything.
#include <atomic>
#include <cuda_bf16.h>

#include "expert.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace mxfp4 {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ int g_status = 0;                     // bounded waits that ran out

template <typename Kern, typename... Args>
cudaError_t launch_dependent(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// ------------------------------------------------------------------ routing --
//
// Stable counting sort of (token, slot) rows by expert.  A token picks an
// expert at most once, so inside a run of 128 tokens an expert's rows are a
// 128-bit mask of tokens (set with atomicOr, whose order does not matter), and
// a row's place among them is the number of set bits before its own.  Blocks
// write their experts' counts; the second kernel adds up the counts of the
// blocks before its own and all of them (integers: any order, the same sum),
// and places its tokens' rows.

constexpr int kRouteThreads = 512;
constexpr int kRouteRun = 128;                   // tokens of one mask
constexpr int kRouteSingle = 64;                 // tokens that one block does alone
constexpr int kRouteMaxBlocks = 304;

// Float -> unsigned that orders the same way; NaN and -inf give 0, which no
// other value does: such an expert is never picked.
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);          // -0 -> +0: equal values tie
    const uint32_t key = b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
    return x > __int_as_float(0xff800000) ? key : 0u;
}

__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// Picking.  LANES lanes share a token; each holds CH * 4 of its experts as keys
// in shared memory, in chunks of four interleaved over the lanes (expert
// (c * LANES + l) * 4 + i is key i of lane l's chunk c), and the chunks' maxima
// in registers.  A pick takes the largest maximum of the lanes, and only the
// lane that owns it looks into one chunk, drops the key and renews one maximum:
// a handful of instructions per pick for each of the 32 / LANES tokens of a warp.
// Ties: a lane's chunks and a chunk's keys are in index order, and where
// several lanes hold the maximum, the lowest of their indexes counts.
// picks: k (expert, exp or sigmoid) pairs of each of the warp's tokens.
template <int LANES, int CH>
__device__ __forceinline__ void route_tokens(const RouteArgs &a, int t, bool live, int bit, int lane, uint4 *keys,
                                             float2 *picks, uint32_t *masks)
{
    const int l = lane & (LANES - 1);
    uint4 *mine = keys + lane;                             // chunk c at mine[32 c]: no bank conflicts
    const bool on = live && !(a.mask && a.mask[t] == 0);
    const int64_t row = static_cast<int64_t>(live ? t : 0) * a.ldl;
    uint32_t top[CH];                                      // the chunks' maxima
    // Loads first, all in flight together.
    float x[CH][4];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int e = (c * LANES + l) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[c][i] = __int_as_float(0xff800000);
        if (on && e < a.E) {
            if (a.fp32) {
                const float *p = static_cast<const float *>(a.logits) + row + e;
                if (a.vec && e + 4 <= a.E) {
                    const float4 v = __ldcs(reinterpret_cast<const float4 *>(p));
                    x[c][0] = v.x;
                    x[c][1] = v.y;
                    x[c][2] = v.z;
                    x[c][3] = v.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (e + i < a.E)
                            x[c][i] = p[i];
                }
            } else {
                const uint16_t *p = static_cast<const uint16_t *>(a.logits) + row + e;
                if (a.vec && e + 4 <= a.E) {
                    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
                    x[c][0] = bf16_lo(v.x);
                    x[c][1] = bf16_hi(v.x);
                    x[c][2] = bf16_lo(v.y);
                    x[c][3] = bf16_hi(v.y);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (e + i < a.E)
                            x[c][i] = bf16_lo(p[i]);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const uint4 k = make_uint4(order_key(x[c][0]), order_key(x[c][1]), order_key(x[c][2]), order_key(x[c][3]));
        mine[32 * c] = k;
        top[c] = max(max(k.x, k.y), max(k.z, k.w));
    }
    uint32_t best = top[0];
#pragma unroll
    for (int c = 1; c < CH; ++c)
        best = max(best, top[c]);
    float2 *my_picks = picks + (lane / LANES) * a.k;
    uint32_t first = 0u;                                   // the token's largest key
    float sum = 0.0f;                                      // of the softmax
    int taken = 0;
    for (; taken < a.k; ++taken) {
        uint32_t m = best;
#pragma unroll
        for (int d = LANES / 2; d > 0; d >>= 1)
            m = max(m, __shfl_xor_sync(kFull, m, d));
        if (taken == 0) {
            first = m;
            if (a.mode == 1 && m != 0u) {
                // Terms far below the largest do not matter to the sum, so the
                // fast exponential (whose relative error grows with its
                // argument) keeps the sum to a few 2^-24 of itself.
                const float xm = key_value(m);
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float z = x[c][i];
                        sum += z == xm ? 1.0f : z > __int_as_float(0xff800000) ? __expf(z - xm) : 0.0f;
                    }
            }
        }
        if (!__any_sync(kFull, m != 0u))
            break;
        int at = 0x7FFFFFFF, chunk = 0, in = 0;
        uint4 k = make_uint4(0u, 0u, 0u, 0u);
        if (m != 0u && best == m) {
#pragma unroll
            for (int c = CH - 1; c >= 0; --c)
                if (top[c] == m)
                    chunk = c;
            k = mine[32 * chunk];
            in = k.x == m ? 0 : k.y == m ? 1 : k.z == m ? 2 : 3;
            at = (chunk * LANES + l) * 4 + in;
        }
        int low = at;
#pragma unroll
        for (int d = LANES / 2; d > 0; d >>= 1)
            low = min(low, __shfl_xor_sync(kFull, low, d));
        if (m != 0u && at == low) {
            k.x = in == 0 ? 0u : k.x;
            k.y = in == 1 ? 0u : k.y;
            k.z = in == 2 ? 0u : k.z;
            k.w = in == 3 ? 0u : k.w;
            mine[32 * chunk] = k;
            const uint32_t left = max(max(k.x, k.y), max(k.z, k.w));
            best = 0u;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                top[c] = c == chunk ? left : top[c];
                best = max(best, top[c]);
            }
            my_picks[taken] = make_float2(__int_as_float(at), key_value(m));
            atomicOr(&masks[at * 4 + (bit >> 5)], 1u << (bit & 31));
        } else if (m == 0u && l == 0) {
            my_picks[taken] = make_float2(__int_as_float(-1), 0.0f);
        }
    }
    __syncwarp();
    // Gates: the lanes of a token share its picks.
    const float vm = key_value(first);
    if (a.mode == 0)
        for (int j = l; j < taken; j += LANES) {
            const float2 p = my_picks[j];
            if (__float_as_int(p.x) >= 0)
                sum += p.y == vm ? 1.0f : expf(p.y - vm);
        }
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1)
        sum += __shfl_xor_sync(kFull, sum, d);
    if (live)
        for (int j = l; j < a.k; j += LANES) {
            const float2 p = j < taken ? my_picks[j] : make_float2(__int_as_float(-1), 0.0f);
            const int id = __float_as_int(p.x);
            float g = 0.0f;
            if (id >= 0)
                g = a.mode == 2 ? 1.0f / (1.0f + expf(-p.y)) : (p.y == vm ? 1.0f : expf(p.y - vm)) / sum;
            a.ids[static_cast<int64_t>(t) * a.k + j] = id;
            a.gates[static_cast<int64_t>(t) * a.k + j] = a.gate_scale * g;
        }
    __syncwarp();                                          // the keys and picks are used again
}

// Exclusive prefix sums of total[0 .. E) over the block, in place; returns
// the sum of all.
__device__ __forceinline__ int block_scan(int *total, int E)
{
    __shared__ int warp_sum[32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, n = (E + kRouteThreads - 1) / kRouteThreads;
    int sum = 0;
    for (int i = 0; i < n; ++i)
        if (t * n + i < E)
            sum += total[t * n + i];
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, d);
        if (lane >= d)
            incl += v;
    }
    if (lane == 31)
        warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - sum, all = 0;
    for (int w = 0; w < kRouteThreads / 32; ++w) {
        before += w < warp ? warp_sum[w] : 0;
        all += warp_sum[w];
    }
    for (int i = 0; i < n; ++i)
        if (t * n + i < E) {
            const int v = total[t * n + i];
            total[t * n + i] = before;
            before += v;
        }
    __syncthreads();
    return all;
}

template <int LANES, int CH>
__global__ void __launch_bounds__(kRouteThreads, 2) route_pick_kernel(const __grid_constant__ RouteArgs a)
{
    constexpr int TPW = 32 / LANES;                        // tokens of a warp
    extern __shared__ __align__(16) uint32_t smem_u32[];
    uint4 *all_keys = reinterpret_cast<uint4 *>(smem_u32); // [warps][CH][32]
    float2 *all_picks = reinterpret_cast<float2 *>(all_keys + kRouteThreads * CH);   // [warps][TPW][k]
    uint32_t *masks = reinterpret_cast<uint32_t *>(all_picks + kRouteThreads / LANES * a.k);   // [E][4]
    int *run = reinterpret_cast<int *>(masks + 4 * a.E);   // [E]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * a.chunk;
    const int t1 = min(a.T, t0 + a.chunk);
    const bool single = gridDim.x == 1;
    for (int i = threadIdx.x; i < a.E; i += kRouteThreads)
        run[i] = 0;
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    for (int s0 = t0; s0 < t1; s0 += kRouteRun) {
        for (int i = threadIdx.x; i < 4 * a.E; i += kRouteThreads)
            masks[i] = 0u;
        __syncthreads();
        const int s1 = min(t1, s0 + kRouteRun);
        for (int q = s0 + warp * TPW; q < s1; q += kRouteThreads / 32 * TPW) {
            const int t = q + lane / LANES;
            route_tokens<LANES, CH>(a, t, t < s1, t - s0, lane, all_keys + warp * CH * 32, all_picks + warp * TPW * a.k,
                                    masks);
        }
        __syncthreads();
        // Each row's place among its expert's rows of this block.
        for (int i = threadIdx.x; i < (s1 - s0) * a.k; i += kRouteThreads) {
            const int64_t at = static_cast<int64_t>(s0) * a.k + i;
            const int e = a.ids[at];
            int place = -1;
            if (e >= 0) {
                const int bit = i / a.k;
                place = run[e];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t m = masks[4 * e + w];
                    place += w < (bit >> 5) ? __popc(m) : w == (bit >> 5) ? __popc(m & ((1u << (bit & 31)) - 1u)) : 0;
                }
            }
            a.slot_row[at] = place;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kRouteThreads)
            run[e] += __popc(masks[4 * e]) + __popc(masks[4 * e + 1]) + __popc(masks[4 * e + 2]) + __popc(masks[4 * e + 3]);
        __syncthreads();
    }
    if (!single) {
        uint16_t *count = a.counts + static_cast<int64_t>(blockIdx.x) * ((a.E + 7) / 8 * 8);
        for (int e = threadIdx.x; e < (a.E + 7) / 8 * 8; e += kRouteThreads)
            count[e] = e < a.E ? static_cast<uint16_t>(run[e]) : uint16_t(0);
        return;
    }
    const int all = block_scan(run, a.E);
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads)
        a.offsets[e] = e < a.E ? run[e] : all;
    for (int i = threadIdx.x; i < a.T * a.k; i += kRouteThreads) {
        const int e = a.ids[i];
        if (e >= 0) {
            const int row = run[e] + a.slot_row[i];
            a.slot_row[i] = row;
            a.row_token[row] = i / a.k;
        }
        if (i >= all)
            a.row_token[i] = -1;
    }
}

__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const __grid_constant__ RouteArgs a)
{
    extern __shared__ __align__(16) uint32_t smem_u32[];
    const int ep = (a.E + 7) / 8 * 8, lanes = ep / 8;      // threads of one block's counts
    const int blocks = gridDim.x, me = blockIdx.x;
    const int at_once = kRouteThreads / lanes;             // blocks whose counts are read together
    uint32_t *part = smem_u32;                             // [at_once][2][ep]: all blocks, the blocks before
    int *total = reinterpret_cast<int *>(part + 2 * at_once * ep);   // [ep]
    int *mine = total + ep;                                // [ep]
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    if (static_cast<int>(threadIdx.x) < at_once * lanes) {
        const int q = threadIdx.x % lanes, g = threadIdx.x / lanes;
        uint32_t all[8], before[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            all[i] = before[i] = 0u;
#pragma unroll 8
        for (int b = g; b < blocks; b += at_once) {
            const uint4 v = *reinterpret_cast<const uint4 *>(a.counts + static_cast<int64_t>(b) * ep + 8 * q);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t c = (w[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
                all[i] += c;
                before[i] += b < me ? c : 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            part[(2 * g) * ep + 8 * q + i] = all[i];
            part[(2 * g + 1) * ep + 8 * q + i] = before[i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * ep; i += kRouteThreads) {
        uint32_t s = 0u;
        for (int g = 0; g < at_once; ++g)
            s += part[2 * g * ep + i];
        total[i] = static_cast<int>(s);                    // total, then mine
    }
    __syncthreads();
    const int sum = block_scan(total, a.E);
    if (me == 0)
        for (int e = threadIdx.x; e <= a.E; e += kRouteThreads)
            a.offsets[e] = e < a.E ? total[e] : sum;
    const int64_t i0 = static_cast<int64_t>(me) * a.chunk * a.k;
    const int64_t i1 = min(static_cast<int64_t>(a.T) * a.k, i0 + static_cast<int64_t>(a.chunk) * a.k);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kRouteThreads) {
        const int e = a.ids[i];
        if (e >= 0) {
            const int row = total[e] + mine[e] + a.slot_row[i];
            a.slot_row[i] = row;
            a.row_token[row] = static_cast<int>(i / a.k);
        }
        if (i >= sum)
            a.row_token[i] = -1;
    }
}

__global__ void route_empty_kernel(int *offsets, int E)
{
    pdl_wait_prerequisites();
    for (int e = threadIdx.x; e <= E; e += blockDim.x)
        offsets[e] = 0;
}

// ------------------------------------------------------- grouped quantiser --
//
// One thread per 1x32 block of a source row: the block is read and rounded
// once and stored at each of the row's destinations.  The four threads of an
// atom's word (four consecutive blocks of a row) put their scale codes
// together and one of them stores the word.  Blocks move in 32-byte accesses,
// a whole sector per thread.  The destinations of four slots are looked up
// together, so that a row costs two dependent round trips (slot, then offset)
// and not two for each slot.

constexpr int kQuantThreads = 256;
constexpr int kQuantSlots = 4;

__device__ __forceinline__ void ld_global_v8(const void *p, uint32_t (&w)[8])
{
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

// WIDE: X's and Q's rows allow 32-byte accesses.
template <QuantFmt Q, bool WIDE>
__global__ void __launch_bounds__(kQuantThreads, 3) group_quantize_kernel(const __grid_constant__ GroupQuantArgs a)
{
    constexpr int W = QuantTraits<Q>::kWords;
    const int kb = a.K / 32;
    const int kb4 = (kb + 3) / 4 * 4;
    const int64_t atoms_row = sf_groups(a.K) * kSfAtomBytes;
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    const int64_t total = static_cast<int64_t>(a.T) * kb4;
    for (int64_t g0 = blockIdx.x * static_cast<int64_t>(blockDim.x); g0 < total;
         g0 += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t g = g0 + threadIdx.x;
        const bool in = g < total;
        const int t = static_cast<int>((in ? g : total - 1) / kb4);
        const int b = static_cast<int>((in ? g : total - 1) - static_cast<int64_t>(t) * kb4);
        const bool real = in && b < kb;
        uint32_t src[16];
        if (real) {
            const uint16_t *x = a.X + static_cast<int64_t>(t) * a.ldx + b * 32;
            if constexpr (WIDE) {
                uint32_t lo[8], hi[8];
                ld_global_v8(x, lo);
                ld_global_v8(x + 16, hi);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    src[i] = lo[i];
                    src[8 + i] = hi[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(x) + i);
                    src[4 * i] = v.x;
                    src[4 * i + 1] = v.y;
                    src[4 * i + 2] = v.z;
                    src[4 * i + 3] = v.w;
                }
            }
        }
        uint32_t out[W];
        uint32_t word = 0x7Fu;
        for (int j0 = 0; j0 < a.k; j0 += kQuantSlots) {
            int row[kQuantSlots], e[kQuantSlots], o[kQuantSlots], end[kQuantSlots];
            if (a.slot_row) {
#pragma unroll
                for (int i = 0; i < kQuantSlots; ++i) {
                    const int64_t at = static_cast<int64_t>(t) * a.k + j0 + i;
                    row[i] = j0 + i < a.k ? a.slot_row[at] : -1;
                    e[i] = j0 + i < a.k ? a.ids[at] : -1;
                }
            } else {
                // The group of row t: the last whose offset is not after it.
                int lo = 0, hi = a.groups - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (a.offsets[mid] <= t)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
#pragma unroll
                for (int i = 0; i < kQuantSlots; ++i) {
                    row[i] = i == 0 ? t : -1;
                    e[i] = lo;
                }
            }
#pragma unroll
            for (int i = 0; i < kQuantSlots; ++i) {
                const bool ok = in && row[i] >= 0 && row[i] < a.rows && e[i] >= 0 && e[i] < a.groups;
                o[i] = ok ? a.offsets[e[i]] : 0;
                end[i] = ok ? a.offsets[e[i] + 1] : 0;
            }
            if (j0 == 0) {
                // Rounded after the look-ups were issued.
                if (real) {
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        x[2 * i] = bf16_lo(src[i]);
                        x[2 * i + 1] = bf16_hi(src[i]);
                    }
                    word = quantize_block<Q>(x, out);
                }
                // total and kb4 are multiples of 4, so a word's four threads
                // are all inside or all outside.
                word <<= 8 * (b & 3);
                word |= __shfl_xor_sync(kFull, word, 1);
                word |= __shfl_xor_sync(kFull, word, 2);
            }
#pragma unroll
            for (int i = 0; i < kQuantSlots; ++i) {
                if (o[i] < 0 || row[i] < o[i] || row[i] >= end[i])
                    continue;
                if (real) {
                    uint8_t *q = a.Q + static_cast<int64_t>(row[i]) * a.ldq_bytes + static_cast<int64_t>(b) * (4 * W);
                    if constexpr (WIDE && W == 8) {
                        st_global_v8(q, out[0], out[1], out[2], out[3], out[4], out[5], out[6], out[7]);
                    } else {
#pragma unroll
                        for (int w = 0; w < W; w += 4)
                            reinterpret_cast<uint4 *>(q)[w / 4] = make_uint4(out[w], out[w + 1], out[w + 2], out[w + 3]);
                    }
                }
                if ((b & 3) == 0) {
                    const int local = row[i] - o[i];
                    const int64_t block = group_sf_block(o[i], e[i]) + local / kSfRowBlock;
                    *reinterpret_cast<uint32_t *>(a.S + block * atoms_row + sf_byte(local % kSfRowBlock, b)) = word;
                }
            }
        }
    }
}

// ------------------------------------------------------------------- join --
//
//   b = sum_j gates[t, j] Y[slot_row[t, j]]          (fp32, slots in order)
//   b = b rsqrt(mean b^2 + eps) w_post               with w_post
//   h = res_scale resid[t] + out_scale b             -> H, one rounding
//   n = h rsqrt(mean h^2 + eps) w_pre                -> Nrm, one rounding, from the fp32 h
//
// One block per token (grid-stride), the row in registers between the two
// sums, so that every input is read once.

constexpr int kCombineThreads = 512;
constexpr int kCombineMaxVec = 8;                // 8-element vectors of one thread

__device__ __forceinline__ void store8(uint16_t *p, int n, int N, int vec, const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    if (vec && n + 8 <= N) {
        *reinterpret_cast<uint4 *>(p + n) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (n + i < N)
                p[n + i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
    }
}

// Sum over the block; every thread gets it.  The two slots alternate so that
// the next call's writes do not meet this one's reads.
__device__ __forceinline__ float block_sum(float v, float *slot)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFull, v, d);
    if ((threadIdx.x & 31) == 0)
        slot[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    const int warps = blockDim.x >> 5;
    for (int w = 0; w < warps; ++w)
        s += slot[w];
    return s;
}

// Raw bf16 pairs of 8 elements, zeros past N.
__device__ __forceinline__ uint4 raw8(const uint16_t *p, int n, int N, int vec)
{
    if (vec && n + 8 <= N)
        return *reinterpret_cast<const uint4 *>(p + n);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (n + i < N)
            w[i / 2] |= static_cast<uint32_t>(p[n + i]) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float pick8(const uint4 &v, int i)
{
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return i & 1 ? bf16_hi(w) : bf16_lo(w);
}

// VPT 8-element vectors per thread, JC slots' rows in flight together.
template <int VPT, int JC>
__global__ void __launch_bounds__(kCombineThreads, VPT <= 2 ? 2 : 1) combine_kernel(const __grid_constant__ CombineArgs a)
{
    __shared__ float slots[4][kCombineThreads / 32];
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
                res[v] = raw8(a.resid + static_cast<int64_t>(t) * a.ldr, n, a.N, a.vec);
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
                        y[j][v] = raw8(a.Y + static_cast<int64_t>(row[j]) * a.ldy, n, a.N, a.vec);
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
            const float r = 1.0f / sqrtf(ss / static_cast<float>(a.N) + a.eps);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int n = (v * blockDim.x + threadIdx.x) * 8;
                if (n < a.N) {
                    const uint4 w = raw8(a.w_post, n, a.N, a.vec);
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
                    res[v] = raw8(a.resid + static_cast<int64_t>(t) * a.ldr, n, a.N, a.vec);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    b[v][i] = a.resid ? fmaf(a.out_scale, b[v][i], a.res_scale * pick8(res[v], i)) : a.out_scale * b[v][i];
                    ss = fmaf(b[v][i], b[v][i], ss);
                }
                if (a.H)
                    store8(a.H + static_cast<int64_t>(t) * a.ldh, n, a.N, a.vec, b[v]);
            }
        }
        if (a.Nrm) {
            ss = block_sum(ss, slots[parity + 1]);
            const float r = 1.0f / sqrtf(ss / static_cast<float>(a.N) + a.eps);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int n = (v * blockDim.x + threadIdx.x) * 8;
                if (n < a.N) {
                    float y[8];
                    if (a.w_pre) {
                        const uint4 w = raw8(a.w_pre, n, a.N, a.vec);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            y[i] = b[v][i] * r * pick8(w, i);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            y[i] = b[v][i] * r;
                    }
                    store8(a.Nrm + static_cast<int64_t>(t) * a.ldn, n, a.N, a.vec, y);
                }
            }
        }
    }
}

// The same for long prefills, where the sums' barriers must not leave HBM
// idle: one persistent block per SM, whose last warp streams the tokens' rows
// (the taken rows of Y, then the residual row) into a ring of whole rows in
// shared memory with bulk copies, as far ahead as the ring holds, while 16
// warps work on the token at hand.  8192 tokens x 4 rows of 8192: see the
// launcher.
constexpr int kRingThreads = kCombineThreads + 32;
constexpr int kRingMaxRows = 32;
constexpr int kRingBytes = 200 * 1024;

struct RingMeta {
    uint64_t full[kRingMaxRows];
    uint64_t empty[kRingMaxRows];
    float gate[kRingMaxRows];
    int last[kRingMaxRows];                      // 1: the token's last entry (its residual row, or nothing)
    float slots[4][kCombineThreads / 32];
    int abort_flag;
};

__device__ __forceinline__ float ring_sum(float v, float *slot)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(kFull, v, d);
    if ((threadIdx.x & 31) == 0)
        slot[threadIdx.x >> 5] = v;
    asm volatile("bar.sync 1, %0;" ::"n"(kCombineThreads) : "memory");
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kCombineThreads / 32; ++w)
        s += slot[w];
    return s;
}

template <int VPT>
__global__ void __launch_bounds__(kRingThreads, 1) combine_ring_kernel(const __grid_constant__ CombineArgs a, int depth)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ RingMeta m;
    const uint32_t row_bytes = static_cast<uint32_t>(a.N) * 2;
    const uint32_t pitch = (row_bytes + 127u) / 128u * 128u;
    volatile int *abort_flag = &m.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < depth; ++s) {
            mbar_init(&m.full[s], 1);
            mbar_init(&m.empty[s], kCombineThreads / 32);
        }
        m.abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    int s = 0;
    uint32_t phase = 0;
    if (warp == kCombineThreads / 32) {
        const uint64_t once = l2_policy_evict_first();
        int issued = 0;
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
            for (int i = 0; i < entries && ok; ++i) {
                const bool last = left == 0u;
                const int j = last ? 0 : __ffs(left) - 1;
                left &= left - 1u;
                const int r = __shfl_sync(kFull, row, j);
                const float gate = __shfl_sync(kFull, g, j);
                if (lane == 0) {
                    ok = mbar_wait(&m.empty[s], phase ^ 1u, abort_flag, a.wait_limit, &g_status);
                    if (ok) {
                        m.gate[s] = gate;
                        m.last[s] = last ? 1 : 0;
                        const uint16_t *src = !last      ? a.Y + static_cast<int64_t>(r) * a.ldy
                                              : a.resid ? a.resid + static_cast<int64_t>(t) * a.ldr
                                                        : nullptr;
                        mbar_arrive_expect_tx(&m.full[s], src ? row_bytes : 0u);
                        if (src)
                            bulk_load(ring + static_cast<size_t>(s) * pitch, src, row_bytes, &m.full[s], once);
                    }
                }
                ok = __shfl_sync(kFull, ok, 0);
                if (ok) {
                    ++issued;
                    if (++s == depth) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
        if (lane == 0 && *abort_flag)
            // Let the copies already issued land before the block exits.
            for (int i = max(0, issued - depth); i < issued; ++i)
                mbar_wait_drain(&m.full[i % depth], (i / depth) & 1u, a.wait_limit);
        return;
    }
    const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
    auto weight = [&](const uint16_t *w, int v) {
        const int n = (v * kCombineThreads + threadIdx.x) * 8;
        return w && n < a.N ? *reinterpret_cast<const uint4 *>(w + n) : ones;
    };
    constexpr bool KEEP = VPT <= 2;              // the norms' weights stay in registers
    uint4 post[VPT], pre[VPT];
    if constexpr (KEEP) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            post[v] = weight(a.w_post, v);
            pre[v] = weight(a.w_pre, v);
        }
    }
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
    int parity = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 2) {
        float b[VPT][8];
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                b[v][i] = 0.0f;
        for (;;) {
            ok = __all_sync(kFull, mbar_wait(&m.full[s], phase, abort_flag, a.wait_limit, &g_status));
            if (!ok || m.last[s])
                break;
            const float g = m.gate[s];
            const uint8_t *y = ring + static_cast<size_t>(s) * pitch;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int n = (v * kCombineThreads + threadIdx.x) * 8;
                if (n < a.N) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(y + 2 * n);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        b[v][i] = fmaf(g, pick8(x, i), b[v][i]);
                }
            }
            release();
        }
        if (a.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int v = 0; v < VPT; ++v)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ss = fmaf(b[v][i], b[v][i], ss);
            ss = ring_sum(ss, m.slots[parity]);
            const float r = 1.0f / sqrtf(ss / static_cast<float>(a.N) + a.eps);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const uint4 w = KEEP ? post[v] : weight(a.w_post, v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    b[v][i] = b[v][i] * r * pick8(w, i);
            }
        }
        float ss = 0.0f;
        const uint8_t *res = ring + static_cast<size_t>(s) * pitch;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = (v * kCombineThreads + threadIdx.x) * 8;
            if (n < a.N) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (a.resid)
                    x = *reinterpret_cast<const uint4 *>(res + 2 * n);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    b[v][i] = a.resid ? fmaf(a.out_scale, b[v][i], a.res_scale * pick8(x, i)) : a.out_scale * b[v][i];
                    ss = fmaf(b[v][i], b[v][i], ss);
                }
            }
        }
        release();
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = (v * kCombineThreads + threadIdx.x) * 8;
            if (n < a.N && a.H && ok)
                store8(a.H + static_cast<int64_t>(t) * a.ldh, n, a.N, 1, b[v]);
        }
        if (a.Nrm) {
            ss = ring_sum(ss, m.slots[parity + 1]);
            const float r = 1.0f / sqrtf(ss / static_cast<float>(a.N) + a.eps);
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int n = (v * kCombineThreads + threadIdx.x) * 8;
                if (n < a.N && ok) {
                    const uint4 w = KEEP ? pre[v] : weight(a.w_pre, v);
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = b[v][i] * r * pick8(w, i);
                    store8(a.Nrm + static_cast<int64_t>(t) * a.ldn, n, a.N, 1, y);
                }
            }
        }
    }
}

template <int VPT>
cudaError_t launch_ring(const CombineArgs &a, int sms, cudaStream_t stream)
{
    auto kern = combine_ring_kernel<VPT>;
    static std::atomic<int> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !configured[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            configured[dev].store(1, std::memory_order_relaxed);
    }
    const int pitch = (a.N * 2 + 127) / 128 * 128;
    const int fit = kRingBytes / pitch;
    const int depth = fit < kRingMaxRows ? fit : kRingMaxRows;
    return launch_dependent(kern, dim3(a.T < sms ? a.T : sms), dim3(kRingThreads), static_cast<size_t>(depth) * pitch,
                            stream, a, depth);
}

template <int LANES, int CH>
cudaError_t launch_pick(const RouteArgs &a, cudaStream_t stream)
{
    const size_t smem = static_cast<size_t>(kRouteThreads) * CH * 16 + static_cast<size_t>(kRouteThreads / LANES) * a.k * 8 +
                        static_cast<size_t>(5 * a.E) * 4;
    auto kern = route_pick_kernel<LANES, CH>;
    static std::atomic<int> configured[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !configured[dev].load(std::memory_order_relaxed)) {
        // The most that any E and k need of this instance.
        const int most = kRouteThreads * CH * 16 + kRouteThreads / LANES * kMaxTopK * 8 + 5 * LANES * CH * 4 * 4;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            configured[dev].store(1, std::memory_order_relaxed);
    }
    return launch_dependent(kern, dim3(a.blocks), dim3(kRouteThreads), smem, stream, a);
}

}  // namespace

int route_blocks(int T, int *chunk)
{
    int c = T <= kRouteSingle ? kRouteSingle : 32;
    if (T > 32 * kRouteMaxBlocks)
        c = ((T + kRouteMaxBlocks - 1) / kRouteMaxBlocks + 31) / 32 * 32;
    *chunk = c;
    return (T + c - 1) / c;
}

cudaError_t launch_route(const RouteArgs &a, int sms, cudaStream_t stream)
{
    if (a.T == 0)
        return launch_dependent(route_empty_kernel, dim3(1), dim3(256), 0, stream, a.offsets, a.E);
    // Lanes per token: as few as hold its experts in 32 registers each, which
    // shares a pick's instructions among the most tokens, once that still
    // leaves every SM 16 warps; otherwise a whole warp per token, the shortest
    // time for one.  (32768 tokens of 256 experts: 8 lanes.)
    int lanes = 1;
    while (lanes * 32 < a.E)
        lanes *= 2;
    cudaError_t e;
    if (static_cast<int64_t>(a.T) * lanes / 32 < static_cast<int64_t>(sms) * 16) {
        e = a.E <= 128   ? launch_pick<32, 1>(a, stream)
            : a.E <= 256 ? launch_pick<32, 2>(a, stream)
            : a.E <= 512 ? launch_pick<32, 4>(a, stream)
                         : launch_pick<32, 8>(a, stream);
    } else {
        switch (lanes) {
        case 1: e = launch_pick<1, 8>(a, stream); break;
        case 2: e = launch_pick<2, 8>(a, stream); break;
        case 4: e = launch_pick<4, 8>(a, stream); break;
        case 8: e = launch_pick<8, 8>(a, stream); break;
        case 16: e = launch_pick<16, 8>(a, stream); break;
        default: e = launch_pick<32, 8>(a, stream); break;
        }
    }
    if (e != cudaSuccess || a.blocks == 1)
        return e;
    const int ep = (a.E + 7) / 8 * 8;
    const size_t smem2 = static_cast<size_t>(2 * (kRouteThreads / (ep / 8)) + 2) * ep * 4;
    return launch_dependent(route_place_kernel, dim3(a.blocks), dim3(kRouteThreads), smem2, stream, a);
}

template <QuantFmt Q>
static cudaError_t launch_quant(const GroupQuantArgs &a, dim3 grid, dim3 block, cudaStream_t stream)
{
    const bool wide = (reinterpret_cast<uintptr_t>(a.X) % 32) == 0 && (a.ldx % 16) == 0 &&
                      (reinterpret_cast<uintptr_t>(a.Q) % 32) == 0 && (a.ldq_bytes % 32) == 0;
    return wide ? launch_dependent(group_quantize_kernel<Q, true>, grid, block, 0, stream, a)
                : launch_dependent(group_quantize_kernel<Q, false>, grid, block, 0, stream, a);
}

cudaError_t launch_group_quantize(const GroupQuantArgs &a, int sms, cudaStream_t stream)
{
    const int64_t total = static_cast<int64_t>(a.T) * ((a.K / 32 + 3) / 4 * 4);
    // Few blocks of work: small CTAs, so that they spread over the SMs.
    const int threads = total < static_cast<int64_t>(sms) * kQuantThreads ? 64 : kQuantThreads;
    const int64_t want = (total + threads - 1) / threads;
    const int64_t most = static_cast<int64_t>(sms) * 32;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most)), block(static_cast<unsigned>(threads));
    switch (a.fmt) {
    case 0: return launch_quant<QuantFmt::kE2M1>(a, grid, block, stream);
    case 1: return launch_quant<QuantFmt::kE4M3>(a, grid, block, stream);
    default: return launch_quant<QuantFmt::kE5M2>(a, grid, block, stream);
    }
}

cudaError_t launch_combine(const CombineArgs &a, int sms, cudaStream_t stream)
{
    // Enough tokens for every SM to have several, and rows long enough that a
    // ring entry's hand-over (some 200 cycles) is short beside them.
    if (a.vec && a.N % 8 == 0 && a.N >= 2048 && a.N <= 16384 && a.T >= 4 * sms) {
        const int per = (a.N / 8 + kCombineThreads - 1) / kCombineThreads;
        return per <= 1   ? launch_ring<1>(a, sms, stream)
               : per <= 2 ? launch_ring<2>(a, sms, stream)
                          : launch_ring<4>(a, sms, stream);
    }
    const int vecs = (a.N + 7) / 8;
    const int threads = vecs < kCombineThreads ? (vecs + 31) / 32 * 32 : kCombineThreads;
    const int per = (vecs + threads - 1) / threads;
    const int most = sms * (2048 / threads);
    const dim3 grid(static_cast<unsigned>(a.T < most ? a.T : most)), block(static_cast<unsigned>(threads));
    if (per <= 1)
        return launch_dependent(combine_kernel<1, 8>, grid, block, 0, stream, a);
    if (per <= 2)
        return launch_dependent(combine_kernel<2, 4>, grid, block, 0, stream, a);
    if (per <= 4)
        return launch_dependent(combine_kernel<4, 2>, grid, block, 0, stream, a);
    if (per <= kCombineMaxVec)
        return launch_dependent(combine_kernel<8, 1>, grid, block, 0, stream, a);
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
