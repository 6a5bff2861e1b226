// Routing of tokens to experts: the largest logits, their gates, and the stable
// grouping of the rows by expert.
#include <cuda_bf16.h>

#include "expert.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace mxfp4 {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ------------------------------------------------------------------ routing --
//
// Stable counting sort of (token, slot) rows by expert.  A token picks an
// expert at most once, so inside a run of tokens an expert's rows are a bit mask
// of tokens (set with atomicOr, whose order does not matter), and a row's place
// among them is the number of set bits before its own.  Blocks write their
// experts' counts; the second kernel adds up the counts of the blocks before its
// own and all of them (integers: any order, the same sum), and places its tokens'
// rows.  Up to 64 tokens one block does it all, without a second launch: 16
// tokens of 128 experts take 4.7 us, which is latency (an empty call takes 2.9).
// 32768 tokens of 256 fp32 logits, top 8: 25 us for 38 MB, 1.5 TB/s; the
// instructions of picking bound it (some 300 per token and warp), then the
// second launch (some 6 us).

constexpr int kPlaceAtOnce = 32;                 // blocks whose counts are read together, at most
constexpr int kRouteThreads = 512;
// Tokens of one mask.  A block's warps do a run without a barrier: 100000 tokens
// of 8 experts 19.9 us with 256, 26.2 with 128; of 256 experts 24.7 against 25.4.
constexpr int kRouteRun = 256;
constexpr int kRunWords = kRouteRun / 32;
// Tokens that one block does alone, without a workspace (64 tokens of 128 experts:
// 7.5 us in one launch and in two).
constexpr int kRouteSingle = 64;
// A block per SM of the board that this is for (a constant: the workspace's size is
// asked for without a device).
constexpr int kRouteMaxBlocks = 152;
// Shared memory of the placing kernel at most: two partial counts per thread's
// eight experts, their sums.
constexpr int kPlaceSmem = (2 * kRouteThreads * 8 + 2 * kMaxGroups) * 4;

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

// A token's picks (expert, logit), of which `taken` exist: gates, ids and mask
// bits.  Its LANES lanes share the work; sum is this lane's part of the softmax
// over all experts, top the largest logit.  ids: the run's, in shared memory.
template <int LANES>
__device__ __forceinline__ void finish_token(const RouteArgs &a, int t, bool live, int bit, int l, int taken, float top,
                                             float sum, const float2 *picks, uint32_t *masks, int *ids)
{
    if (a.mode == 0)
        for (int j = l; j < taken; j += LANES) {
            const float2 p = picks[j];
            if (__float_as_int(p.x) >= 0)
                sum += p.y == top ? 1.0f : expf(p.y - top);
        }
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1)
        sum += __shfl_xor_sync(kFull, sum, d);
    if (live)
        for (int j = l; j < a.k; j += LANES) {
            const float2 p = j < taken ? picks[j] : make_float2(__int_as_float(-1), 0.0f);
            const int id = __float_as_int(p.x);
            float g = 0.0f;
            if (id >= 0) {
                g = a.mode == 2 ? 1.0f / (1.0f + expf(-p.y)) : (p.y == top ? 1.0f : expf(p.y - top)) / sum;
                atomicOr(&masks[id * kRunWords + (bit >> 5)], 1u << (bit & 31));
            }
            ids[bit * a.k + j] = id;
            a.ids[static_cast<int64_t>(t) * a.k + j] = id;
            a.gates[static_cast<int64_t>(t) * a.k + j] = a.gate_scale * g;
        }
    __syncwarp();                                          // the picks are used again
}

// Expert (c LANES + l) 4 + i of a token -> x[c][i], -inf where there is none;
// all loads in flight together.
template <int LANES, int CH>
__device__ __forceinline__ void load_logits(const RouteArgs &a, bool on, int64_t row, int l, float (&x)[CH][4])
{
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int e = (c * LANES + l) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[c][i] = __int_as_float(0xff800000);
        if (!on || e >= a.E)
            continue;
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
                                             float2 *picks, uint32_t *masks, int *ids)
{
    const int l = lane & (LANES - 1);
    uint4 *mine = keys + lane;                             // chunk c at mine[32 c]: no bank conflicts
    const bool on = live && !(a.mask && a.mask[t] == 0);
    const int64_t row = static_cast<int64_t>(live ? t : 0) * a.ldl;
    uint32_t top[CH];                                      // the chunks' maxima
    float x[CH][4];
    load_logits<LANES, CH>(a, on, row, l, x);
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
        } else if (m == 0u && l == 0) {
            my_picks[taken] = make_float2(__int_as_float(-1), 0.0f);
        }
    }
    __syncwarp();
    finish_token<LANES>(a, t, live, bit, l, taken, key_value(first), sum, my_picks, masks, ids);
}

// Exclusive prefix sums of total[0 .. E) over the block, in place; returns
// the sum of all.
__device__ __forceinline__ int block_scan(int *total, int E)
{
    __shared__ int warp_sum[32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, n = (E + blockDim.x - 1) / blockDim.x;
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
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
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

// Bounding, k <= 8.  The k-th largest of the maxima of the token's groups of
// experts (CH / NG chunks of four, NG groups per lane) is a bound that the k-th
// largest logit is not below: the lanes sort their maxima and merge the lists in
// a butterfly.  The logits at or above the bound, little more than k, are set
// down in shared memory, and each one's place is the number of larger ones (and
// of equal ones with a lower index).  Where more than fit are left, as among
// many equal logits, the warp picks its tokens one expert at a time instead.
// Against picking, a quarter of the instructions, and for a lone token five
// exchanges in a row where picking eight experts takes eighty.
template <int LANES>
constexpr int kCandidates = LANES == 4 ? 16 : 64;        // of one token (4 lanes: all of its experts)

__device__ __forceinline__ void exchange(float &hi, float &lo)
{
    const float a = fmaxf(hi, lo), b = fminf(hi, lo);
    hi = a;
    lo = b;
}

// exp(z) for z <= 0 as 2^(z log2 e); 0 for NaN and below the smallest normal
// number, which is nothing beside the largest logit's 1.
__device__ __forceinline__ float exp_below(float z)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaxf(z, -200.0f) * 1.4426950408889634f));
    return r;
}

// NaN counts as nothing.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Bitonic sequence of eight -> descending.
__device__ __forceinline__ void settle8(float (&v)[8])
{
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((i & d) == 0)
                exchange(v[i], v[i | d]);
}

template <int LANES, int CH>
__device__ __forceinline__ void bound_tokens(const RouteArgs &a, int t, bool live, int bit, int lane, uint4 *keys,
                                             float2 *picks, float2 *found, uint32_t *masks, int *ids)
{
    constexpr int NG = CH < 4 ? CH : 4;
    constexpr int CAP = kCandidates<LANES>;
    const float ninf = __int_as_float(0xff800000);
    const int l = lane & (LANES - 1);
    const bool on = live && !(a.mask && a.mask[t] == 0);
    float2 *my_picks = picks + (lane / LANES) * a.k;
    found += (lane / LANES) * CAP;
    float x[CH][4];
    load_logits<LANES, CH>(a, on, static_cast<int64_t>(live ? t : 0) * a.ldl, l, x);
    float best[8];                                         // descending
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        best[g] = ninf;
        if (g >= NG)
            continue;
#pragma unroll
        for (int c = g * (CH / NG); c < (g + 1) * (CH / NG); ++c) {
            best[g] = max3(max3(best[g], x[c][0], x[c][1]), x[c][2], x[c][3]);
            reinterpret_cast<float4 *>(keys)[32 * c + lane] = make_float4(x[c][0], x[c][1], x[c][2], x[c][3]);
        }
    }
    if constexpr (NG >= 2)
        exchange(best[0], best[1]);
    if constexpr (NG == 4) {
        exchange(best[2], best[3]);
        exchange(best[0], best[2]);
        exchange(best[1], best[3]);
        exchange(best[1], best[2]);
    }
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) {
        // The elementwise maxima of one list and the other reversed are the
        // eight largest of both, as a bitonic sequence (both lanes read each
        // other's list as it was).
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = __shfl_xor_sync(kFull, best[i], d);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            best[i] = fmaxf(best[i], w[7 - i]);
        settle8(best);
    }
    const float top = best[0];
    float bar = best[0];
#pragma unroll
    for (int j = 1; j < 8; ++j)
        bar = j < a.k ? best[j] : bar;
    float sum = 0.0f;
    if (a.mode == 1 && top > ninf) {
        // Terms far below the largest do not matter to the sum, so the fast
        // exponential keeps it to a few 2^-24 of itself.
        if (top < __int_as_float(0x7f800000)) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum += exp_below(x[c][i] - top);
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum += x[c][i] == top ? 1.0f : 0.0f;   // infinite logits share the whole
        }
    }
    const float low = fmaxf(bar, -3.402823466e38f);        // -inf is no candidate
    uint32_t hits = 0u;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            hits |= x[c][i] >= low ? 1u << (4 * c + i) : 0u;
    // This lane's place among the token's candidates, and their number.
    const int own = __popc(hits);
    int upto = own;
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) {
        const int v = __shfl_up_sync(kFull, upto, d, LANES);
        if (l >= d)
            upto += v;
    }
    const int n = __shfl_sync(kFull, upto, LANES - 1, LANES);
    __syncwarp();
    if (__any_sync(kFull, n > CAP)) {
        route_tokens<LANES, CH>(a, t, live, bit, lane, keys, picks, masks, ids);
        return;
    }
    for (int at = upto - own; hits; ++at) {
        const int b = __ffs(hits) - 1;
        hits &= hits - 1u;
        const float z = reinterpret_cast<const float *>(keys + 32 * (b >> 2) + lane)[b & 3];
        found[at] = make_float2(__int_as_float(((b >> 2) * LANES + l) * 4 + (b & 3)), z);
    }
    __syncwarp();
    for (int i = l; i < n; i += LANES) {
        const float2 f = found[i];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const float2 o = found[j];
            place += o.y > f.y || (o.y == f.y && __float_as_int(o.x) < __float_as_int(f.x)) ? 1 : 0;
        }
        if (place < a.k)
            my_picks[place] = f;
    }
    __syncwarp();
    finish_token<LANES>(a, t, live, bit, l, min(n, a.k), top, sum, my_picks, masks, ids);
}

// The place of slot i of the run among its expert's rows of the run: the
// tokens before its own in the expert's mask.
__device__ __forceinline__ int place_in_run(const uint32_t *masks, int e, int bit)
{
    int place = 0;
#pragma unroll
    for (int w = 0; w < kRunWords; ++w) {
        const uint32_t m = masks[kRunWords * e + w];
        place += w < (bit >> 5) ? __popc(m) : w == (bit >> 5) ? __popc(m & ((1u << (bit & 31)) - 1u)) : 0;
    }
    return place;
}

// BOUND: bound_tokens (k <= 8), else route_tokens.
template <int THREADS, int BLOCKS, int LANES, int CH, bool BOUND>
__global__ void __launch_bounds__(THREADS, BLOCKS) route_pick_kernel(const __grid_constant__ RouteArgs a)
{
    constexpr int TPW = 32 / LANES;                        // tokens of a warp
    constexpr int WARPS = THREADS / 32;
    extern __shared__ __align__(16) uint32_t smem_u32[];
    uint4 *all_keys = reinterpret_cast<uint4 *>(smem_u32); // [warps][CH][32]
    float2 *all_picks = reinterpret_cast<float2 *>(all_keys + THREADS * CH);         // [warps][TPW][k]
    float2 *all_found = all_picks + WARPS * TPW * a.k;                               // [warps][TPW][candidates]
    uint32_t *masks = reinterpret_cast<uint32_t *>(all_found + (BOUND ? WARPS * TPW * kCandidates<LANES> : 0));   // [E][kRunWords]
    int *run = reinterpret_cast<int *>(masks + kRunWords * a.E);   // [E]
    int *ids = run + a.E;                                  // [tokens of a run][k]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * a.chunk;
    const int t1 = min(a.T, t0 + a.chunk);
    for (int i = threadIdx.x; i < (kRunWords + 1) * a.E; i += THREADS)
        masks[i] = 0u;                                     // run too
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    for (int s0 = t0; s0 < t1; s0 += kRouteRun) {
        __syncthreads();
        const int s1 = min(t1, s0 + kRouteRun);
        for (int q = s0 + warp * TPW; q < s1; q += WARPS * TPW) {
            const int t = q + lane / LANES;
            if (t + WARPS * TPW < t1) {                    // this warp's next logits, on their way to L2
                const int64_t size = a.fp32 ? 4 : 2;
                const char *next = static_cast<const char *>(a.logits) + static_cast<int64_t>(t + WARPS * TPW) * a.ldl * size;
                for (int64_t o = 128 * (lane & (LANES - 1)); o < a.E * size; o += 128 * LANES)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(next + o));
            }
            uint4 *keys = all_keys + warp * CH * 32;
            float2 *picks = all_picks + warp * TPW * a.k;
            if constexpr (BOUND)
                bound_tokens<LANES, CH>(a, t, t < s1, t - s0, lane, keys, picks,
                                        all_found + warp * TPW * kCandidates<LANES>, masks, ids);
            else
                route_tokens<LANES, CH>(a, t, t < s1, t - s0, lane, keys, picks, masks, ids);
        }
        __syncthreads();
        if (a.blocks == 1)
            break;                                         // one run: kRouteSingle tokens at most
        for (int i = threadIdx.x; i < (s1 - s0) * a.k; i += THREADS) {
            const int e = ids[i];
            a.slot_row[static_cast<int64_t>(s0) * a.k + i] = e >= 0 ? run[e] + place_in_run(masks, e, i / a.k) : -1;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += THREADS) {
            int n = 0;
#pragma unroll
            for (int w = 0; w < kRunWords; ++w) {
                n += __popc(masks[kRunWords * e + w]);
                masks[kRunWords * e + w] = 0u;
            }
            run[e] += n;
        }
    }
    if (a.blocks > 1) {
        __syncthreads();
        const int ep = (a.E + 7) / 8 * 8;
        uint16_t *count = a.counts + static_cast<int64_t>(blockIdx.x) * ep;
        for (int e = threadIdx.x; e < ep; e += THREADS)
            count[e] = e < a.E ? static_cast<uint16_t>(run[e]) : uint16_t(0);
        return;
    }
    for (int e = threadIdx.x; e < a.E; e += THREADS) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < kRouteSingle / 32; ++w)        // a lone block's tokens
            n += __popc(masks[kRunWords * e + w]);
        run[e] = n;
    }
    __syncthreads();
    const int all = block_scan(run, a.E);
    for (int e = threadIdx.x; e <= a.E; e += THREADS)
        a.offsets[e] = e < a.E ? run[e] : all;
    for (int i = threadIdx.x; i < a.T * a.k; i += THREADS) {
        const int e = ids[i], t = i / a.k;
        const int row = e >= 0 ? run[e] + place_in_run(masks, e, t) : -1;
        a.slot_row[i] = row;
        if (row >= 0)
            a.row_token[row] = t;
        if (i >= all)
            a.row_token[i] = -1;
    }
}

__host__ __device__ constexpr int place_at_once(int ep)
{
    return kRouteThreads / (ep / 8) < kPlaceAtOnce ? kRouteThreads / (ep / 8) : kPlaceAtOnce;
}

// Each block adds up all picking blocks' counts and those before its own, then
// places the rows of the tokens that picking block had.
__global__ void __launch_bounds__(kRouteThreads) route_place_kernel(const __grid_constant__ RouteArgs a)
{
    extern __shared__ __align__(16) uint32_t smem_u32[];
    const int ep = (a.E + 7) / 8 * 8, lanes = ep / 8;      // threads of one block's counts
    const int me = blockIdx.x;
    const int at_once = place_at_once(ep);                 // blocks whose counts are read together
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
        // Two counts share a word while their sums stay below 2^16.
        const int safe = 65535 / a.chunk * at_once;
        for (int f = g; f < a.blocks; f += safe) {
            uint4 s = make_uint4(0u, 0u, 0u, 0u), p = s;
#pragma unroll 8
            for (int b = f; b < min(a.blocks, f + safe); b += at_once) {
                const uint4 v = *reinterpret_cast<const uint4 *>(a.counts + static_cast<int64_t>(b) * ep + 8 * q);
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
                if (b < me) {
                    p.x += v.x;
                    p.y += v.y;
                    p.z += v.z;
                    p.w += v.w;
                }
            }
            const uint32_t sw[4] = {s.x, s.y, s.z, s.w}, pw[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                all[i] += (sw[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
                before[i] += (pw[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
            }
        }
        uint4 *mine_part = reinterpret_cast<uint4 *>(part + 2 * g * ep + 8 * q);
        mine_part[0] = make_uint4(all[0], all[1], all[2], all[3]);
        mine_part[1] = make_uint4(all[4], all[5], all[6], all[7]);
        mine_part = reinterpret_cast<uint4 *>(part + (2 * g + 1) * ep + 8 * q);
        mine_part[0] = make_uint4(before[0], before[1], before[2], before[3]);
        mine_part[1] = make_uint4(before[4], before[5], before[6], before[7]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * ep; i += kRouteThreads) {
        uint32_t s = 0u;
#pragma unroll 4
        for (int g = 0; g < at_once; ++g)
            s += part[2 * g * ep + i];
        total[i] = static_cast<int>(s);                    // total, then mine
    }
    __syncthreads();
    const int sum = block_scan(total, a.E);
    if (me == 0)
        for (int e = threadIdx.x; e <= a.E; e += kRouteThreads)
            a.offsets[e] = e < a.E ? total[e] : sum;
    // (T k fits an int.)
    const int span = a.chunk * a.k;
    const int i0 = me * span;
    const int i1 = static_cast<int>(min(static_cast<int64_t>(a.T) * a.k, static_cast<int64_t>(i0) + span));
#pragma unroll 4
    for (int i = i0 + threadIdx.x; i < i1; i += kRouteThreads) {
        const int e = a.ids[i], place = a.slot_row[i];
        if (e >= 0) {
            const int row = total[e] + mine[e] + place;
            a.slot_row[i] = row;
            a.row_token[row] = i / a.k;
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

template <int THREADS, int BLOCKS, int LANES, int CH, bool BOUND>
cudaError_t launch_pick(const RouteArgs &a, cudaStream_t stream)
{
    constexpr auto kern = route_pick_kernel<THREADS, BLOCKS, LANES, CH, BOUND>;
    auto bytes = [](int k, int E) {
        return THREADS * CH * 16 + THREADS / LANES * (k + (BOUND ? kCandidates<LANES> : 0)) * 8 +
               (kRunWords + 1) * E * 4 + kRouteRun * k * 4;
    };
    // The most that any E and k need of this instance.
    const cudaError_t e = opt_in<kern>(bytes(BOUND ? 8 : kMaxTopK, LANES * CH * 4));
    if (e != cudaSuccess)
        return e;
    return launch_dependent(kern, dim3(a.blocks), dim3(THREADS), static_cast<size_t>(bytes(a.k, a.E)), stream, a);
}

// A warp per token, four experts per chunk and lane.
template <bool BOUND>
cudaError_t launch_warps(const RouteArgs &a, cudaStream_t stream)
{
    return a.E <= 128   ? launch_pick<kRouteThreads, 2, 32, 1, BOUND>(a, stream)
           : a.E <= 256 ? launch_pick<kRouteThreads, 2, 32, 2, BOUND>(a, stream)
           : a.E <= 512 ? launch_pick<kRouteThreads, 2, 32, 4, BOUND>(a, stream)
                        : launch_pick<kRouteThreads, 1, 32, 8, BOUND>(a, stream);
}

// LANES lanes per token, `chunks` chunks of four experts per lane.  One block of
// 32 warps per SM: with three of 8 the placing kernel has three times the counts
// to read (32768 tokens of 256 experts: 26.9 against 31.5 us for both kernels).
template <int LANES, bool BOUND>
cudaError_t launch_chunks(const RouteArgs &a, int chunks, cudaStream_t stream)
{
    if (chunks <= 2)
        return launch_pick<1024, 1, LANES, 2, BOUND>(a, stream);
    if (chunks <= 4)
        return launch_pick<1024, 1, LANES, 4, BOUND>(a, stream);
    return launch_pick<1024, 1, LANES, 8, BOUND>(a, stream);
}

template <bool BOUND>
cudaError_t launch_lanes(const RouteArgs &a, int lanes, cudaStream_t stream)
{
    const int chunks = (a.E + 4 * lanes - 1) / (4 * lanes);
    switch (lanes) {
    case 4: return launch_pick<1024, 1, 4, 2, BOUND>(a, stream);
    case 8: return launch_chunks<8, BOUND>(a, chunks, stream);
    case 16: return launch_chunks<16, BOUND>(a, chunks, stream);
    default: return launch_pick<1024, 1, 32, 8, BOUND>(a, stream);
    }
}

}  // namespace

int route_blocks(int T, int *chunk)
{
    int c = T <= kRouteSingle ? kRouteSingle : 32;
    if (T > 32 * kRouteMaxBlocks)
        c = (T + kRouteMaxBlocks - 1) / kRouteMaxBlocks;
    *chunk = c;
    return (T + c - 1) / c;
}

cudaError_t launch_route(const RouteArgs &a, int sms, cudaStream_t stream)
{
    if (a.T == 0)
        return launch_dependent(route_empty_kernel, dim3(1), dim3(256), 0, stream, a.offsets, a.E);
    // Lanes per token: as many as let the block's warps do its tokens (128 of
    // them, if a block has more) in one pass, which has the latency, and at least as many as hold
    // the experts in 32 registers each.  32768 tokens: 64 experts 14.6 us, with
    // the fewest lanes 22; 8 experts 10.8 against 37.  5000 tokens of 256 experts:
    // 11.8 us, with the fewest lanes 12.7, with a warp per token 14.4.  A warp per
    // token also runs in blocks of 16 warps, for up to 16 tokens.
    const int tokens = min(min(a.T, a.chunk), 128);
    int lanes = 4;
    while (lanes < 32 && (lanes * 32 < a.E || (lanes * 4 < a.E && tokens * lanes * 2 / 32 <= (lanes < 16 ? 32 : 16))))
        lanes *= 2;
    // (16 tokens of 128 experts 4.8 us by bounding, 6.0 by picking; 32768 of 256 24.3
    // and 31.3.)
    const bool bound = a.k <= 8, many = lanes < 32 || tokens > 16;
    const cudaError_t picked = many ? (bound ? launch_lanes<true>(a, lanes, stream) : launch_lanes<false>(a, lanes, stream))
                                    : (bound ? launch_warps<true>(a, stream) : launch_warps<false>(a, stream));
    if (picked != cudaSuccess || a.blocks == 1)
        return picked;
    const int ep = (a.E + 7) / 8 * 8;
    const size_t smem = static_cast<size_t>(2 * place_at_once(ep) + 2) * ep * 4;
    const cudaError_t e = opt_in<route_place_kernel>(kPlaceSmem);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(route_place_kernel, dim3(a.blocks), dim3(kRouteThreads), smem, stream, a);
}

}  // namespace mxfp4
