// Expert-layer operators around the grouped products: routing, the grouped
// quantiser and the gated join with its norms.  All three are bound by HBM
// traffic at prefill sizes and by latency at decoding sizes; every kernel is a
// programmatic dependent of the work before it on the stream and waits for that
// work before it reads anything.
#include <cuda_bf16.h>

#include "expert.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace mxfp4 {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

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

// Experts lane * V .. lane * V + V - 1 of one token's logits as keys.
template <int V>
__device__ __forceinline__ void load_keys(const RouteArgs &a, int t, int lane, uint32_t (&key)[V])
{
    const int64_t at = static_cast<int64_t>(t) * a.ldl + lane * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        float x = __int_as_float(0xff800000);
        if (e < a.E)
            x = a.fp32 ? static_cast<const float *>(a.logits)[at + v]
                       : bf16_lo(static_cast<const uint16_t *>(a.logits)[at + v]);
        key[v] = order_key(x);
    }
}

// One warp, one token: its k experts into mask bits, ids and gates.
template <int V>
__device__ __forceinline__ void route_token(const RouteArgs &a, int t, int bit, int lane, uint32_t *masks)
{
    uint32_t key[V];
    load_keys<V>(a, t, lane, key);
    const bool off = a.mask && a.mask[t] == 0;
    if (off) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = 0u;
    }
    // Lane 0 of the order has the lowest experts, so among equal keys the
    // first lane's first register is the lowest index.
    float sum_all = 0.0f;
    uint32_t top = 0u;
    uint32_t my_key = 0u;                                  // lane j: the j-th pick
    int my_id = -1;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v)
            best = max(best, key[v]);
        const uint32_t m = __reduce_max_sync(kFull, best);
        if (m == 0u)
            break;
        if (j == 0) {
            top = m;
            if (a.mode == 1) {
                const float xm = key_value(m);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (key[v])
                        sum_all += key[v] == m ? 1.0f : expf(key_value(key[v]) - xm);
            }
        }
        const int owner = __ffs(__ballot_sync(kFull, best == m)) - 1;
        int at = 0;
        if (lane == owner) {
            bool found = false;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (!found && key[v] == m) {
                    found = true;
                    at = lane * V + v;
                    key[v] = 0u;
                }
        }
        at = __shfl_sync(kFull, at, owner);
        if (lane == j) {
            my_key = m;
            my_id = at;
        }
    }
    const float x = key_value(my_key), xm = key_value(top);
    float g = 0.0f;
    if (my_id >= 0)
        g = a.mode == 2 ? 1.0f / (1.0f + expf(-x)) : my_key == top ? 1.0f : expf(x - xm);
    if (a.mode != 2) {
        float sum = a.mode == 1 ? sum_all : g;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            sum += __shfl_xor_sync(kFull, sum, d);
        g = my_id >= 0 ? g / sum : 0.0f;
    }
    if (lane < a.k) {
        a.ids[static_cast<int64_t>(t) * a.k + lane] = my_id;
        a.gates[static_cast<int64_t>(t) * a.k + lane] = a.gate_scale * g;
        if (my_id >= 0)
            atomicOr(&masks[my_id * 4 + (bit >> 5)], 1u << (bit & 31));
    }
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

template <int V>
__global__ void __launch_bounds__(kRouteThreads) route_pick_kernel(const __grid_constant__ RouteArgs a)
{
    extern __shared__ uint32_t smem_u32[];
    uint32_t *masks = smem_u32;                            // [E][4]
    int *run = reinterpret_cast<int *>(smem_u32 + 4 * a.E);   // [E]
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
        for (int t = s0 + warp; t < s1; t += kRouteThreads / 32)
            route_token<V>(a, t, t - s0, lane, masks);
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
    extern __shared__ uint32_t smem_u32[];
    int *total = reinterpret_cast<int *>(smem_u32);        // [E rounded up to 8]
    int *mine = total + (a.E + 7) / 8 * 8;
    const int ep = (a.E + 7) / 8 * 8, lanes = ep / 8;      // threads of one block's counts
    const int blocks = gridDim.x, me = blockIdx.x;
    for (int i = threadIdx.x; i < 2 * ep; i += kRouteThreads)
        total[i] = 0;
    __syncthreads();
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    const int rows_at_once = kRouteThreads / lanes;
    if (static_cast<int>(threadIdx.x) < rows_at_once * lanes) {
        const int q = threadIdx.x % lanes;
        int all[8], before[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            all[i] = before[i] = 0;
#pragma unroll 4
        for (int b = threadIdx.x / lanes; b < blocks; b += rows_at_once) {
            const uint4 v = *reinterpret_cast<const uint4 *>(a.counts + static_cast<int64_t>(b) * ep + 8 * q);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int c = (w[i / 2] >> (16 * (i & 1))) & 0xFFFF;
                all[i] += c;
                before[i] += b < me ? c : 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (all[i])
                atomicAdd(&total[8 * q + i], all[i]);
            if (before[i])
                atomicAdd(&mine[8 * q + i], before[i]);
        }
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
// together and one of them stores the word.

constexpr int kQuantThreads = 256;

template <QuantFmt Q>
__global__ void __launch_bounds__(kQuantThreads) group_quantize_kernel(const __grid_constant__ GroupQuantArgs a)
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
        uint32_t out[W];
        uint32_t code = 0x7Fu;
        if (real) {
            const uint4 *src = reinterpret_cast<const uint4 *>(a.X + static_cast<int64_t>(t) * a.ldx + b * 32);
            float x[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = __ldcs(src + i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[8 * i + 2 * j] = bf16_lo(w[j]);
                    x[8 * i + 2 * j + 1] = bf16_hi(w[j]);
                }
            }
            code = quantize_block<Q>(x, out);
        }
        // total and kb4 are multiples of 4, so a word's four threads are all
        // inside or all outside.
        uint32_t word = code << (8 * (b & 3));
        word |= __shfl_xor_sync(kFull, word, 1);
        word |= __shfl_xor_sync(kFull, word, 2);
        if (!in)
            continue;
        for (int j = 0; j < a.k; ++j) {
            int row = t, e;
            if (a.slot_row) {
                const int64_t at = static_cast<int64_t>(t) * a.k + j;
                row = a.slot_row[at];
                e = a.ids[at];
                if (row < 0 || row >= a.rows || e < 0 || e >= a.groups)
                    continue;
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
                e = lo;
            }
            const int o = a.offsets[e];
            if (o < 0 || row < o || row >= a.offsets[e + 1])
                continue;
            if (real) {
                uint4 *q = reinterpret_cast<uint4 *>(a.Q + static_cast<int64_t>(row) * a.ldq_bytes +
                                                     static_cast<int64_t>(b) * (4 * W));
#pragma unroll
                for (int w = 0; w < W; w += 4)
                    q[w / 4] = make_uint4(out[w], out[w + 1], out[w + 2], out[w + 3]);
            }
            if ((b & 3) == 0) {
                const int local = row - o;
                const int64_t block = group_sf_block(o, e) + local / kSfRowBlock;
                *reinterpret_cast<uint32_t *>(a.S + block * atoms_row + sf_byte(local % kSfRowBlock, b)) = word;
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

__device__ __forceinline__ void load8(const uint16_t *p, int n, int N, int vec, float (&x)[8])
{
    if (vec && n + 8 <= N) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p + n);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = n + i < N ? bf16_lo(p[n + i]) : 0.0f;
    }
}

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

template <int VPT>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const __grid_constant__ CombineArgs a)
{
    __shared__ float slots[4][kCombineThreads / 32];
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    int parity = 0;
    for (int t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 2) {
        float b[VPT][8];
#pragma unroll
        for (int v = 0; v < VPT; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                b[v][i] = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int64_t at = static_cast<int64_t>(t) * a.k + j;
            const int row = a.slot_row ? a.slot_row[at] : t;
            if (row < 0 || row >= a.rows)
                continue;
            const float g = a.gates ? a.gates[at] : 1.0f;
            const uint16_t *y = a.Y + static_cast<int64_t>(row) * a.ldy;
#pragma unroll
            for (int v = 0; v < VPT; ++v) {
                const int n = (v * blockDim.x + threadIdx.x) * 8;
                if (n < a.N) {
                    float x[8];
                    load8(y, n, a.N, a.vec, x);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        b[v][i] = fmaf(g, x[i], b[v][i]);
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
                    float w[8];
                    load8(a.w_post, n, a.N, a.vec, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        b[v][i] = b[v][i] * r * w[i];
                }
            }
        }
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
            const int n = (v * blockDim.x + threadIdx.x) * 8;
            if (n < a.N) {
                float x[8];
                if (a.resid) {
                    load8(a.resid + static_cast<int64_t>(t) * a.ldr, n, a.N, a.vec, x);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    b[v][i] = a.resid ? fmaf(a.out_scale, b[v][i], a.res_scale * x[i]) : a.out_scale * b[v][i];
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
                    float w[8], y[8];
                    if (a.w_pre) {
                        load8(a.w_pre, n, a.N, a.vec, w);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w[i] = 1.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = b[v][i] * r * w[i];
                    store8(a.Nrm + static_cast<int64_t>(t) * a.ldn, n, a.N, a.vec, y);
                }
            }
        }
    }
}

template <int V>
cudaError_t launch_pick(const RouteArgs &a, size_t smem, cudaStream_t stream)
{
    return launch_dependent(route_pick_kernel<V>, dim3(a.blocks), dim3(kRouteThreads), smem, stream, a);
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

cudaError_t launch_route(const RouteArgs &a, cudaStream_t stream)
{
    if (a.T == 0)
        return launch_dependent(route_empty_kernel, dim3(1), dim3(256), 0, stream, a.offsets, a.E);
    const size_t smem = static_cast<size_t>(5 * a.E) * 4;
    cudaError_t e;
    if (a.E <= 32)
        e = launch_pick<1>(a, smem, stream);
    else if (a.E <= 64)
        e = launch_pick<2>(a, smem, stream);
    else if (a.E <= 128)
        e = launch_pick<4>(a, smem, stream);
    else if (a.E <= 256)
        e = launch_pick<8>(a, smem, stream);
    else if (a.E <= 512)
        e = launch_pick<16>(a, smem, stream);
    else
        e = launch_pick<32>(a, smem, stream);
    if (e != cudaSuccess || a.blocks == 1)
        return e;
    const size_t smem2 = static_cast<size_t>(2 * ((a.E + 7) / 8 * 8)) * 4;
    return launch_dependent(route_place_kernel, dim3(a.blocks), dim3(kRouteThreads), smem2, stream, a);
}

cudaError_t launch_group_quantize(const GroupQuantArgs &a, int sms, cudaStream_t stream)
{
    const int64_t total = static_cast<int64_t>(a.T) * ((a.K / 32 + 3) / 4 * 4);
    const int64_t want = (total + kQuantThreads - 1) / kQuantThreads;
    const int64_t most = static_cast<int64_t>(sms) * 32;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    switch (a.fmt) {
    case 0: return launch_dependent(group_quantize_kernel<QuantFmt::kE2M1>, grid, dim3(kQuantThreads), 0, stream, a);
    case 1: return launch_dependent(group_quantize_kernel<QuantFmt::kE4M3>, grid, dim3(kQuantThreads), 0, stream, a);
    default: return launch_dependent(group_quantize_kernel<QuantFmt::kE5M2>, grid, dim3(kQuantThreads), 0, stream, a);
    }
}

cudaError_t launch_combine(const CombineArgs &a, int sms, cudaStream_t stream)
{
    const int vecs = (a.N + 7) / 8;
    const int threads = vecs < kCombineThreads ? (vecs + 31) / 32 * 32 : kCombineThreads;
    const int per = (vecs + threads - 1) / threads;
    const int most = sms * (2048 / threads);
    const dim3 grid(static_cast<unsigned>(a.T < most ? a.T : most)), block(static_cast<unsigned>(threads));
    if (per <= 1)
        return launch_dependent(combine_kernel<1>, grid, block, 0, stream, a);
    if (per <= 2)
        return launch_dependent(combine_kernel<2>, grid, block, 0, stream, a);
    if (per <= 4)
        return launch_dependent(combine_kernel<4>, grid, block, 0, stream, a);
    if (per <= kCombineMaxVec)
        return launch_dependent(combine_kernel<8>, grid, block, 0, stream, a);
    return cudaErrorInvalidValue;
}

}  // namespace mxfp4
