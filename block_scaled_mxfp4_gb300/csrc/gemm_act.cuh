// Epilogue of the products with bias, activation and residual (included by
// gemm_sm103.cu).
//
//   z = alpha * acc + bias[n]                       -> Z, 1x32 blocks along n
//   d = act(z) + res_scale * R[m, n]                -> D (bf16), H (1x32 blocks along n)
//
// in fp32, each output rounded once.  A block of 32 columns is a thread's
// (row-wise forms), eight neighbouring lanes' (cluster reduction), or a warp's
// (swapped forms, where a lane holds one n).  The activation is a uniform
// branch on its code, around 32 values at a time: one kernel per tile shape
// and not five.
#pragma once

#include "act.cuh"
#include "quant.cuh"

namespace mxfp4 {

template <int N>
__device__ __forceinline__ void act_apply(int act, float (&v)[N])
{
    auto each = [&](auto tag) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 h = parts(act_value2<decltype(tag)::value>(f2(v[i], v[i + 1])));
            v[i] = h.x;
            v[i + 1] = h.y;
        }
    };
    switch (act) {
    case 1: each(ActTag<Act::kRelu>{}); break;
    case 2: each(ActTag<Act::kGelu>{}); break;
    case 3: each(ActTag<Act::kGeluTanh>{}); break;
    case 4: each(ActTag<Act::kSilu>{}); break;
    default: break;
    }
}

__device__ __forceinline__ float act_bias(const ActGemmArgs &a, int n)
{
    return a.bias_fp32 ? __ldg(static_cast<const float *>(a.bias) + n)
                       : bf16_bits_to_float(__ldg(static_cast<const uint16_t *>(a.bias) + n));
}

// What to add where there is no bias: x + -0 is x for every x, where x + 0 makes 0 of -0.
constexpr float kNoBias = -0.0f;

// bias[n0 .. n0 + 31], zeros past N.
__device__ __forceinline__ void act_bias_chunk(const ActGemmArgs &a, int n0, float (&b)[32])
{
    if (a.bias_vec && n0 + 32 <= a.N) {
        if (a.bias_fp32) {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.bias) + n0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 v = __ldg(p + i);
                b[4 * i] = v.x;
                b[4 * i + 1] = v.y;
                b[4 * i + 2] = v.z;
                b[4 * i + 3] = v.w;
            }
        } else {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.bias) + n0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = __ldg(p + i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    b[8 * i + 2 * j] = bf16_lo(w[j]);
                    b[8 * i + 2 * j + 1] = bf16_hi(w[j]);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            b[i] = n0 + i < a.N ? act_bias(a, n0 + i) : 0.0f;
    }
}

// One block in a thread: codes of row m, columns n0 ..+31; the scale code.
template <QuantFmt Q>
__device__ __forceinline__ uint32_t act_put_block(const ActCodes &o, int m, int n0, const float (&v)[32])
{
    constexpr int W = QuantTraits<Q>::kWords;
    uint32_t w[W], code;
    if constexpr (Q == QuantFmt::kE2M1)
        code = quantize_block<Q>(v, w);
    else
        code = quantize_block_pairs<Q>(v, w);
    uint8_t *q = o.q + m * o.ldq + (Q == QuantFmt::kE2M1 ? n0 / 2 : n0);
    if constexpr (W == 8) {
        if (o.wide) {
            st_global_v8_hint(q, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7], l2_policy_evict_first());
            return code;
        }
        reinterpret_cast<uint4 *>(q)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    reinterpret_cast<uint4 *>(q)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    return code;
}

__device__ __forceinline__ uint32_t act_put_codes(const ActCodes &o, int m, int n0, const float (&v)[32])
{
    if (o.fmt == 0)
        return act_put_block<QuantFmt::kE4M3>(o, m, n0, v);
    if (o.fmt == 1)
        return act_put_block<QuantFmt::kE5M2>(o, m, n0, v);
    return act_put_block<QuantFmt::kE2M1>(o, m, n0, v);
}

// Scale codes of up to four neighbouring blocks of row m, the first of column n0,
// in the bytes of `codes`.  One store where it may be: the rows of a warp's lanes are
// apart, and every store of them costs as many lines as it has lanes.
__device__ __forceinline__ void act_put_scales(const ActCodes &o, int m, int n0, int N, int count, uint32_t codes)
{
    uint8_t *s = o.s + m * o.lds + n0 / 32;
    if (count == 4 && o.pack && n0 + 128 <= N) {
        *reinterpret_cast<uint32_t *>(s) = codes;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < count && n0 + 32 * i < N)
            s[i] = static_cast<uint8_t>(codes >> (8 * i));
}

// The scales of a run of chunks, as they come.
struct ActScales {
    uint32_t z = 0, h = 0;
};

// Rows of D and R off 16-byte boundaries, and the last columns of others: 16
// columns of the warp's 32 rows go through a piece of shared memory, so that lanes
// move neighbouring elements of a row.  (One lane a row instead, 32 rows apart in
// every access of two bytes: a product of 2048 x 4010 x 1024 with GELU and residual
// took 87 us for 37, 26 with 4096 columns.)  Rows are 9 words apart: no bank conflicts
// either way.
constexpr int kActPitch = 18;                    // 16-bit elements
constexpr int kActPieceBytes = 32 * kActPitch * 2;

// Rows m0 .. + 31 and columns n0 + 16 h .. + 15 of R, the lane's row into r as packed pairs.
__device__ __forceinline__ void act_fetch_piece(const uint16_t *src, int64_t ld, int M, int N, int m0, int n, int lane, uint16_t *piece,
                                                uint32_t (&r)[8])
{
    const int c = lane & 15;
    uint16_t x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int m = m0 + 2 * i + (lane >> 4);
        x[i] = m < M && n + c < N ? src[m * ld + n + c] : uint16_t(0);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        piece[(2 * i + (lane >> 4)) * kActPitch + c] = x[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        r[i] = *reinterpret_cast<const uint32_t *>(piece + lane * kActPitch + 2 * i);
    __syncwarp();
}

__device__ __forceinline__ void act_put_piece(uint16_t *dst, int64_t ld, int M, int N, int m0, int n, int lane, uint16_t *piece,
                                              const uint32_t (&d)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint32_t *>(piece + lane * kActPitch + 2 * i) = d[i];
    __syncwarp();
    const int c = lane & 15;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int m = m0 + 2 * i + (lane >> 4);
        const uint16_t x = piece[(2 * i + (lane >> 4)) * kActPitch + c];
        if (m < M && n + c < N)
            dst[m * ld + n + c] = x;
    }
    __syncwarp();
}

// The L2 lines of R's row m from column n on.
__device__ __forceinline__ void act_prefetch_row(const ActGemmArgs &a, int m, int n, int count)
{
    if (!a.R || m >= a.M || n >= a.N)
        return;
    const uint16_t *r = a.R + m * a.ldr + n;
    const int have = min(count, a.N - n);
    for (int c = 0; c < have; c += 64)
        prefetch_l2(r + c);
    prefetch_l2(r + have - 1);
}

// Columns n0 .. + 31 of R's row m for act_row_chunk, issued ahead of it: a load's 32
// rows are 32 lines, which take long under the operands' traffic.
__device__ __forceinline__ void act_fetch_row(const ActGemmArgs &a, int m, int n0, uint4 (&r4)[4])
{
    if (!a.R || !a.r_vec || m >= a.M || n0 + 32 > a.N)
        return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r4[i] = *reinterpret_cast<const uint4 *>(a.R + m * a.ldr + n0 + 8 * i);
}

// Rows m0 .. m0 + 31 (m0 < M), one a lane, columns n0 .. n0 + 31 (n0 < N): v holds
// the accumulators.  All lanes call it; `piece`: kActPieceBytes of the warp's own.
// The blocks' scale codes go to byte `at` of `scales`; `r4`: what act_fetch_row left; `bias`: the 32
// columns' in shared memory, or null.
__device__ __forceinline__ void act_row_chunk(const ActGemmArgs &a, int m0, int n0, int lane, float (&v)[32], const uint4 (&r4)[4],
                                              uint16_t *piece, int at, ActScales &scales, const float *bias = nullptr)
{
    const int m = m0 + lane;
    const bool real = m < a.M, full = n0 + 32 <= a.N;
    if (a.bias && bias) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 b = *reinterpret_cast<const float4 *>(bias + i);
            v[i] = fmaf(a.alpha, v[i], b.x);
            v[i + 1] = fmaf(a.alpha, v[i + 1], b.y);
            v[i + 2] = fmaf(a.alpha, v[i + 2], b.z);
            v[i + 3] = fmaf(a.alpha, v[i + 3], b.w);
        }
    } else if (a.bias) {
        float b[32];
        act_bias_chunk(a, n0, b);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] = fmaf(a.alpha, v[i], b[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] *= a.alpha;
    }
    if (a.Z.q) {
        if (!full) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (n0 + i >= a.N)
                    v[i] = 0.0f;                         // the block's end: zeros, not counted
        }
        if (real)
            scales.z |= act_put_codes(a.Z, m, n0, v) << (8 * at);
    }
    act_apply(a.act, v);
    if (a.R) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t r[8];
            if (a.r_vec && full) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 w = r4[2 * h + i];
                    r[4 * i] = w.x;
                    r[4 * i + 1] = w.y;
                    r[4 * i + 2] = w.z;
                    r[4 * i + 3] = w.w;
                }
            } else {
                act_fetch_piece(a.R, a.ldr, a.M, a.N, m0, n0 + 16 * h, lane, piece, r);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = 16 * h + 2 * i;
                const float2 y = parts(fma2(f2(a.res_scale), f2(bf16_lo(r[i]), bf16_hi(r[i])), f2(v[k], v[k + 1])));
                v[k] = y.x;
                v[k + 1] = y.y;
            }
        }
    }
    if (a.D) {
        if (a.vec_ok && full) {
            if (real)
                put_d_row(a, m, n0, v);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t d[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = pack_bf16x2(v[16 * h + 2 * i], v[16 * h + 2 * i + 1]);
                act_put_piece(a.D, a.ldd, a.M, a.N, m0, n0 + 16 * h, lane, piece, d);
            }
        }
    }
    if (a.H.q && real)
        scales.h |= act_put_codes(a.H, m, n0, v) << (8 * at);
}

// After `count` chunks from column n0 on.
__device__ __forceinline__ void act_row_scales(const ActGemmArgs &a, int m, int n0, int count, const ActScales &scales)
{
    if (m >= a.M)
        return;
    if (a.Z.q)
        act_put_scales(a.Z, m, n0, a.N, count, scales.z);
    if (a.H.q)
        act_put_scales(a.H, m, n0, a.N, count, scales.h);
}

// A block across a warp: lane's value of column n (0 where there is none), row m.
// Every lane of the warp calls it; `in`: n is below the row's whole blocks.
__device__ __forceinline__ void act_put_lane(const ActCodes &o, int m, int n, bool in, float v)
{
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu);
    const bool finite = top < 0x7F800000u;               // not for infinities and NaN
    const float amax = finite ? __uint_as_float(top) : 0.0f;
    const int s = o.fmt == 2 ? block_exponent(amax) : block_exponent8(amax, o.fmt == 0 ? 8 : 15);
    const float y = v * exp2_neg(s);
    const uint32_t code = finite ? static_cast<uint32_t>(s + 127) : 0xFFu;
    if (o.fmt == 2) {
        const uint32_t two = e2m1x2(y, __shfl_down_sync(0xffffffffu, y, 1));
        if (in && (n & 1) == 0)
            o.q[m * o.ldq + n / 2] = static_cast<uint8_t>(two);
    } else if (in) {
        o.q[m * o.ldq + n] = static_cast<uint8_t>(o.fmt == 0 ? f8x2<0>(y, 0.0f) : f8x2<1>(y, 0.0f));
    }
    if (in && (n & 31) == 0)
        o.s[m * o.lds + n / 32] = static_cast<uint8_t>(code);
}

// Swapped forms: lane's column n, rows m0 .. m0 + COUNT - 1; v holds the
// accumulators.  The 32 lanes hold the columns of one block; every lane calls it.
template <int COUNT>
__device__ __forceinline__ void act_col_chunk(const ActGemmArgs &a, int m0, int n, float (&v)[COUNT])
{
    const int mcount = min(COUNT, a.M - m0);
    const bool real = n < a.N, in = n - (n & 31) < a.N;
    const float b = a.bias ? (real ? act_bias(a, n) : 0.0f) : kNoBias;
    uint16_t r[COUNT];
#pragma unroll
    for (int i = 0; i < COUNT; ++i)                      // before any store: R may alias D
        r[i] = a.R && real && i < mcount ? a.R[(m0 + i) * a.ldr + n] : uint16_t(0);
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
        v[i] = real ? fmaf(a.alpha, v[i], b) : 0.0f;
    if (a.Z.q) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i)
            if (i < mcount)
                act_put_lane(a.Z, m0 + i, n, in, v[i]);
    }
    act_apply(a.act, v);
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
        if (i < mcount) {
            if (a.R)
                v[i] = fmaf(a.res_scale, bf16_bits_to_float(r[i]), v[i]);
            if (a.D && real) {
                const __nv_bfloat16 d = __float2bfloat16_rn(v[i]);
                a.D[(m0 + i) * a.ldd + n] = *reinterpret_cast<const uint16_t *>(&d);
            }
            if (a.H.q)
                act_put_lane(a.H, m0 + i, n, in, v[i]);
        }
}

// Four columns n .. n + 3 of row m, the block's other values in the seven
// lanes beside (all 32 lanes call it).  `in`: n is below the row's whole blocks.
__device__ __forceinline__ void act_put_four(const ActCodes &o, int m, int n, bool in, const float (&v)[4])
{
    float amax = max_abs3(max_abs3(0.0f, v[0], v[1]), v[2], v[3]);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1)
        amax = max_abs3(0.0f, amax, __shfl_xor_sync(0xffffffffu, amax, d));
    const bool finite = amax <= 3.402823466e38f;
    if (!finite)
        amax = 0.0f;
    const int s = o.fmt == 2 ? block_exponent(amax) : block_exponent8(amax, o.fmt == 0 ? 8 : 15);
    const float inv = exp2_neg(s);
    if (!in)
        return;
    if (o.fmt == 2) {
        *reinterpret_cast<uint16_t *>(o.q + m * o.ldq + n / 2) =
            static_cast<uint16_t>(e2m1x2(v[0] * inv, v[1] * inv) | (e2m1x2(v[2] * inv, v[3] * inv) << 8));
    } else {
        const uint32_t w = o.fmt == 0 ? f8x2<0>(v[0] * inv, v[1] * inv) | (f8x2<0>(v[2] * inv, v[3] * inv) << 16)
                                      : f8x2<1>(v[0] * inv, v[1] * inv) | (f8x2<1>(v[2] * inv, v[3] * inv) << 16);
        *reinterpret_cast<uint32_t *>(o.q + m * o.ldq + n) = w;
    }
    if ((n & 31) == 0)
        o.s[m * o.lds + n / 32] = static_cast<uint8_t>(finite ? s + 127 : 0xFF);
}

// Rows of a tile that one rank of a cluster of `split` sums: whole 32-blocks
// where the rows are n.
template <bool SWAP>
__device__ __forceinline__ int act_rank_rows(int split)
{
    const int rows = (kTileM + split - 1) / split;
    return SWAP ? (rows + 31) / 32 * 32 : rows;
}

__device__ __forceinline__ void st_smem_v4(uint32_t at, const float (&x)[4])
{
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]) : "memory");
}
__device__ __forceinline__ void ld_smem_v4(uint32_t at, float (&x)[4])
{
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(at) : "memory");
}

// reduce_tile_cluster with this epilogue: the partials are summed in split
// order, four columns of a tile row at a time.
template <bool SWAP>
__device__ __forceinline__ void act_reduce_cluster(const ActGemmArgs &a, uint32_t part_smem, int stride, int p0, int q0, int t)
{
    const int S = a.split_k;
    const int R = act_rank_rows<SWAP>(S);
    const int r0 = min(kTileM, static_cast<int>(cluster_ctarank()) * R);
    const int r1 = min(kTileM, r0 + R);
    const int warp = t >> 5, lane = t & 31;
    const int qvalid = min(a.part_cols, (SWAP ? a.M : a.N) - q0);
    auto sum4 = [&](int row, int ch, float (&x)[4]) {
        const uint32_t off = part_smem + static_cast<uint32_t>((row * stride + 4 * ch) * 4);
        float4 v[8];
#pragma unroll
        for (int z = 0; z < 8; ++z)
            if (z < S)
                v[z] = ld_dsmem_v4(map_to_rank(off, static_cast<uint32_t>(z)));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = 0.0f;
#pragma unroll
        for (int z = 0; z < 8; ++z)
            if (z < S) {
                x[0] += v[z].x;
                x[1] += v[z].y;
                x[2] += v[z].z;
                x[3] += v[z].w;
            }
    };
    if constexpr (SWAP) {
        const int nch = (qvalid + 3) / 4;
        // Two passes: sums, a row's neighbouring pieces to neighbouring lanes, to this rank's own part
        // (only this thread reads that place); then a block's 32 columns to a warp's lanes.  Peers' memory
        // read in the second order, 16 bytes from each row, made the product of 64 x 8192 x 4096 MXFP8
        // 17.4 us, of 16 rows 11.5; so they take 14.7 and 10.8, the plain products 14.7 and 10.3 (15.8 and
        // 11.1 with bias and GELU).
        const int items = max(0, min(r1, a.N - p0) - r0) * nch;
#pragma unroll 1
        for (int it = t; it < items; it += kGemmThreadsC) {
            float x[4];
            sum4(r0 + it / nch, it % nch, x);
            st_smem_v4(part_smem + static_cast<uint32_t>(((r0 + it / nch) * stride + 4 * (it % nch)) * 4), x);
        }
        __syncthreads();
        const int units = (r1 - r0) / 32 * nch;
#pragma unroll 1
        for (int u = warp; u < units; u += kGemmThreadsC / 32) {
            const int row = r0 + u / nch * 32 + lane, ch = u % nch;
            if (p0 + row - lane >= a.N)
                continue;                                // a whole block past the last column
            float x[4];
            ld_smem_v4(part_smem + static_cast<uint32_t>((row * stride + 4 * ch) * 4), x);
            act_col_chunk<4>(a, q0 + 4 * ch, p0 + row, x);
        }
    } else {
        const int nrows = max(0, min(r1, a.M - p0) - r0);
        const int nch = (qvalid + 31) / 32 * 8;          // whole blocks of eight lanes
        const int items = nrows * nch;
        for (int base = warp * 32; base < items; base += kGemmThreadsC) {
            const int it = base + lane;
            const bool in = it < items;
            const int row = r0 + (in ? it / nch : 0), ch = in ? it % nch : 0;
            const int m = p0 + row, n = q0 + 4 * ch;
            const int cnt = in ? max(0, min(4, qvalid - 4 * ch)) : 0;
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (cnt > 0)
                sum4(row, ch, x);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = j < cnt ? fmaf(a.alpha, x[j], a.bias ? act_bias(a, n + j) : kNoBias) : 0.0f;
            if (a.Z.q)
                act_put_four(a.Z, m, n, in, x);
            act_apply(a.act, x);
            if (a.R) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < cnt)
                        x[j] = fmaf(a.res_scale, bf16_bits_to_float(a.R[m * a.ldr + n + j]), x[j]);
            }
            if (a.D) {
                if (a.vec_ok && cnt == 4) {
                    *reinterpret_cast<uint2 *>(a.D + m * a.ldd + n) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < cnt) {
                            const __nv_bfloat16 d = __float2bfloat16_rn(x[j]);
                            a.D[m * a.ldd + n + j] = *reinterpret_cast<const uint16_t *>(&d);
                        }
                }
            }
            if (a.H.q)
                act_put_four(a.H, m, n, in, x);
        }
    }
}

// Bring the lines of R that this CTA's share of the cluster reduction reads
// into L2 (called while the CTA waits for its peers).
template <bool SWAP>
__device__ __forceinline__ void act_prefetch_share(const ActGemmArgs &a, int p0, int q0, int t)
{
    const int R = act_rank_rows<SWAP>(a.split_k);
    const int r0 = min(kTileM, static_cast<int>(cluster_ctarank()) * R);
    const int nrows = max(0, min(min(kTileM, r0 + R), (SWAP ? a.N : a.M) - p0) - r0);
    const int qvalid = min(a.part_cols, (SWAP ? a.M : a.N) - q0);
    if (nrows <= 0 || qvalid <= 0)
        return;
    if (SWAP) {
        for (int i = t; i < qvalid; i += kGemmThreadsC) {
            const uint16_t *row = a.R + (q0 + i) * a.ldr + p0 + r0;
            prefetch_l2(row);
            prefetch_l2(row + nrows - 1);
        }
    } else {
        for (int i = t; i < nrows; i += kGemmThreadsC) {
            const uint16_t *row = a.R + (p0 + r0 + i) * a.ldr + q0;
            for (int c = 0; c < qvalid; c += 64)
                prefetch_l2(row + c);
            prefetch_l2(row + qvalid - 1);
        }
    }
}

}  // namespace mxfp4
