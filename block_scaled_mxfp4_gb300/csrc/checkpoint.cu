// 8-bit checkpoints: bf16 rows to MXFP8 in two orientations, and the
// activation's backward pass that reads one.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "act.cuh"
#include "dense.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace mxfp4 {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ------------------------------------------------- the transposing quantiser --
//
//   by_row[r, c]: blocks of 32 columns, s = floor(log2 amax) - emax per block
//   by_col[c, r]: blocks of 32 rows, likewise
//   sums[c] = sum_r value[r, c], fp32
// of value = x, or of value = dh act'(z) with z = code 2^s read from its 8-bit
// checkpoint (and then also act(z), blocks of 32 rows).  Values stay fp32 from
// the load to the one rounding of each orientation.
//
// A warp's tile is 32 rows by 8 RPT columns: lane (g, c) holds rows g RPT ..
// + RPT - 1 of eight columns, so that a load instruction takes whole row segments, a
// block's largest magnitude is a maximum over registers and two (three)
// shuffles in either orientation, and both forms leave in full 32-byte sectors
// without a pass through shared memory.  A block of eight warps stacks four
// tiles along the rows, so that a column's codes fill a line, and walks down its strip of rows with
// the column sums in registers.

constexpr int kWarps = 8;
constexpr int kDown = 4;                         // warps of a block along the rows
constexpr int kAcross = kWarps / kDown;
constexpr int kTileRows = 32 * kDown;

__host__ __device__ constexpr int tile_cols(bool backward) { return (backward ? 4 : 8) * 8 * kAcross; }

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A block's scale from its largest magnitude: the scale code, and 2^-s.
__device__ __forceinline__ uint32_t block_scale8(float amax, int fmt, float &inv)
{
    const bool finite = amax <= 3.402823466e38f;         // not for infinities and NaN
    const int s = block_exponent8(finite ? amax : 0.0f, fmt == 0 ? 8 : 15);
    inv = exp2_neg(s);
    return finite ? static_cast<uint32_t>(s + 127) : 0xFFu;
}

// N (4 or 8) values -> N / 4 words of codes.
template <int N>
__device__ __forceinline__ void codes_of(const float (&v)[N], int fmt, uint32_t (&w)[N / 4])
{
    if (fmt == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            w[i] = f8x2<0>(v[4 * i], v[4 * i + 1]) | (f8x2<0>(v[4 * i + 2], v[4 * i + 3]) << 16);
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            w[i] = f8x2<1>(v[4 * i], v[4 * i + 1]) | (f8x2<1>(v[4 * i + 2], v[4 * i + 3]) << 16);
    }
}

// Two codes -> two floats (exact: every E4M3 and E5M2 value is an fp16 value).
__device__ __forceinline__ float2 values_of(uint32_t two, int fmt)
{
    uint32_t h;
    const uint16_t in = static_cast<uint16_t>(two);
    if (fmt == 0)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
    else
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(in));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// 2^(code - 127), NaN for 0xFF.
__device__ __forceinline__ float e8m0_value(uint32_t code)
{
    return code == 0u ? __uint_as_float(0x00400000u) : code == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float(code << 23);
}

// v[i][j]: row i of the lane's RPT rows, column j of its eight.  Blocks along the
// columns: 32 rows = RPT registers and the 32 / RPT lanes of one c.
template <int RPT>
__device__ __forceinline__ void store_by_col(const CodesOut &o, const float (&v)[RPT][8], int64_t row0, int64_t col0, int cols, int g)
{
    constexpr int CG = RPT;                              // lanes along the columns
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < RPT; i += 2)
            amax = max_abs3(amax, v[i][j], v[i + 1][j]);
#pragma unroll
        for (int d = CG; d < 32; d <<= 1)
            amax = max_nan(amax, __shfl_xor_sync(kFull, amax, d));
        float inv;
        const uint32_t code = block_scale8(amax, o.fmt, inv);
        float y[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            y[i] = v[i][j] * inv;
        uint32_t w[RPT / 4];
        codes_of<RPT>(y, o.fmt, w);
        if (col0 + j < cols) {
            uint8_t *q = o.q + (col0 + j) * o.ldq + row0 + g * RPT;
            if constexpr (RPT == 8)
                *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t *>(q) = w[0];
            if (g == 0)
                o.s[(col0 + j) * o.lds + row0 / 32] = static_cast<uint8_t>(code);
        }
    }
}

// Blocks along the rows: 32 columns = eight registers and four lanes.
template <int RPT>
__device__ __forceinline__ void store_by_row(const CodesOut &o, const float (&v)[RPT][8], int64_t row0, int64_t col0, int rows, int cols,
                                             int g)
{
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            amax = max_abs3(amax, v[i][j], v[i][j + 1]);
        amax = max_nan(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = max_nan(amax, __shfl_xor_sync(kFull, amax, 2));
        float inv;
        const uint32_t code = block_scale8(amax, o.fmt, inv);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = v[i][j] * inv;
        uint32_t w[2];
        codes_of<8>(y, o.fmt, w);
        const int64_t row = row0 + g * RPT + i;
        if (row < rows && col0 / 32 * 32 < cols) {       // whole blocks: columns past the last are zeros
            *reinterpret_cast<uint2 *>(o.q + row * o.ldq + col0) = make_uint2(w[0], w[1]);
            if ((col0 & 31) == 0)
                o.s[row * o.lds + col0 / 32] = static_cast<uint8_t>(code);
        }
    }
}

template <bool BACKWARD, Act ACT>
__global__ void __launch_bounds__(kWarps * 32, 2) checkpoint_kernel(const __grid_constant__ CheckpointArgs a)
{
    constexpr int RPT = BACKWARD ? 4 : 8;
    constexpr int CG = RPT;
    __shared__ float part[kDown][tile_cols(BACKWARD)];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int down = warp % kDown, across = warp / kDown;
    const int g = lane / CG, c = lane % CG;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * tile_cols(BACKWARD) + across * CG * 8 + c * 8;
    const int64_t tiles = (static_cast<int64_t>(a.rows) + kTileRows - 1) / kTileRows;
    const int64_t tile0 = tiles * blockIdx.y / gridDim.y, tile1 = tiles * (blockIdx.y + 1) / gridDim.y;
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        sum[j] = 0.0f;
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    for (int64_t t = tile0; t < tile1; ++t) {
        const int64_t row0 = t * kTileRows + down * 32;
        if (row0 >= a.rows)
            break;                                       // a warp's own: no barrier inside the loop
        uint4 raw[RPT];
        uint2 zq[RPT];
        uint32_t zs[RPT];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int64_t row = row0 + g * RPT + i;
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            zq[i] = make_uint2(0u, 0u);
            zs[i] = 127u;
            if (row < a.rows && col0 < a.cols) {
                const uint16_t *src = a.x + row * a.ldx + col0;
                if (col0 + 8 <= a.cols) {
                    raw[i] = __ldcs(reinterpret_cast<const uint4 *>(src));
                } else {
                    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < 7; ++j)
                        if (col0 + j < a.cols)
                            w[j / 2] |= static_cast<uint32_t>(src[j]) << (16 * (j & 1));
                    raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if constexpr (BACKWARD) {
                    zq[i] = __ldcs(reinterpret_cast<const uint2 *>(a.z + row * a.ldz + col0));
                    zs[i] = a.sz[row * a.ld_sz + col0 / 32];
                }
            }
        }
        float v[RPT][8];
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][2 * j] = bf16_lo(w[j]);
                v[i][2 * j + 1] = bf16_hi(w[j]);
            }
        }
        if constexpr (BACKWARD) {
            float h[RPT][8];
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float scale = e8m0_value(zs[i]);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const uint32_t w = j < 4 ? zq[i].x : zq[i].y;
                    const float2 z = values_of((w >> (8 * (j & 2))) & 0xFFFFu, a.fmt_z);
                    float slope;
                    // Columns past the last hold codes of no value: they count as zeros.
                    act_and_slope<ACT>(col0 + j < a.cols ? z.x * scale : 0.0f, h[i][j], slope);
                    v[i][j] *= slope;
                    act_and_slope<ACT>(col0 + j + 1 < a.cols ? z.y * scale : 0.0f, h[i][j + 1], slope);
                    v[i][j + 1] *= slope;
                }
            }
            if (a.act_by_col.q)
                store_by_col<RPT>(a.act_by_col, h, row0, col0, a.cols, g);
            if (a.dz) {
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const int64_t row = row0 + g * RPT + i;
                    if (row >= a.rows || col0 >= a.cols)
                        continue;
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 p = __floats2bfloat162_rn(v[i][2 * j], v[i][2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t *>(&p);
                    }
                    uint16_t *dst = a.dz + row * a.lddz + col0;
                    if (a.vec_dz && col0 + 8 <= a.cols) {
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (col0 + j < a.cols)
                                dst[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
                    }
                }
            }
        }
        if (a.sums) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < RPT; ++i)
                    sum[j] += v[i][j];
        }
        if (a.by_row.q)
            store_by_row<RPT>(a.by_row, v, row0, col0, a.rows, a.cols, g);
        if (a.by_col.q)
            store_by_col<RPT>(a.by_col, v, row0, col0, a.cols, g);
    }
    if (!a.sums)
        return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int d = CG; d < 32; d <<= 1)
            sum[j] += __shfl_xor_sync(kFull, sum[j], d);
        if (g == 0)
            part[down][across * CG * 8 + c * 8 + j] = sum[j];
    }
    __syncthreads();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * tile_cols(BACKWARD) + threadIdx.x;
    if (threadIdx.x < tile_cols(BACKWARD) && col < a.cols) {
        float s = 0.0f;
#pragma unroll
        for (int d = 0; d < kDown; ++d)
            s += part[d][threadIdx.x];
        (gridDim.y > 1 ? a.partials + static_cast<int64_t>(blockIdx.y) * a.cols : a.sums)[col] = s;
    }
}

// ------------------------------------------------------------ column sums --
//
// The second step of sums over rows: the strips' values, one row of na + nb of
// them per strip, to the arrays a and b (null: not wanted).  A block takes 32
// columns; its eight warps take every eighth strip, in order, and their sums
// are added in the warps' order.
__global__ void __launch_bounds__(256) sum_partials_kernel(float *a, int64_t na, float *b, int64_t nb, const float *partials, int strips)
{
    __shared__ float part[8][32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane, cols = na + nb;
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    float s = 0.0f;
    if (col < cols)
        for (int k = warp; k < strips; k += 8)
            s += partials[k * cols + col];
    part[warp][lane] = s;
    __syncthreads();
    float *out = col < na ? a : b;
    if (warp == 0 && col < cols && out) {
#pragma unroll
        for (int k = 1; k < 8; ++k)
            s += part[k][lane];
        out[col < na ? col : col - na] = s;
    }
}

}  // namespace

int checkpoint_strips(int rows, int cols, bool backward)
{
    const int64_t across = (static_cast<int64_t>(cols) + tile_cols(backward) - 1) / tile_cols(backward);
    const int64_t tiles = (static_cast<int64_t>(rows) + kTileRows - 1) / kTileRows;
    // Blocks for four rounds of two per SM of a GB300's 152.
    int64_t strips = (4 * 2 * 152 + across - 1) / across;
    strips = strips < tiles ? strips : tiles;
    return static_cast<int>(strips < 1 ? 1 : strips > 65535 ? 65535 : strips);
}

cudaError_t launch_sum_partials(float *a, int64_t na, float *b, int64_t nb, const float *partials, int strips, cudaStream_t stream)
{
    return launch_dependent(sum_partials_kernel, dim3(static_cast<unsigned>((na + nb + 31) / 32)), dim3(256), 0, stream, a, na, b, nb,
                            partials, strips);
}

cudaError_t launch_checkpoint(const CheckpointArgs &a, bool backward, cudaStream_t stream)
{
    const int across = tile_cols(backward);
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.cols) + across - 1) / across), static_cast<unsigned>(a.strips));
    cudaError_t e;
    if (!backward)
        e = launch_dependent(checkpoint_kernel<false, Act::kNone>, grid, dim3(kWarps * 32), 0, stream, a);
    else
        e = with_act(a.act, [&](auto tag) {
            return launch_dependent(checkpoint_kernel<true, decltype(tag)::value>, grid, dim3(kWarps * 32), 0, stream, a);
        });
    if (e == cudaSuccess && a.sums && a.strips > 1)
        e = launch_sum_partials(a.sums, a.cols, nullptr, 0, a.partials, a.strips, stream);
    return e;
}

}  // namespace mxfp4
