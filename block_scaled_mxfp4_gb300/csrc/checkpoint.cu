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

// ------------------------------------------------- the transposing quantiser --
//
//   by_row[r, c]: blocks of 32 columns, s = floor(log2 amax) - emax per block
//   by_col[c, r]: blocks of 32 rows, likewise
//   sums[c] = sum_r value[r, c], fp32
// of value = x, or of value = dh act'(z) with z = code 2^s read from its 8-bit
// checkpoint (and then also act(z), blocks of 32 rows).  Values stay fp32 from
// the load to the one rounding of each orientation.
//
// A warp takes 32 x 32 values at a time, a lane one row of them: the block along
// the row is then one lane's, and its input and codes are whole 32-byte sectors.
// The values go through the warp's piece of shared memory, and a lane takes one
// column: that block is one lane's too, no orientation needs a shuffle, and
// the codes leave as sectors again.  A warp does kAcross such tiles side by side
// and `steps` below one another, a block kDown warps on top of each other and two
// beside.

constexpr int kWarps = 8;
constexpr int kDown = 4;                         // warps of a block along the rows
constexpr int kBeside = kWarps / kDown;
constexpr int kAcross = 2;                       // tiles of a warp along the columns
constexpr int kBlockCols = 32 * kAcross * kBeside;
constexpr int kPitch = 36;                       // floats between rows in shared memory: no bank conflict either way

__device__ __forceinline__ void ld_sector(const void *p, uint32_t *w)
{
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

__device__ __forceinline__ void st_sector(void *p, const uint32_t (&w)[8], bool wide)
{
    if (wide) {
        st_global_v8(p, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// One block of a lane: its codes to q; the scale code.
__device__ __forceinline__ uint32_t put_block(const float (&v)[32], int fmt, uint8_t *q, bool wide, bool store)
{
    uint32_t w[8];
    const uint32_t code = fmt == 0 ? quantize_block<QuantFmt::kE4M3>(v, w) : quantize_block<QuantFmt::kE5M2>(v, w);
    if (store)
        st_sector(q, w, wide);
    return code;
}

// Two codes -> two floats (exact: every E4M3 and E5M2 value is an fp16 value).
template <int FMT>
__device__ __forceinline__ F2 values_of(uint32_t two)
{
    uint32_t h;
    const uint16_t in = static_cast<uint16_t>(two);
    if constexpr (FMT == 0)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
    else
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(in));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return f2(f.x, f.y);
}

// 2^(code - 127), NaN for 0xFF.
__device__ __forceinline__ float e8m0_value(uint32_t code)
{
    return code == 0u ? __uint_as_float(0x00400000u) : code == 0xFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float(code << 23);
}

// 32 bf16 values of a row from column col0 on, zeros past the last one.
__device__ __forceinline__ void load_row(const CheckpointArgs &a, int64_t row, int64_t col0, uint32_t (&w)[16])
{
    const uint16_t *src = a.x + row * a.ldx + col0;
    if (col0 + 32 <= a.cols) {
        if (a.wide_x) {
            ld_sector(src, w);
            ld_sector(src + 16, w + 8);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t lo = col0 + 2 * i < a.cols ? src[2 * i] : 0u, hi = col0 + 2 * i + 1 < a.cols ? src[2 * i + 1] : 0u;
            w[i] = lo | hi << 16;
        }
    }
}

// act(z) to the lane's row of the tile, v *= act'(z).
template <Act ACT, int FMT>
__device__ __forceinline__ void back_row(const uint32_t (&zw)[8], float scale, int count, float *tile, float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        float h[4];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            F2 z = values_of<FMT>((zw[i / 4] >> (8 * j)) & 0xFFFFu) * f2(scale);
            if (count < 32) {                            // codes past the last column count as zeros
                const float2 p = parts(z);
                z = f2(i + j < count ? p.x : 0.0f, i + j + 1 < count ? p.y : 0.0f);
            }
            F2 act, slope;
            act_and_slope2<ACT>(z, act, slope);
            const float2 p = parts(f2(v[i + j], v[i + j + 1]) * slope), q = parts(act);
            v[i + j] = p.x;
            v[i + j + 1] = p.y;
            h[j] = q.x;
            h[j + 1] = q.y;
        }
        *reinterpret_cast<float4 *>(tile + i) = make_float4(h[0], h[1], h[2], h[3]);
    }
}

// The lane's column of the tile.
__device__ __forceinline__ void read_col(const float *tile, int lane, float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = tile[i * kPitch + lane];
}

template <bool BACKWARD, Act ACT>
__global__ void __launch_bounds__(kWarps * 32, BACKWARD ? 2 : 3) checkpoint_kernel(const __grid_constant__ CheckpointArgs a)
{
    __shared__ __align__(16) float tiles[kWarps][32 * kPitch];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    float *tile = tiles[warp];
    const int64_t strip = blockIdx.x / a.col_blocks, col_block = blockIdx.x % a.col_blocks;
    const int64_t row_first = (strip * kDown + warp % kDown) * 32 * a.steps;
    const int64_t col_first = col_block * kBlockCols + warp / kDown * 32 * kAcross;
    float sum[kAcross];
#pragma unroll
    for (int k = 0; k < kAcross; ++k)
        sum[k] = 0.0f;
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    for (int step = 0; step < a.steps; ++step) {
        const int64_t row0 = row_first + 32 * step, row = row0 + lane;
        if (row0 >= a.rows)
            break;
        const bool have = row < a.rows;
#pragma unroll
        for (int k = 0; k < kAcross; ++k) {
            const int64_t col0 = col_first + 32 * k, col = col0 + lane;
            if (col0 >= a.cols)
                break;
            float v[32];
            {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[i] = 0u;
                uint32_t zw[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                uint32_t zs = 127u;
                if (have) {
                    load_row(a, row, col0, w);
                    if constexpr (BACKWARD) {
                        const uint8_t *z = a.z + row * a.ldz + col0;
                        if (a.wide_z) {
                            ld_sector(z, zw);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(z) + i);
                                zw[4 * i] = q.x;
                                zw[4 * i + 1] = q.y;
                                zw[4 * i + 2] = q.z;
                                zw[4 * i + 3] = q.w;
                            }
                        }
                        zs = a.sz[row * a.ld_sz + col0 / 32];
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    v[2 * i] = bf16_lo(w[i]);
                    v[2 * i + 1] = bf16_hi(w[i]);
                }
                if constexpr (BACKWARD) {
                    const int count = static_cast<int>(col0 + 32 <= a.cols ? 32 : a.cols - col0);
                    if (a.fmt_z == 0)
                        back_row<ACT, 0>(zw, e8m0_value(zs), count, tile + lane * kPitch, v);
                    else
                        back_row<ACT, 1>(zw, e8m0_value(zs), count, tile + lane * kPitch, v);
                }
            }
            if constexpr (BACKWARD) {
                __syncwarp();
                if (a.act_by_col.q) {
                    float h[32];
                    read_col(tile, lane, h);
                    const uint32_t code = put_block(h, a.act_by_col.fmt, a.act_by_col.q + col * a.act_by_col.ldq + row0, a.wide_ht, col < a.cols);
                    if (col < a.cols)
                        a.act_by_col.s[col * a.act_by_col.lds + row0 / 32] = static_cast<uint8_t>(code);
                }
                __syncwarp();
                if (a.dz && have) {
                    uint16_t *dst = a.dz + row * a.lddz + col0;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __nv_bfloat162 p = __floats2bfloat162_rn(v[i + 2 * j], v[i + 2 * j + 1]);
                            w[j] = *reinterpret_cast<const uint32_t *>(&p);
                        }
                        if (a.vec_dz && col0 + i + 8 <= a.cols) {
                            *reinterpret_cast<uint4 *>(dst + i) = make_uint4(w[0], w[1], w[2], w[3]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (col0 + i + j < a.cols)
                                    dst[i + j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
                        }
                    }
                }
            }
            if (a.by_col.q || a.sums) {
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<float4 *>(tile + lane * kPitch + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
            if (a.by_row.q) {
                const uint32_t code = put_block(v, a.by_row.fmt, a.by_row.q + row * a.by_row.ldq + col0, a.wide_q, have);
                if (have)
                    a.by_row.s[row * a.by_row.lds + col0 / 32] = static_cast<uint8_t>(code);
            }
            if (a.by_col.q || a.sums) {
                __syncwarp();
                read_col(tile, lane, v);
                if (a.sums) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        sum[k] += v[i];
                }
                if (a.by_col.q) {
                    const uint32_t code = put_block(v, a.by_col.fmt, a.by_col.q + col * a.by_col.ldq + row0, a.wide_qt, col < a.cols);
                    if (col < a.cols)
                        a.by_col.s[col * a.by_col.lds + row0 / 32] = static_cast<uint8_t>(code);
                }
                __syncwarp();
            }
        }
    }
    if (!a.sums)
        return;
#pragma unroll
    for (int k = 0; k < kAcross; ++k)
        tile[32 * k + lane] = sum[k];
    __syncthreads();
    const int64_t col = col_block * kBlockCols + threadIdx.x;
    if (threadIdx.x < kBlockCols && col < a.cols) {
        const int beside = threadIdx.x / (32 * kAcross), at = threadIdx.x % (32 * kAcross);
        float s = 0.0f;
#pragma unroll
        for (int d = 0; d < kDown; ++d)
            s += tiles[beside * kDown + d][at];
        (a.strips > 1 ? a.partials + strip * a.cols : a.sums)[col] = s;
    }
}

// ------------------------------------------------------------ column sums --
//
// The second step of sums over rows: the strips' values, one row of na + nb of
// them per strip, to the arrays a and b (null: not wanted).  A block takes 32
// columns; its 32 warps take every 32nd strip, in order, and their sums are added
// in the warps' order.
__global__ void __launch_bounds__(1024) sum_partials_kernel(float *a, int64_t na, float *b, int64_t nb, const float *partials, int strips)
{
    __shared__ float part[32][33];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane, cols = na + nb;
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    float s = 0.0f;
    if (col < cols)
        for (int k = warp; k < strips; k += 32)
            s += partials[k * cols + col];
    part[warp][lane] = s;
    __syncthreads();
    float *out = col < na ? a : b;
    if (warp == 0 && col < cols && out) {
#pragma unroll
        for (int k = 1; k < 32; ++k)
            s += part[k][lane];
        out[col < na ? col : col - na] = s;
    }
}

}  // namespace

int64_t checkpoint_strips(int rows, int cols, int *steps)
{
    const int64_t across = (static_cast<int64_t>(cols) + kBlockCols - 1) / kBlockCols;
    auto strips = [&](int n) { return (static_cast<int64_t>(rows) + 32 * kDown * n - 1) / (32 * kDown * n); };
    // Four tiles down a warp where that still fills a GB300's 152 SMs three times, else one.
    *steps = strips(4) * across >= 3 * 152 ? 4 : 1;
    return strips(*steps);
}

cudaError_t launch_sum_partials(float *a, int64_t na, float *b, int64_t nb, const float *partials, int strips, cudaStream_t stream)
{
    return launch_dependent(sum_partials_kernel, dim3(static_cast<unsigned>((na + nb + 31) / 32)), dim3(1024), 0, stream, a, na, b, nb,
                            partials, strips);
}

cudaError_t launch_checkpoint(CheckpointArgs &a, bool backward, cudaStream_t stream)
{
    a.col_blocks = (static_cast<int64_t>(a.cols) + kBlockCols - 1) / kBlockCols;
    auto wide = [](const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 32 == 0 && bytes % 32 == 0; };
    a.wide_x = wide(a.x, 2 * a.ldx);
    a.wide_z = wide(a.z, a.ldz);
    a.wide_q = wide(a.by_row.q, a.by_row.ldq);
    a.wide_qt = wide(a.by_col.q, a.by_col.ldq);
    a.wide_ht = wide(a.act_by_col.q, a.act_by_col.ldq);
    const dim3 grid(static_cast<unsigned>(a.strips * a.col_blocks));
    cudaError_t e;
    if (!backward)
        e = launch_dependent(checkpoint_kernel<false, Act::kNone>, grid, dim3(kWarps * 32), 0, stream, a);
    else
        e = with_act(a.act, [&](auto tag) {
            return launch_dependent(checkpoint_kernel<true, decltype(tag)::value>, grid, dim3(kWarps * 32), 0, stream, a);
        });
    if (e == cudaSuccess && a.sums && a.strips > 1)
        e = launch_sum_partials(a.sums, a.cols, nullptr, 0, a.partials, static_cast<int>(a.strips), stream);
    return e;
}

}  // namespace mxfp4
