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
// A block of 256 threads takes tiles of 128 rows, one below the other, by 128
// columns (64 in the backward pass), copied to shared memory asynchronously while
// the tile before is worked on.  A lane then takes 32 values of a row, and 32 of a
// column: a block of either orientation is one lane's, and nothing needs a
// shuffle.  Lanes are dealt so that a warp's accesses fall into whole
// lines (128 bytes of codes are four lanes') and on different banks.  In the
// backward pass the computed values go through shared memory as fp32, act(z) and
// dz in turn.
//
// Why not straight from global memory, a row or column per lane: each such
// access touches 32 lines, and the L1's tag stage, one line a cycle, was 80 %
// busy at half of HBM's rate.

constexpr int kThreads = 256;
constexpr int kTileRows = 128;

template <bool BACKWARD>
struct Tile {
    static constexpr int kCols = BACKWARD ? 64 : 128;
    static constexpr int kPitch = 2 * kCols + 16;        // bytes between x's rows: 4 words past a multiple of 32
    static constexpr int kSkew = 32;                     // more before each 32 rows: lanes 32 rows apart meet no bank twice
    static constexpr int kXBytes = kTileRows * kPitch + 4 * kSkew;
    static constexpr int kZPitch = 80;
    static constexpr int kZBytes = BACKWARD ? kTileRows * kZPitch : 0;
    static constexpr int kStage = kXBytes + kZBytes;
    static constexpr int kFPitch = 68;                   // floats between rows of computed values
    static constexpr int kFBytes = BACKWARD ? (kTileRows * kFPitch + 32) * 4 : 0;
    static constexpr int kBytes = 2 * kStage + kFBytes;
    static constexpr int kUnits = kTileRows * kCols / 32 / kThreads;   // row blocks of a thread

    static __device__ __forceinline__ int x_at(int row) { return row * kPitch + row / 32 * kSkew; }
    static __device__ __forceinline__ int f_at(int row) { return row * kFPitch + row / 32 * 8; }
    // Row and 32-column block of a thread's unit k: eight neighbouring rows to eight neighbouring lanes.
    static __device__ __forceinline__ void unit(int warp, int lane, int k, int &row, int &b)
    {
        if (BACKWARD) {
            row = warp * 16 + (lane & 7) + 8 * (lane >> 4);
            b = (lane >> 3) & 1;
        } else {
            row = (k * 8 + warp) * 8 + (lane & 7);
            b = lane >> 3;
        }
    }
};

// 16 bytes, the first `have` of them from src and the rest zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int have)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have) : "memory");
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

// Start the copies of one tile; what lies past the last row or column becomes zeros.
template <bool BACKWARD>
__device__ __forceinline__ void load_tile(const CheckpointArgs &a, uint32_t stage, int64_t row0, int64_t col0, int t)
{
    using T = Tile<BACKWARD>;
    constexpr int kChunks = T::kCols / 8;                // 16-byte pieces of a row
#pragma unroll
    for (int i = 0; i < kTileRows * kChunks / kThreads; ++i) {
        const int at = i * kThreads + t, r = at / kChunks, c = at % kChunks * 8;
        const int64_t left = row0 + r < a.rows ? a.cols - (col0 + c) : 0;
        const int have = left >= 8 ? 16 : left > 0 ? static_cast<int>(left) * 2 : 0;
        copy16(stage + T::x_at(r) + 2 * c, have ? a.x + (row0 + r) * a.ldx + col0 + c : a.x, have);
    }
    if constexpr (BACKWARD) {
        constexpr int kZChunks = T::kCols / 16;
#pragma unroll
        for (int i = 0; i < kTileRows * kZChunks / kThreads; ++i) {
            const int at = i * kThreads + t, r = at / kZChunks, c = at % kZChunks * 16;
            const int64_t left = row0 + r < a.rows ? a.cols - (col0 + c) : 0;
            const int have = left >= 16 ? 16 : left > 0 ? static_cast<int>(left) : 0;
            copy16(stage + T::kXBytes + r * T::kZPitch + c, have ? a.z + (row0 + r) * a.ldz + col0 + c : a.z, have);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// act(z) to h, v *= act'(z).
template <Act ACT, int FMT>
__device__ __forceinline__ void back_row(const uint32_t (&zw)[8], float scale, float *h, float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const F2 z = values_of<FMT>((zw[i / 4] >> (8 * j)) & 0xFFFFu) * f2(scale);
            F2 act, slope;
            act_and_slope2<ACT>(z, act, slope);
            const float2 p = parts(f2(v[i + j], v[i + j + 1]) * slope), q = parts(act);
            v[i + j] = p.x;
            v[i + j + 1] = p.y;
            x[j] = q.x;
            x[j + 1] = q.y;
        }
        *reinterpret_cast<float4 *>(h + i) = make_float4(x[0], x[1], x[2], x[3]);
    }
}

// dz of one row block as bf16.
__device__ __forceinline__ void put_dz(const CheckpointArgs &a, int64_t row, int64_t col0, const float (&v)[32])
{
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

// One column block's codes and scale.
__device__ __forceinline__ void put_col(const CodesOut &o, bool wide, int64_t col, int64_t row0, const float (&v)[32])
{
    const uint32_t code = put_block(v, o.fmt, o.q + col * o.ldq + row0, wide, true);
    o.s[col * o.lds + row0 / 32] = static_cast<uint8_t>(code);
}

template <bool BACKWARD, Act ACT>
__global__ void __launch_bounds__(kThreads, BACKWARD ? 2 : 3) checkpoint_kernel(const __grid_constant__ CheckpointArgs a)
{
    using T = Tile<BACKWARD>;
    extern __shared__ __align__(128) uint8_t smem[];
    float *computed = reinterpret_cast<float *>(smem + 2 * T::kStage);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t strip = blockIdx.x / a.col_blocks;
    const int64_t col_first = blockIdx.x % a.col_blocks * T::kCols;
    const int64_t row_first = strip * a.steps * kTileRows;
    const int64_t left = (a.rows - row_first + kTileRows - 1) / kTileRows;
    const int steps = static_cast<int>(left < a.steps ? left : a.steps);
    // The thread's column block: eight neighbouring (pairs of) columns to eight lanes, the four row
    // blocks of a column to lanes eight apart.
    const int rb = lane >> 3, cl = warp * 8 + (lane & 7);
    constexpr int kSums = BACKWARD ? 1 : 2;
    float sum[kSums];
#pragma unroll
    for (int k = 0; k < kSums; ++k)
        sum[k] = 0.0f;
    pdl_wait_prerequisites();
    if (threadIdx.x == 0)
        pdl_launch_dependents();
    load_tile<BACKWARD>(a, smem_addr(smem), row_first, col_first, threadIdx.x);
    for (int step = 0; step < steps; ++step) {
        const int64_t row0 = row_first + static_cast<int64_t>(step) * kTileRows;
        const uint8_t *stage = smem + (step & 1) * T::kStage;
        uint32_t zs[T::kUnits];
        if constexpr (BACKWARD) {
#pragma unroll
            for (int k = 0; k < T::kUnits; ++k) {
                int r, b;
                T::unit(warp, lane, k, r, b);
                const int64_t row = row0 + r, col0 = col_first + 32 * b;
                zs[k] = row < a.rows && col0 < a.cols ? a.sz[row * a.ld_sz + col0 / 32] : 127u;
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        // Every thread is past the tile before, whose memory the next one takes.
        if (step + 1 < steps)
            load_tile<BACKWARD>(a, smem_addr(smem + ((step + 1) & 1) * T::kStage), row0 + kTileRows, col_first, threadIdx.x);
        if (BACKWARD || a.by_row.q) {
#pragma unroll
            for (int k = 0; k < T::kUnits; ++k) {
                int r, b;
                T::unit(warp, lane, k, r, b);
                const int64_t row = row0 + r, col0 = col_first + 32 * b;
                const bool have = row < a.rows && col0 < a.cols;
                float v[32];
                const uint4 *x = reinterpret_cast<const uint4 *>(stage + T::x_at(r) + 64 * b);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 q = x[i];
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[8 * i + 2 * j] = bf16_lo(w[j]);
                        v[8 * i + 2 * j + 1] = bf16_hi(w[j]);
                    }
                }
                if constexpr (BACKWARD) {
                    float *mine = computed + T::f_at(r) + 32 * b;
                    const uint4 *z = reinterpret_cast<const uint4 *>(stage + T::kXBytes + r * T::kZPitch + 32 * b);
                    const uint4 lo = z[0], hi = z[1];
                    const uint32_t zw[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    if (a.fmt_z == 0)
                        back_row<ACT, 0>(zw, e8m0_value(zs[k]), mine, v);
                    else
                        back_row<ACT, 1>(zw, e8m0_value(zs[k]), mine, v);
                    const int64_t col = col_first + cl, block0 = row0 + 32 * rb;
                    const bool have_col = col < a.cols && block0 < a.rows;
                    float u[32];
                    if (a.act_by_col.q) {
                        __syncthreads();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            u[i] = computed[T::f_at(32 * rb) + i * T::kFPitch + cl];
                        if (have_col)
                            put_col(a.act_by_col, a.wide_ht, col, block0, u);
                    }
                    __syncthreads();
                    if (a.by_col.q || a.sums) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(mine + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                    if (a.dz && have)
                        put_dz(a, row, col0, v);
                    if (a.by_row.q && have) {
                        const uint32_t code = put_block(v, a.by_row.fmt, a.by_row.q + row * a.by_row.ldq + col0, a.wide_q, true);
                        a.by_row.s[row * a.by_row.lds + col0 / 32] = static_cast<uint8_t>(code);
                    }
                    if (a.by_col.q || a.sums) {
                        __syncthreads();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            u[i] = computed[T::f_at(32 * rb) + i * T::kFPitch + cl];
                        if (a.sums) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                sum[0] += u[i];
                        }
                        if (a.by_col.q && have_col)
                            put_col(a.by_col, a.wide_qt, col, block0, u);
                    }
                } else if (have) {
                    const uint32_t code = put_block(v, a.by_row.fmt, a.by_row.q + row * a.by_row.ldq + col0, a.wide_q, true);
                    a.by_row.s[row * a.by_row.lds + col0 / 32] = static_cast<uint8_t>(code);
                }
            }
        }
        if constexpr (!BACKWARD) {
            if (a.by_col.q || a.sums) {
                uint32_t w[32];
                const uint8_t *x = stage + T::x_at(32 * rb) + 4 * cl;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    w[i] = *reinterpret_cast<const uint32_t *>(x + i * T::kPitch);
                const int64_t block0 = row0 + 32 * rb;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int64_t col = col_first + 2 * cl + k;
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = k ? bf16_hi(w[i]) : bf16_lo(w[i]);
                    if (a.sums) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            sum[k] += v[i];
                    }
                    if (a.by_col.q && col < a.cols && block0 < a.rows)
                        put_col(a.by_col, a.wide_qt, col, block0, v);
                }
            }
        }
    }
    if (!a.sums)
        return;
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 8);
        sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 16);
        const int64_t col = col_first + kSums * cl + k;
        if (rb == 0 && col < a.cols)
            (a.strips > 1 ? a.partials + strip * a.cols : a.sums)[col] = sum[k];
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

int64_t checkpoint_strips(int rows, int cols, bool backward, int *steps)
{
    const int wide = backward ? Tile<true>::kCols : Tile<false>::kCols;
    const int64_t down = (static_cast<int64_t>(rows) + kTileRows - 1) / kTileRows;
    const int64_t tiles = down * ((static_cast<int64_t>(cols) + wide - 1) / wide);
    // Resident blocks on a GB300's 152 SMs; tiles below one another in a block as long as that
    // leaves several rounds of blocks.
    const int64_t resident = 152 * (backward ? 2 : 3);
    *steps = tiles >= 16 * resident ? 4 : tiles >= 4 * resident ? 2 : 1;
    return (down + *steps - 1) / *steps;
}

cudaError_t launch_sum_partials(float *a, int64_t na, float *b, int64_t nb, const float *partials, int strips, cudaStream_t stream)
{
    return launch_dependent(sum_partials_kernel, dim3(static_cast<unsigned>((na + nb + 31) / 32)), dim3(1024), 0, stream, a, na, b, nb,
                            partials, strips);
}

template <bool BACKWARD, Act ACT>
static cudaError_t start_checkpoint(const CheckpointArgs &a, cudaStream_t stream)
{
    constexpr int kBytes = Tile<BACKWARD>::kBytes;
    const cudaError_t e = opt_in<checkpoint_kernel<BACKWARD, ACT>>(kBytes);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(checkpoint_kernel<BACKWARD, ACT>, dim3(static_cast<unsigned>(a.strips * a.col_blocks)), dim3(kThreads), kBytes,
                            stream, a);
}

cudaError_t launch_checkpoint(CheckpointArgs &a, bool backward, cudaStream_t stream)
{
    const int wide_cols = backward ? Tile<true>::kCols : Tile<false>::kCols;
    a.col_blocks = (static_cast<int64_t>(a.cols) + wide_cols - 1) / wide_cols;
    auto wide = [](const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 32 == 0 && bytes % 32 == 0; };
    a.wide_q = wide(a.by_row.q, a.by_row.ldq);
    a.wide_qt = wide(a.by_col.q, a.by_col.ldq);
    a.wide_ht = wide(a.act_by_col.q, a.act_by_col.ldq);
    cudaError_t e = backward ? with_act(a.act, [&](auto tag) { return start_checkpoint<true, decltype(tag)::value>(a, stream); })
                             : start_checkpoint<false, Act::kNone>(a, stream);
    if (e == cudaSuccess && a.sums && a.strips > 1)
        e = launch_sum_partials(a.sums, a.cols, nullptr, 0, a.partials, static_cast<int>(a.strips), stream);
    return e;
}

}  // namespace mxfp4
