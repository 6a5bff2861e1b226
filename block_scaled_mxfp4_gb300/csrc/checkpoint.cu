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
// columns (64 in the backward pass), copied to shared memory by TMA while the tile
// before is worked on.  A lane then takes 32 values of a row, and 32 of a
// column: a block of either orientation is one lane's, and nothing needs a
// shuffle.  Lanes are dealt so that a warp's stores fall into whole lines (128
// bytes of codes are four lanes') and its shared-memory reads on different banks:
// TMA's swizzle moves 16-byte pieces by the row, and lanes 32 rows apart read
// their column's rows in orders of their own (put_col).  In the backward pass the
// computed values go through shared memory as fp32.
//
// Why not straight from global memory, a row or column per lane: each such
// access touches 32 lines, and the L1's tag stage, one line a cycle, was 80 %
// busy at half of HBM's rate.  Copies by cp.async instead of TMA took as many of
// its cycles as all stores together.

constexpr int kThreads = 256;
constexpr int kTileRows = 128;

template <bool BACKWARD>
struct Tile {
    static constexpr int kCols = BACKWARD ? 64 : 128;
    static constexpr int kBox = kTileRows * 128;         // 64 columns of x: 128-byte rows, 128-byte swizzle
    static constexpr int kXBytes = kCols / 64 * kBox;
    static constexpr int kZBytes = BACKWARD ? kTileRows * 64 : 0;   // 64-byte rows, 64-byte swizzle
    static constexpr int kStage = kXBytes + kZBytes;
    // The backward pass has one stage: the row pass empties it, and it fills again under the column passes.
    static constexpr int kStages = BACKWARD ? 1 : 2;
    static constexpr int kFPitch = 68;                   // floats between rows of computed values
    static constexpr int kF = BACKWARD ? kTileRows * kFPitch + 32 : 0;     // floats of act(z), and of dz
    static constexpr int kBytes = kStages * kStage + 2 * kF * 4 + 1024;    // with the alignment that the swizzle asks for
    static constexpr int kUnits = kTileRows * kCols / 32 / kThreads;   // row blocks of a thread

    // Eight floats more before each 32 rows: lanes 32 rows apart meet no bank twice.
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

__device__ int g_status = 0;                     // bounded waits that ran out

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
__device__ __forceinline__ uint32_t put_block(const float (&v)[32], int fmt, uint8_t *q, bool wide)
{
    uint32_t w[8];
    const uint32_t code = fmt == 0 ? quantize_block_pairs<QuantFmt::kE4M3>(v, w) : quantize_block_pairs<QuantFmt::kE5M2>(v, w);
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

// Start the copies of one tile; what lies past the last row or column arrives as zeros.
template <bool BACKWARD>
__device__ __forceinline__ void load_tile(const CUtensorMap *x, const CUtensorMap *z, uint8_t *stage, uint64_t *full, int64_t row0, int64_t col0)
{
    using T = Tile<BACKWARD>;
    const uint64_t policy = l2_policy_evict_first();
    mbar_arrive_expect_tx(full, T::kStage);
#pragma unroll
    for (int k = 0; k < T::kCols / 64; ++k)
        tma_load_2d(stage + k * T::kBox, x, full, static_cast<int>(col0) + 64 * k, static_cast<int>(row0), policy);
    if constexpr (BACKWARD)
        tma_load_2d(stage + T::kXBytes, z, full, static_cast<int>(col0), static_cast<int>(row0), policy);
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

// One column block's codes and scale.  v[i] is row i ^ ROWS of the block (0, 2, 4 or 6): the codes
// change places accordingly, in units of two.
template <bool PERMUTED>
__device__ __forceinline__ void put_col(const CodesOut &o, bool wide, int64_t col, int64_t row0, int rows, const float (&v)[32])
{
    uint32_t w[8];
    const uint32_t code = o.fmt == 0 ? quantize_block_pairs<QuantFmt::kE4M3>(v, w) : quantize_block_pairs<QuantFmt::kE5M2>(v, w);
    if constexpr (PERMUTED) {
        const uint32_t order = rows & 2 ? 0x1032u : 0x3210u;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint32_t lo = __byte_perm(w[i], 0u, order), hi = __byte_perm(w[i + 1], 0u, order);
            w[i] = rows & 4 ? hi : lo;
            w[i + 1] = rows & 4 ? lo : hi;
        }
    }
    st_sector(o.q + col * o.ldq + row0, w, wide);
    o.s[col * o.lds + row0 / 32] = static_cast<uint8_t>(code);
}

template <bool BACKWARD, Act ACT>
__global__ void __launch_bounds__(kThreads, BACKWARD ? 2 : 3)
    checkpoint_kernel(const __grid_constant__ CheckpointArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mz)
{
    using T = Tile<BACKWARD>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[2];
    __shared__ int abort_flag;
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
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
    F2 sum = f2(0.0f);                                   // of two columns, or of one column's rows two by two
    if (threadIdx.x == 0) {
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait_prerequisites();
    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        load_tile<BACKWARD>(&mx, &mz, smem, &full[0], row_first, col_first);
    }
    // The scale of the thread's row block of z, in the tile that starts at row0.
    auto z_scale = [&](int64_t row0) -> uint32_t {
        int r, b;
        T::unit(warp, lane, 0, r, b);
        const int64_t row = row0 + r, col0 = col_first + 32 * b;
        return row < a.rows && col0 < a.cols ? a.sz[row * a.ld_sz + col0 / 32] : 127u;
    };
    uint32_t zs = 127u;
    if constexpr (BACKWARD)
        zs = z_scale(row_first);
    for (int step = 0; step < steps; ++step) {
        const int64_t row0 = row_first + static_cast<int64_t>(step) * kTileRows;
        const int at = step % T::kStages;
        const uint32_t phase = step / T::kStages & 1;
        const uint8_t *stage = smem + at * T::kStage;
        const bool ok = mbar_wait(&full[at], phase, &abort_flag, a.wait_limit, &g_status);
        if (__syncthreads_or(!ok)) {
            if (threadIdx.x == 0)
                mbar_wait_drain(&full[at], phase, a.wait_limit);     // its copies land before the block leaves
            return;
        }
        // Every thread is past the tile before.
        if (!BACKWARD && step + 1 < steps && threadIdx.x == 0)
            load_tile<BACKWARD>(&mx, &mz, smem + (at ^ 1) * T::kStage, &full[at ^ 1], row0 + kTileRows, col_first);
        if (BACKWARD || a.by_row.q) {
#pragma unroll
            for (int k = 0; k < T::kUnits; ++k) {
                int r, b;
                T::unit(warp, lane, k, r, b);
                const int64_t row = row0 + r, col0 = col_first + 32 * b;
                const bool have = row < a.rows && col0 < a.cols;
                float v[32];
                const uint8_t *x = stage + (b >> 1) * T::kBox + r * 128;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(x + (((b & 1) * 4 + i) ^ (r & 7)) * 16);
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[8 * i + 2 * j] = bf16_lo(w[j]);
                        v[8 * i + 2 * j + 1] = bf16_hi(w[j]);
                    }
                }
                if constexpr (BACKWARD) {
                    float *h = reinterpret_cast<float *>(smem + T::kStage) + T::f_at(r) + 32 * b;
                    const uint8_t *z = stage + T::kXBytes + r * 64;
                    const uint4 lo = *reinterpret_cast<const uint4 *>(z + ((2 * b) ^ ((r >> 1) & 3)) * 16);
                    const uint4 hi = *reinterpret_cast<const uint4 *>(z + ((2 * b + 1) ^ ((r >> 1) & 3)) * 16);
                    const uint32_t zw[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    if (a.fmt_z == 0)
                        back_row<ACT, 0>(zw, e8m0_value(zs), h, v);
                    else
                        back_row<ACT, 1>(zw, e8m0_value(zs), h, v);
                    if (step + 1 < steps)
                        zs = z_scale(row0 + kTileRows);
                    if (a.by_col.q || a.sums) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4 *>(h + T::kF + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                    if (a.dz && have)
                        put_dz(a, row, col0, v);
                }
                if (a.by_row.q && have) {
                    const uint32_t code = put_block(v, a.by_row.fmt, a.by_row.q + row * a.by_row.ldq + col0, a.wide_q);
                    a.by_row.s[row * a.by_row.lds + col0 / 32] = static_cast<uint8_t>(code);
                }
            }
        }
        const int64_t block0 = row0 + 32 * rb;
        if constexpr (BACKWARD) {
            __syncthreads();
            if (step + 1 < steps && threadIdx.x == 0)
                load_tile<BACKWARD>(&mx, &mz, smem, &full[0], row0 + kTileRows, col_first);
            const int64_t col = col_first + cl;
            const bool have = col < a.cols && block0 < a.rows;
            const float *h = reinterpret_cast<const float *>(smem + T::kStage) + T::f_at(32 * rb) + cl;
            float u[32];
            if (a.act_by_col.q) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    u[i] = h[i * T::kFPitch];
                if (have)
                    put_col<false>(a.act_by_col, a.wide_ht, col, block0, 0, u);
            }
            if (a.by_col.q || a.sums) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    u[i] = h[T::kF + i * T::kFPitch];
                if (a.sums) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        sum = sum + f2(u[i], u[i + 1]);
                }
                if (a.by_col.q && have)
                    put_col<false>(a.by_col, a.wide_qt, col, block0, 0, u);
            }
        } else if (a.by_col.q || a.sums) {
            // Word cl of the tile's rows (two columns): piece (cl % 32) / 4 of box cl / 32.
            uint32_t w[32];
            const uint8_t *x = stage + (cl >> 5) * T::kBox + 32 * rb * 128 + 4 * (cl & 3);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int r = i ^ (2 * rb);
                w[i] = *reinterpret_cast<const uint32_t *>(x + r * 128 + (((cl & 31) >> 2) ^ (r & 7)) * 16);
            }
            if (a.sums) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    sum = sum + f2(bf16_lo(w[i]), bf16_hi(w[i]));
            }
            if (a.by_col.q) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int64_t col = col_first + 2 * cl + k;
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] = k ? bf16_hi(w[i]) : bf16_lo(w[i]);
                    if (col < a.cols && block0 < a.rows)
                        put_col<true>(a.by_col, a.wide_qt, col, block0, 2 * rb, v);
                }
            }
        }
    }
    if (!a.sums)
        return;
    const float2 two = parts(sum);
    float total[2] = {BACKWARD ? two.x + two.y : two.x, two.y};
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
        total[k] += __shfl_xor_sync(0xffffffffu, total[k], 8);
        total[k] += __shfl_xor_sync(0xffffffffu, total[k], 16);
        const int64_t col = col_first + kSums * cl + k;
        if (rb == 0 && col < a.cols)
            (a.strips > 1 ? a.partials + strip * a.cols : a.sums)[col] = total[k];
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
static cudaError_t start_checkpoint(const CheckpointArgs &a, const CUtensorMap &mx, const CUtensorMap &mz, cudaStream_t stream)
{
    constexpr int kBytes = Tile<BACKWARD>::kBytes;
    const cudaError_t e = opt_in<checkpoint_kernel<BACKWARD, ACT>>(kBytes);
    if (e != cudaSuccess)
        return e;
    return launch_dependent(checkpoint_kernel<BACKWARD, ACT>, dim3(static_cast<unsigned>(a.strips * a.col_blocks)), dim3(kThreads), kBytes,
                            stream, a, mx, mz);
}

cudaError_t launch_checkpoint(CheckpointArgs &a, const CUtensorMap &mx, const CUtensorMap &mz, bool backward, cudaStream_t stream)
{
    const int wide_cols = backward ? Tile<true>::kCols : Tile<false>::kCols;
    a.col_blocks = (static_cast<int64_t>(a.cols) + wide_cols - 1) / wide_cols;
    auto wide = [](const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 32 == 0 && bytes % 32 == 0; };
    a.wide_q = wide(a.by_row.q, a.by_row.ldq);
    a.wide_qt = wide(a.by_col.q, a.by_col.ldq);
    a.wide_ht = wide(a.act_by_col.q, a.act_by_col.ldq);
    cudaError_t e = backward ? with_act(a.act, [&](auto tag) { return start_checkpoint<true, decltype(tag)::value>(a, mx, mz, stream); })
                             : start_checkpoint<false, Act::kNone>(a, mx, mz, stream);
    if (e == cudaSuccess && a.sums && a.strips > 1)
        e = launch_sum_partials(a.sums, a.cols, nullptr, 0, a.partials, static_cast<int>(a.strips), stream);
    return e;
}

cudaError_t read_checkpoint_status(int *status, int reset)
{
    const cudaError_t e = cudaMemcpyFromSymbol(status, g_status, sizeof(int));
    if (e != cudaSuccess || !reset)
        return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
}

}  // namespace mxfp4
