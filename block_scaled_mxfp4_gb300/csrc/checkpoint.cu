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
// A block of 256 threads takes tiles of 128 rows, one below the other, by 128 columns
// (128 threads, 64 by 64 in the backward pass), copied to shared memory by TMA while the
// tile before is worked on.
//
// Why not straight from global memory, a row or column per lane: each such
// access touches 32 lines, and the L1's tag stage, one line a cycle, was 80 %
// busy at half of HBM's rate.  Copies by cp.async instead of TMA took as many of
// its cycles as all stores together.

constexpr int kSms = 152;

template <bool BACKWARD>
struct Tile {
    static constexpr int kThreads = BACKWARD ? 128 : 256;
    static constexpr int kRows = BACKWARD ? 64 : 128;
    static constexpr int kCols = BACKWARD ? 64 : 128;
    static constexpr int kBox = kRows * 128;             // 64 columns of x: 128-byte rows, 128-byte swizzle
    static constexpr int kXBytes = kCols / 64 * kBox;
    static constexpr int kZBytes = BACKWARD ? kRows * 64 : 0;       // 64-byte rows, 64-byte swizzle
    static constexpr int kStage = kXBytes + kZBytes;
    static constexpr int kDz = BACKWARD ? kRows * 256 : 0;          // dz, fp32
    static constexpr int kCodes = BACKWARD ? kRows * kCols : 0;     // of one output of a tile
    static constexpr int kScales = BACKWARD ? 2 * kThreads * 4 : 0; // z's scales of two tiles
    static constexpr int kAlign = BACKWARD ? 2048 : 1024;           // the swizzle's, and that of dz's rows
    static constexpr int kBytes = 2 * kStage + kDz + 3 * kCodes + kScales + kAlign - 1024;   // (the base is on 1024)
    static constexpr int kResident = BACKWARD ? 4 : 3;
};

__device__ int g_status = 0;                     // bounded waits that ran out

// A block's part of a column's sum.
__device__ __forceinline__ void put_sum(const CheckpointArgs &a, int64_t strip, int64_t col, float v)
{
    (a.strips > 1 ? a.partials + strip * a.cols : a.sums)[col] = v;
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
__device__ __forceinline__ uint32_t put_block(const float (&v)[32], int fmt, uint8_t *q, bool wide)
{
    uint32_t w[8];
    const uint32_t code = fmt == 0 ? quantize_block_pairs<QuantFmt::kE4M3>(v, w) : quantize_block_pairs<QuantFmt::kE5M2>(v, w);
    st_sector(q, w, wide);
    return code;
}

// Two codes -> two floats (exact: every E4M3 and E5M2 value is an fp16 value).
template <int FMT>
__device__ __forceinline__ F2 values_of(uint16_t in)
{
    uint32_t h;
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
__device__ __forceinline__ void load_tile(const CUtensorMap *x, const CUtensorMap *z, uint8_t *stage, uint64_t *full, int64_t row, int64_t col)
{
    using T = Tile<BACKWARD>;
    const int row0 = static_cast<int>(row), col0 = static_cast<int>(col);
    const uint64_t policy = l2_policy_evict_first();
    mbar_arrive_expect_tx(full, T::kStage);
#pragma unroll
    for (int k = 0; k < T::kCols / 64; ++k)
        tma_load_2d(stage + k * T::kBox, x, full, col0 + 64 * k, row0, policy);
    if constexpr (BACKWARD)
        tma_load_2d(stage + T::kXBytes, z, full, col0, row0, policy);
}

// One column block's codes and scale.  v[i] is row i ^ rows of the block (0, 2, 4 or 6): the codes
// change places accordingly, in units of two.
__device__ __forceinline__ void put_col(const CodesOut &o, bool wide, int64_t col, int64_t row0, int rows, const float (&v)[32])
{
    uint32_t w[8];
    const uint32_t code = o.fmt == 0 ? quantize_block_pairs<QuantFmt::kE4M3>(v, w) : quantize_block_pairs<QuantFmt::kE5M2>(v, w);
    const uint32_t order = rows & 2 ? 0x1032u : 0x3210u;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint32_t lo = __byte_perm(w[i], 0u, order), hi = __byte_perm(w[i + 1], 0u, order);
        w[i] = rows & 4 ? hi : lo;
        w[i + 1] = rows & 4 ? lo : hi;
    }
    st_sector(o.q + col * o.ldq + row0, w, wide);
    o.s[col * o.lds + row0 / 32] = static_cast<uint8_t>(code);
}

// x in both orientations.  A lane takes 32 values of a row, and 32 of a column: a block
// of either orientation is one lane's, and nothing needs a shuffle.  Lanes are dealt so
// that a warp's stores fall into whole lines (128 bytes of codes are four lanes') and
// its shared-memory reads on different banks: TMA's swizzle moves 16-byte pieces by the
// row, and lanes 32 rows apart read their column's rows in orders of their own.
__global__ void __launch_bounds__(Tile<false>::kThreads, Tile<false>::kResident)
    checkpoint_kernel(const __grid_constant__ CheckpointArgs a, const __grid_constant__ CUtensorMap mx)
{
    using T = Tile<false>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t full[2];
    __shared__ int abort_flag;
    uint8_t *smem = smem_raw;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t strip = blockIdx.x / a.across, col_first = blockIdx.x % a.across * static_cast<int64_t>(T::kCols);
    const int64_t row_first = strip * a.steps * T::kRows;
    const int tiles = static_cast<int>(min((a.rows - row_first + T::kRows - 1) / T::kRows, static_cast<int64_t>(a.steps)));
    // The thread's column block: eight neighbouring pairs of columns to eight lanes, the four row
    // blocks of a column to lanes eight apart.
    const int rb = lane >> 3, cl = warp * 8 + (lane & 7);
    F2 sum = f2(0.0f);                                   // of two columns
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
        load_tile<false>(&mx, nullptr, smem, &full[0], row_first, col_first);
    }
    for (int n = 0; n < tiles; ++n) {
        const int64_t row0 = row_first + static_cast<int64_t>(n) * T::kRows;
        const uint32_t phase = n / 2 & 1;
        const uint8_t *stage = smem + (n & 1) * T::kStage;
        const bool ok = mbar_wait(&full[n & 1], phase, &abort_flag, a.wait_limit, &g_status);
        if (__syncthreads_or(!ok)) {
            if (threadIdx.x == 0)
                mbar_wait_drain(&full[n & 1], phase, a.wait_limit);     // its copies land before the block leaves
            return;
        }
        // Every thread is past the tile before.
        if (n + 1 < tiles && threadIdx.x == 0)
            load_tile<false>(&mx, nullptr, smem + (~n & 1) * T::kStage, &full[~n & 1], row0 + T::kRows, col_first);
        if (a.by_row.q) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // Eight neighbouring rows to eight neighbouring lanes.
                const int r = (k * 8 + warp) * 8 + (lane & 7), b = lane >> 3;
                const int64_t row = row0 + r, col0 = col_first + 32 * b;
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
                if (row < a.rows && col0 < a.cols) {
                    const uint32_t code = put_block(v, a.by_row.fmt, a.by_row.q + row * a.by_row.ldq + col0, a.wide_q);
                    a.by_row.s[row * a.by_row.lds + col0 / 32] = static_cast<uint8_t>(code);
                }
            }
        }
        if (a.by_col.q || a.sums) {
            // Word cl of the tile's rows (two columns): piece (cl % 32) / 4 of box cl / 32.
            const int64_t block0 = row0 + 32 * rb;
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
                        put_col(a.by_col, a.wide_qt, col, block0, 2 * rb, v);
                }
            }
        }
    }
    if (!a.sums)
        return;
    const float2 two = parts(sum);
    float total[2] = {two.x, two.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        total[k] += __shfl_xor_sync(0xffffffffu, total[k], 8);
        total[k] += __shfl_xor_sync(0xffffffffu, total[k], 16);
        const int64_t col = col_first + 2 * cl + k;
        if (rb == 0 && col < a.cols)
            put_sum(a, strip, col, total[k]);
    }
}

// -------------------------------------------------- the activation's backward --
//
// Two passes over a tile.  Down the columns: a lane takes two neighbouring columns of
// 16 rows, computes act(z) and dz there, and rounds both along the columns at once,
// from registers (two lanes share a block of 32 rows and exchange its largest
// magnitude).  dz alone goes through shared memory, and the second pass rounds it along
// the rows, a block per lane.  Computing along the rows sent act(z) and dz through
// shared memory, 19 bytes of its traffic per value against 14.  Codes are gathered in
// shared memory too and leave it as whole boxes by TMA: stored by the lanes, each 32-byte
// sector took the L1's data stage most of a cycle, a third of all its work.
//
// 8192 x 16384 with GELU, all outputs but dz itself: 207 us, 4.0 TB/s, of 121 that its
// bytes need; 191 with its tanh form, 190 with SiLU, 188 with none.  (Computing along the rows 245, with the
// lanes' own stores 239 of then 233, in blocks of 256 threads and tiles of 128 rows, whose
// passes overlap less, 233.)  What bounds it is issue: 41 instructions per value, 14 of
// them GELU's, on 16 warps an SM, which act(z) and dz of 32 values in registers allow.
//
// A warp has 16 columns and all 64 rows: a column's 64 codes are one row of its
// box.  Its four groups of 16 rows take them in orders of their own, row i ^ key with the
// keys 0, 4, 2 and 6, and TMA's swizzle (the row's low bits move a 16-byte piece) spreads
// each step's four rows, two pieces of x each, over all banks.  dz is laid out by the
// same rule in rows of 256 bytes; a half-warp's keys, four apart, spread its four pieces of
// either row too.  Offsets of row i ^ key are the key's with i's bits flipped.

// Two columns' values in the lane's 16 rows: their codes to shared memory (the first column's row of
// them at `codes`, in its 16-byte piece `at`, moved by the column's bits), and the scales of the first
// `have` of them.
template <QuantFmt Q>
__device__ __forceinline__ void put_two_columns(const CodesOut &o, uint8_t *codes, int have, int64_t col, int64_t row, int key, int half, const float2 (&v)[16])
{
    float amax[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        amax[0] = max_abs3(amax[0], v[i].x, v[i + 1].x);
        amax[1] = max_abs3(amax[1], v[i].y, v[i + 1].y);
    }
    uint32_t code[2];
    float inv[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float other = __shfl_xor_sync(0xffffffffu, amax[k], 8);      // the block's other 16 rows
        code[k] = block_scale8<Q>(max_abs3(amax[k], other, other), inv[k]);
    }
    constexpr int kF = Q == QuantFmt::kE4M3 ? 0 : 1;
    uint32_t w[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 *p = v + 4 * i;
        w[0][i] = f8x2<kF>(p[0].x * inv[0], p[1].x * inv[0]) | (f8x2<kF>(p[2].x * inv[0], p[3].x * inv[0]) << 16);
        w[1][i] = f8x2<kF>(p[0].y * inv[1], p[1].y * inv[1]) | (f8x2<kF>(p[2].y * inv[1], p[3].y * inv[1]) << 16);
    }
    // Row i ^ key to place i: bytes within a word by the key's low bits, words in pairs by its third.
    const uint32_t order = 0x3210u ^ (0x1111u * (key & 3));
    const bool swap = key & 4;
    const int at = (static_cast<int>(row / 16) & 3) ^ (static_cast<int>(col / 2) & 3);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = __byte_perm(w[k][i], 0u, order);
        *reinterpret_cast<uint4 *>(codes + 64 * k + at * 16) =
            make_uint4(swap ? u[1] : u[0], swap ? u[0] : u[1], swap ? u[3] : u[2], swap ? u[2] : u[3]);
    }
    // One of the block's two lanes stores the one column's scale, one the other's.
    if (have > half)
        o.s[(col + half) * o.lds + row / 32] = static_cast<uint8_t>(half ? code[1] : code[0]);
}

__device__ __forceinline__ void put_two_columns(const CodesOut &o, uint8_t *codes, int have, int64_t col, int64_t row, int key, int half, const float2 (&v)[16])
{
    if (o.fmt == 0)
        put_two_columns<QuantFmt::kE4M3>(o, codes, have, col, row, key, half, v);
    else
        put_two_columns<QuantFmt::kE5M2>(o, codes, have, col, row, key, half, v);
}

// act(z) and dz of the lane's 16 rows, dz to its place in shared memory too.  The addresses are
// those of row `key` of its group, in arrays aligned to their XOR's range.
template <Act ACT, int FMT>
__device__ __forceinline__ void back_columns(uint32_t xa, uint32_t za, uint32_t sa, uint32_t pa, float2 (&h)[16], float2 (&d)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int lo = i & 7, hi = i >> 3;
        uint32_t x;
        uint16_t z;
        float s;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"((xa ^ (lo * 144)) + hi * 1024));
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(z) : "r"((za ^ (lo * 64 + (lo >> 1) * 16)) + hi * 512));
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"((sa ^ (lo * 4)) + hi * 32));
        F2 act, slope;
        act_and_slope2<ACT>(values_of<FMT>(z) * f2(s), act, slope);
        h[i] = parts(act);
        d[i] = parts(f2(bf16_lo(x), bf16_hi(x)) * slope);
    }
    // (after the loads: a store between them, which could be of their bytes, would keep them in order)
#pragma unroll
    for (int i = 0; i < 16; ++i)
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"((pa ^ ((i & 7) * 272)) + (i >> 3) * 2048), "f"(d[i].x), "f"(d[i].y) : "memory");
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

template <Act ACT>
__global__ void __launch_bounds__(Tile<true>::kThreads, Tile<true>::kResident)
    act_backward_kernel(const __grid_constant__ CheckpointArgs a, const __grid_constant__ BackwardMaps maps)
{
    using T = Tile<true>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t full[2];
    __shared__ int abort_flag;
    uint8_t *smem = smem_raw + ((T::kAlign - smem_addr(smem_raw) % T::kAlign) % T::kAlign);
    uint8_t *dz = smem + 2 * T::kStage, *h_codes = dz + T::kDz, *dz_codes = h_codes + T::kCodes, *row_codes = dz_codes + T::kCodes,
            *scales = row_codes + T::kCodes;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t strip = blockIdx.x / a.across, col_first = blockIdx.x % a.across * static_cast<int64_t>(T::kCols);
    const int64_t row_first = strip * a.steps * T::kRows;
    const int tiles = static_cast<int>(min((a.rows - row_first + T::kRows - 1) / T::kRows, static_cast<int64_t>(a.steps)));
    // The column pass: pair of columns, group of rows, and the offsets of the group's row `key`.
    const int pair = lane & 7, group = lane >> 3, key = (group & 1) << 2 | (group & 2);
    const int top = 16 * group + key;
    const uint32_t xo = top * 128 + ((2 * warp + (pair >> 2)) ^ key) * 16 + 4 * (pair & 3);
    const uint32_t zo = top * 64 + (warp ^ (key >> 1)) * 16 + 2 * pair;
    const uint32_t so = (warp >> 1) * (4 * T::kRows) + top * 4;
    const uint32_t po = top * 256 + ((4 * warp + (pair >> 1)) ^ key) * 16 + 8 * (pair & 1);
    float2 sum = make_float2(0.0f, 0.0f);                // of two columns
    // The row pass: eight neighbouring rows to eight neighbouring lanes, the two blocks of a row to lanes eight apart.
    const int rr = warp * 16 + (lane & 7) + 8 * (lane >> 4), rb = (lane >> 3) & 1;
    if (threadIdx.x == 0) {
        mbar_init(&full[0], 1);
        mbar_init(&full[1], 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait_prerequisites();
    auto load = [&](int stage, int64_t row0) {
        load_tile<true>(&maps.x, &maps.z, smem + stage * T::kStage, &full[stage], row0, col_first);
    };
    // The scale of z in the tile's row threadIdx % 64, block threadIdx / 64.
    auto z_scale = [&](int64_t row0) -> uint32_t {
        const int64_t row = row0 + threadIdx.x % T::kRows, col0 = col_first + threadIdx.x / T::kRows * 32;
        return row < a.rows && col0 < a.cols ? a.sz[row * a.ld_sz + col0 / 32] : 127u;
    };
    auto put_scale = [&](int n, uint32_t code) {
        *reinterpret_cast<float *>(scales + (n & 1) * (4 * T::kThreads) + 4 * threadIdx.x) = e8m0_value(code);
    };
    if (threadIdx.x == 0) {
        pdl_launch_dependents();
        load(0, row_first);
        if (tiles > 1)
            load(1, row_first + T::kRows);
    }
    put_scale(0, z_scale(row_first));
    for (int n = 0; n < tiles; ++n) {
        const int64_t row0 = row_first + static_cast<int64_t>(n) * T::kRows;
        const uint32_t phase = n / 2 & 1;
        const uint8_t *stage = smem + (n & 1) * T::kStage;
        const bool ok = mbar_wait(&full[n & 1], phase, &abort_flag, a.wait_limit, &g_status);
        if (threadIdx.x == 0)
            bulk_wait_read();                            // the codes along the columns are on their way
        if (__syncthreads_or(!ok)) {
            if (threadIdx.x == 0) {                      // the copies in flight land before the block leaves
                mbar_wait_drain(&full[n & 1], phase, a.wait_limit);
                if (n + 1 < tiles)
                    mbar_wait_drain(&full[~n & 1], (n + 1) / 2 & 1, a.wait_limit);
                bulk_wait();
            }
            return;
        }
        // Every thread is past the tile before, its codes and the scales are in place.
        if (n > 0 && a.by_row.q && threadIdx.x == 0) {
            tma_store_2d(&maps.by_row, row_codes, static_cast<int>(col_first), static_cast<int>(row0) - T::kRows);
            bulk_commit();
        }
        const uint32_t code = n + 1 < tiles ? z_scale(row0 + T::kRows) : 0u;
        const bool rows_too = a.by_row.q || a.dz;
        {
            float2 h[16], d[16];
            const uint32_t xa = smem_addr(stage) + xo, za = smem_addr(stage) + T::kXBytes + zo,
                           sa = smem_addr(scales) + (n & 1) * (4 * T::kThreads) + so, pa = smem_addr(dz) + po;
            if (a.fmt_z == 0)
                back_columns<ACT, 0>(xa, za, sa, pa, h, d);
            else
                back_columns<ACT, 1>(xa, za, sa, pa, h, d);
            const int64_t col = col_first + 16 * warp + 2 * pair, row = row0 + 16 * group;
            const int have = (row & ~int64_t{31}) >= a.rows ? 0 : static_cast<int>(min(a.cols - col, int64_t{2}));
            if (a.act_by_col.q)
                put_two_columns(a.act_by_col, h_codes + (16 * warp + 2 * pair) * 64, have, col, row, key, group & 1, h);
            if (a.sums) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sum.x += d[i].x;
                    sum.y += d[i].y;
                }
            }
            if (a.by_col.q)
                put_two_columns(a.by_col, dz_codes + (16 * warp + 2 * pair) * 64, have, col, row, key, group & 1, d);
        }
        if (n + 1 < tiles)
            put_scale(n + 1, code);
        fence_proxy_async_smem();
        if (threadIdx.x == 0)
            bulk_wait_read();                            // the last tile's codes along the rows are on their way
        __syncthreads();
        if (threadIdx.x == 0) {
            if (n + 2 < tiles)
                load(n & 1, row0 + 2 * T::kRows);
            if (a.act_by_col.q)
                tma_store_2d(&maps.act_by_col, h_codes, static_cast<int>(row0), static_cast<int>(col_first));
            if (a.by_col.q)
                tma_store_2d(&maps.by_col, dz_codes, static_cast<int>(row0), static_cast<int>(col_first));
            bulk_commit();
        }
        const int64_t row = row0 + rr, col0 = col_first + 32 * rb;
        if (rows_too && row < a.rows && col0 < a.cols) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 p = *reinterpret_cast<const float4 *>(dz + rr * 256 + ((8 * rb + i) ^ (rr & 7)) * 16);
                v[4 * i] = p.x;
                v[4 * i + 1] = p.y;
                v[4 * i + 2] = p.z;
                v[4 * i + 3] = p.w;
            }
            if (col0 + 32 > a.cols) {
                // Behind the last column z is 0 times the block's scale: NaN where that is.
#pragma unroll
                for (int i = 1; i < 32; ++i)
                    if (col0 + i >= a.cols)
                        v[i] = 0.0f;
            }
            if (a.dz)
                put_dz(a, row, col0, v);
            if (a.by_row.q) {
                uint32_t w[8];
                const uint32_t scale = a.by_row.fmt == 0 ? quantize_block_pairs<QuantFmt::kE4M3>(v, w) : quantize_block_pairs<QuantFmt::kE5M2>(v, w);
                a.by_row.s[row * a.by_row.lds + col0 / 32] = static_cast<uint8_t>(scale);
                uint4 *q = reinterpret_cast<uint4 *>(row_codes + rr * 64);
                q[(2 * rb) ^ ((rr >> 1) & 3)] = make_uint4(w[0], w[1], w[2], w[3]);
                q[(2 * rb + 1) ^ ((rr >> 1) & 3)] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
        fence_proxy_async_smem();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        if (a.by_row.q) {
            tma_store_2d(&maps.by_row, row_codes, static_cast<int>(col_first), static_cast<int>(row_first) + (tiles - 1) * T::kRows);
            bulk_commit();
        }
        bulk_wait();
    }
    if (!a.sums)
        return;
    float total[2] = {sum.x, sum.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int m = 8; m < 32; m *= 2)
            total[k] += __shfl_xor_sync(0xffffffffu, total[k], m);
        const int64_t col = col_first + 16 * warp + 2 * pair + k;
        if (group == 0 && col < a.cols)
            put_sum(a, strip, col, total[k]);
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

void checkpoint_shape(CheckpointArgs &a, bool backward)
{
    const int wide = backward ? Tile<true>::kCols : Tile<false>::kCols;
    const int tall = backward ? Tile<true>::kRows : Tile<false>::kRows;
    const int64_t down = (static_cast<int64_t>(a.rows) + tall - 1) / tall;
    a.across = (static_cast<int64_t>(a.cols) + wide - 1) / wide;
    // Tiles below one another in a block as long as that leaves several rounds of blocks.  16384 x 8192
    // in both forms with sums took 104 us with 4 of them, 106 with 2, 111 with 8, and 115 shared out among
    // resident blocks beforehand; the backward pass of 8192 x 16384 205 with 4, 220 with 2, 204 with 8.
    const int64_t resident = kSms * (backward ? Tile<true>::kResident : Tile<false>::kResident), tiles = down * a.across;
    a.steps = tiles >= 16 * resident ? 4 : tiles >= 4 * resident ? 2 : 1;
    a.strips = (down + a.steps - 1) / a.steps;
}

cudaError_t launch_sum_partials(float *a, int64_t na, float *b, int64_t nb, const float *partials, int strips, cudaStream_t stream)
{
    return launch_dependent(sum_partials_kernel, dim3(static_cast<unsigned>((na + nb + 31) / 32)), dim3(1024), 0, stream, a, na, b, nb,
                            partials, strips);
}

template <Act ACT>
static cudaError_t start_backward(const CheckpointArgs &a, const BackwardMaps &maps, cudaStream_t stream)
{
    constexpr int kBytes = Tile<true>::kBytes;
    const cudaError_t e = opt_in<act_backward_kernel<ACT>, kBytes>();
    if (e != cudaSuccess)
        return e;
    return launch_dependent(act_backward_kernel<ACT>, dim3(static_cast<unsigned>(a.strips * a.across)), dim3(Tile<true>::kThreads), kBytes, stream, a, maps);
}

static cudaError_t finish_sums(const CheckpointArgs &a, cudaStream_t stream)
{
    return a.sums && a.strips > 1 ? launch_sum_partials(a.sums, a.cols, nullptr, 0, a.partials, static_cast<int>(a.strips), stream) : cudaSuccess;
}

cudaError_t launch_checkpoint(CheckpointArgs &a, const CUtensorMap &mx, cudaStream_t stream)
{
    auto wide = [](const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 32 == 0 && bytes % 32 == 0; };
    a.wide_q = wide(a.by_row.q, a.by_row.ldq);
    a.wide_qt = wide(a.by_col.q, a.by_col.ldq);
    constexpr int kBytes = Tile<false>::kBytes;
    cudaError_t e = opt_in<checkpoint_kernel, kBytes>();
    if (e == cudaSuccess)
        e = launch_dependent(checkpoint_kernel, dim3(static_cast<unsigned>(a.strips * a.across)), dim3(Tile<false>::kThreads), kBytes, stream, a, mx);
    return e == cudaSuccess ? finish_sums(a, stream) : e;
}

cudaError_t launch_act_backward(const CheckpointArgs &a, const BackwardMaps &maps, cudaStream_t stream)
{
    const cudaError_t e = with_act(a.act, [&](auto tag) { return start_backward<decltype(tag)::value>(a, maps, stream); });
    return e == cudaSuccess ? finish_sums(a, stream) : e;
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
