// Products grouped by expert with ragged sizes, on CTA pairs or single CTAs
// (tcgen05 cta_group::2 or ::1, block-scaled FP4 or byte formats):
//
//   plain  D[r, n] = alpha * sum_k A[r, k] B[e, n, k]             (bf16)
//   gated  h[r, f] = silu(alpha * g) * (alpha * u), g and u the products with
//          the gate and the up rows of B[e], quantised in 1x32 blocks along f
//          to the operand form the next product takes
//
// for every row r of group e, offsets[e] <= r < offsets[e + 1].
//
// A cluster of two CTAs computes a tile of 256 rows (of one group) x 256
// accumulator columns, as one M = 256, N = 256 MMA: CTA `rank` holds rows
// 128 rank .. +127 of the tile and half of B's rows in its shared memory and
// its 128 rows of the fp32 accumulator in its tensor memory.  Plain tiles take
// 256 columns of D.  A gated tile takes 128 columns f: accumulator columns
// 128 h + [0, 64) are the gate products of f0 + 64 h + [0, 64) and
// 128 h + [64, 128) the up products of the same f, so one thread of the
// epilogue finds g and u of 64 consecutive f in its own tensor-memory lane:
// activation, block maxima and rounding need no exchange between threads.
// Where the groups are small (launch_grouped has the rule) a CTA takes a tile of
// 128 rows x 256 columns by itself, one M = 128, N = 256 MMA, with all of B's rows
// in its own shared memory: twice as many tiles run together.  "Pair" below is
// then one CTA, and the leader.
// The rows of one group are the M side although decoding leaves most of them
// empty: a stage's MMAs take 512 tensor cycles whatever the rows, less than its
// 32 KB of weights take to stream from HBM.
//
// The grid is persistent: pair i takes tiles i, i + pairs, ... of a list that
// every CTA derives from `offsets` (prefix sums of the groups' row tiles in
// shared memory), row tiles fastest, so tiles that run together share weight
// panels in L2.  Empty groups have no tile and their weights are not read.
//
// Roles per CTA (512 threads): warps 4, 6, 7 load A rows with their scale atoms,
// B rows and B's scale atoms by TMA (a thread waits out each copy it issues,
// hence several); warps 12-15 move each stage's scale lines into tensor memory; warp 5
// of the leading CTA issues the MMAs; warps 0-3 and 8-11 are the epilogue, for
// accumulator columns [0, 128) and [128, 256).  A rows come from a 2-D map, so a
// tile may start at any row; rows past the group's end are loaded and computed
// but not stored, and what their scales hold reaches only their own row of the
// accumulator.  A CTA of which no row belongs to the group loads none.
// The atoms of A follow the grouped scale layout (expert.h).  MMAs that start
// beyond K are not issued, so scale bytes past K / 32 rounded up to the MMA's
// own are never used.
//
// What bounds it.  Decoding: the weights' bytes (64 groups, 26 of them with
// rows, N = K = 4096 in FP4: 232 MB in 37 us, 6.2 TB/s, 93 % of a plain copy's
// rate).  Prefill: the tensor pipe and its feed.  Groups of whole tiles in FP4:
// 7.2 PFLOP/s at K = 8192; at K = 2048 a tile is 8 stages, and its hand-overs
// show (32768 rows in ragged groups, N = 4000: 118 us, 4.6 PFLOP/s, the tensor
// pipe 61 % busy).  Bytes, gated (16384 rows in ragged groups, F = 2048,
// K = 4096): 250 us, 2.2 PFLOP/s, the pipe 77 % busy, of which 78 % of the tiles'
// rows exist; long runs are held at 1.6 to 1.75 GHz by the board's power.
#include <atomic>
#include <cuda_bf16.h>

#include "expert.h"
#include "ptx.cuh"
#include "quant.cuh"

namespace mxfp4 {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ int g_status = 0;

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z,
                                            int w, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
        : "memory");
}

// Byte formats: K = 32 per instruction, one E8M0 scale per row (scale_vec::1X),
// issued by one elected lane of a converged warp.
__device__ __forceinline__ void mma_mxf8_pair_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                    uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// The same by one CTA for its own accumulator.
__device__ __forceinline__ void mma_mxf8_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_mxf4_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` (of both CTAs of a pair) when the MMAs issued so far are done.
template <int SOLO>
__device__ __forceinline__ void commit_elect(uint64_t *bar, uint16_t mask)
{
    if constexpr (SOLO)
        asm volatile(
            "{\n\t.reg .pred e;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
            : "memory");
    else
        mma_commit_pair_elect(bar, mask);
}

// Registers move from the warpgroups that load and issue to the epilogue's,
// which holds a warp's 128 accumulator columns at once.  Their shares, 256
// threads each, stay within what the block was launched with (128 x 512; the
// launcher checks it).
constexpr int kEpilogueRegs = 192, kOtherRegs = 56;
static_assert((kEpilogueRegs + kOtherRegs) * 256 <= 128 * 512, "register split");

__device__ __forceinline__ void take_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
}

__device__ __forceinline__ void give_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

constexpr int kOutBoxBytes = 32 * 64;            // one epilogue warp's 32 rows x 32 bf16

// BYTES8: byte formats, 128 K and one scale atom per stage and 128-row block;
// otherwise packed E2M1, 256 K and two atoms.
// The plain form's epilogue keeps a 2 KB box per warp beside the ring.  Six
// stages then leave little room for the tile list, so that more groups than
// that (WIDE) run with five: 32768 rows, N = 4096, K = 2048: 107 against 113 us.
//
// SOLO: CTAs by themselves, tiles of 128 rows, a stage's B all of the tile's 256.
// With 32, at most 32 rows exist: a stage's A is those (the MMA's others are what
// lies behind, and reach only themselves).
template <bool BYTES8, bool GATED, bool WIDE, int SOLO>
struct GroupedCfg {
    static constexpr int STAGES = SOLO == 128 ? 4 : SOLO || (!GATED && WIDE) ? 5 : 6;
    static constexpr int ROWS = SOLO ? 128 : 256;
    static constexpr int OUT_BYTES = GATED ? 0 : (SOLO == 32 ? 2 : 8) * kOutBoxBytes;
    static constexpr int G = BYTES8 ? 1 : 2;
    static constexpr int A_BYTES = (SOLO == 32 ? 32 : 128) * 128;
    static constexpr int B_BYTES = (SOLO ? 256 : 128) * 128;
    static constexpr int SFA_BYTES = G * kSfAtomBytes;
    static constexpr int SFB_BYTES = 2 * G * kSfAtomBytes;
    static constexpr int STAGE_BYTES = (A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES + 1023) / 1024 * 1024;
    static constexpr int RING_BYTES = STAGES * STAGE_BYTES;
    static constexpr int BAR_BYTES = 256;
    static constexpr int MAX_GROUPS = GATED || SOLO == 32 ? kMaxGroups : SOLO ? 860 : WIDE ? kMaxGroups : 80;
    static constexpr int TABLE_BYTES = 2 * (MAX_GROUPS + 1) * 4;   // offsets and row-tile prefix sums
    static constexpr int USED_BYTES = RING_BYTES + OUT_BYTES + BAR_BYTES + TABLE_BYTES;
    // The ring wants 1024-byte alignment.  Dynamic shared memory starts on such
    // a boundary in a kernel without static shared memory; where there is
    // room, the start may still be rounded up.
    static constexpr int SLACK = USED_BYTES + 1024 <= 227 * 1024 ? 1024 : 0;
    static constexpr int SMEM_BYTES = USED_BYTES + SLACK;
    static constexpr int SF_COLS_A = 4 * G;
    static constexpr int SF_COLS_B = 8 * G;
    static constexpr int SF_COLS = SF_COLS_A + SF_COLS_B;
    static constexpr int ACC_COLS = 256;
    static constexpr int TMEM_COLS = 512;
    static constexpr int THREADS = 512;
    static constexpr int K_STAGE = BYTES8 ? 128 : 256;
    static constexpr int K_MMA = BYTES8 ? 32 : 64;
    static_assert(ACC_COLS + STAGES * SF_COLS <= TMEM_COLS, "tensor memory budget");
    static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// The tile list: groups' offsets and row-tile prefix sums in shared memory.
struct TileTable {
    const int *off;     // [groups + 1], clamped to [0, rows]
    const int *base;    // [groups + 1]: row tiles before the group
    int groups, nt;

    __device__ int tiles() const { return base[groups] * nt; }
};

struct Tile {
    int e;              // group
    int row0;           // first row of the tile
    int end;            // end of the group's rows
    int sfa;            // 128-row scale block of row0
    int q;              // column tile
    bool single;        // the group has no other row tile
};

template <int ROWS>
__device__ __forceinline__ Tile tile_at(const TileTable &t, int i)
{
    // The last group whose first tile is not after i (empty groups share their
    // successor's base and are passed over).
    int lo = 0, hi = t.groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.base[mid] * t.nt <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    Tile r;
    const int mt = t.base[lo + 1] - t.base[lo];
    const int local = i - t.base[lo] * t.nt;
    r.single = mt == 1;
    r.q = r.single ? local : local / mt;
    const int p = r.single ? 0 : local - r.q * mt;
    r.e = lo;
    r.row0 = t.off[lo] + p * ROWS;
    r.end = t.off[lo + 1];
    r.sfa = static_cast<int>(group_sf_block(t.off[lo], lo)) + ROWS / 128 * p;
    return r;
}

// Fill the tables: thread t takes groups 2t and 2t + 1 of up to 1024.  Up to 64
// groups are one warp's work and need no exchange between warps.  warp_sum: 16
// words of shared memory.  Ends with a block barrier.
//
// Ascending offsets make at most rows / ROWS + groups row tiles, which the host
// has checked to fit an int times the column tiles.  Offsets out of order can make
// up to groups / 2 times rows / ROWS: 32 unsigned bits hold that, and the table is
// cut off at the bound, so that a tile's number stays one whatever the offsets.
template <int ROWS>
__device__ __forceinline__ void build_tables(const int *offsets, int groups, int rows, int *off, int *base,
                                             int *warp_sum)
{
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const bool one_warp = groups <= 64;
    if (!one_warp || warp == 0) {
        int o[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const int e = 2 * t + i;
            o[i] = e <= groups ? min(max(offsets[e], 0), rows) : 0;
        }
        uint32_t c[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            c[i] = 2 * t + i < groups ? static_cast<uint32_t>(max(o[i + 1] - o[i], 0) + ROWS - 1) / ROWS : 0u;
        uint32_t sum = c[0] + c[1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(kFull, sum, d);
            if (lane >= d)
                sum += v;
        }
        const uint32_t bound = static_cast<uint32_t>(rows / ROWS) + static_cast<uint32_t>(min(groups, rows));
        uint32_t before = sum - c[0] - c[1];
        if (!one_warp) {
            if (lane == 31)
                warp_sum[warp] = static_cast<int>(sum);
            __syncthreads();
            for (int w = 0; w < warp; ++w)
                before += static_cast<uint32_t>(warp_sum[w]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 2 * t + i;
            if (e <= groups) {
                off[e] = o[i];
                base[e] = static_cast<int>(min(before, bound));
                before += c[i];
            }
        }
        if (2 * t + 2 == groups) {     // the entry past this thread's pair
            off[groups] = o[2];
            base[groups] = static_cast<int>(min(before, bound));
        }
    }
    __syncthreads();
}

// Cluster barrier at the end: the epilogue's stores need no ordering with the
// peer, and waiting for them here would delay the exit by their round trip.
__device__ __forceinline__ void cluster_leave(bool stored)
{
    if (stored)
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    else
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 2-D tiled bulk-tensor store from shared memory (x innermost), in this
// thread's current bulk group.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_addr(src)), "r"(x), "r"(y)
                 : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The group's shared memory has been read / its writes are done.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// 32 columns: alpha, one rounding, bf16 pairs.
__device__ __forceinline__ void round_bf16(const GroupedArgs &a, const uint32_t (&x)[32], uint32_t (&out)[16])
{
#pragma unroll
    for (int j = 0; j < 16; ++j)
        out[j] = bf16x2(a.alpha * __uint_as_float(x[2 * j]), a.alpha * __uint_as_float(x[2 * j + 1]));
}

// 32 columns of row r from n0 on, by this thread alone (rows of whole 16 bytes).
__device__ __forceinline__ void store_bf16(const GroupedArgs &a, int r, int n0, const uint32_t (&x)[32])
{
    if (n0 >= a.N)
        return;
    uint32_t out[16];
    round_bf16(a, x, out);
    uint16_t *d = a.D + static_cast<int64_t>(r) * a.ldd + n0;
    if (a.vec32_ok && n0 + 32 <= a.N) {
#pragma unroll
        for (int j = 0; j < 16; j += 8)
            st_global_v8(d + 2 * j, out[j], out[j + 1], out[j + 2], out[j + 3], out[j + 4], out[j + 5], out[j + 6],
                         out[j + 7]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        if (n0 + 2 * j + 8 <= a.N) {
            *reinterpret_cast<uint4 *>(d + 2 * j) = make_uint4(out[j], out[j + 1], out[j + 2], out[j + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (n0 + 2 * j + i < a.N)
                    d[2 * j + i] = static_cast<uint16_t>(out[j + i / 2] >> (16 * (i & 1)));
        }
    }
}

// A warp's 32 rows x 32 columns, rounded, into its 2 KB box (64-byte rows, 64-byte
// swizzle): chunk j of 16 bytes of row i at chunk j ^ (i / 2 % 4).
__device__ __forceinline__ void fill_box(uint8_t *box, int lane, const uint32_t (&out)[16])
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4 *>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16)) =
            make_uint4(out[4 * j], out[4 * j + 1], out[4 * j + 2], out[4 * j + 3]);
}

// The box's first `rows` rows to D[first ..][n0 ..] one element per lane: for
// rows that no wider store fits (an odd ldd puts every second one off a 4-byte
// boundary).  A row's 64 bytes leave together, where a thread that stored its
// own row's elements would touch 32 rows at a time.
__device__ __forceinline__ void store_box(const GroupedArgs &a, const uint8_t *box, int lane, int first, int rows, int n0)
{
    if (n0 + lane >= a.N)
        return;
    uint16_t *d = a.D + static_cast<int64_t>(first) * a.ldd + n0 + lane;
#pragma unroll 8
    for (int i = 0; i < rows; ++i, d += a.ldd)
        *d = *reinterpret_cast<const uint16_t *>(box + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) * 16) + (lane & 7) * 2);
}

// silu(alpha g) * (alpha u) in fp32.  The exponent's argument is rounded once,
// so the sigmoid is good to |g| 2^-24, and the reciprocal to 1 ulp: beside the
// products' own accumulation error.  A large negative g gives e = inf and 0.
__device__ __forceinline__ float gated_value(float alpha, uint32_t gate, uint32_t up)
{
    const float g = alpha * __uint_as_float(gate);
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));
    return g * s * (alpha * __uint_as_float(up));
}

// Columns f0 .. f0 + 63 of row r (row `local` of the 128-row scale block whose
// atoms start at byte `block`): activation in fp32, one rounding into the
// block's format.  gate, up: the products of columns [0, 32) and [32, 64).
template <QuantFmt Q>
__device__ __forceinline__ void store_gated(const GroupedArgs &a, int r, int local, int64_t block, int f0,
                                            const uint32_t (&gate0)[32], const uint32_t (&gate1)[32],
                                            const uint32_t (&up0)[32], const uint32_t (&up1)[32])
{
    constexpr int W = QuantTraits<Q>::kWords;
    if (f0 >= a.N)
        return;
    float h[32];
    uint32_t lo[W], hi[W];
#pragma unroll
    for (int i = 0; i < 32; ++i)
        h[i] = gated_value(a.alpha, gate0[i], up0[i]);
    uint32_t codes = quantize_block<Q>(h, lo);
    const bool both = f0 + 32 < a.N;
    // An odd last block's partner in the same MMA of the next product: any
    // finite scale serves its zero codes.
    uint32_t second = 0x7Fu;
    if (both) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            h[i] = gated_value(a.alpha, gate1[i], up1[i]);
        second = quantize_block<Q>(h, hi);
    }
    *reinterpret_cast<uint16_t *>(a.SH + block + sf_byte(local, f0 / 32)) = static_cast<uint16_t>(codes | (second << 8));
    uint8_t *q = a.H + static_cast<int64_t>(r) * a.ldh + (Q == QuantFmt::kE2M1 ? f0 / 2 : f0);
    if (a.vec32_ok && both) {
        if constexpr (W == 4) {
            st_global_v8(q, lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]);
        } else {
            st_global_v8(q, lo[0], lo[1], lo[2], lo[3], lo[4], lo[5], lo[6], lo[7]);
            st_global_v8(q + 32, hi[0], hi[1], hi[2], hi[3], hi[4], hi[5], hi[6], hi[7]);
        }
        return;
    }
#pragma unroll
    for (int w = 0; w < W; w += 4) {
        reinterpret_cast<uint4 *>(q)[w / 4] = make_uint4(lo[w], lo[w + 1], lo[w + 2], lo[w + 3]);
        if (both)
            reinterpret_cast<uint4 *>(q)[W / 4 + w / 4] = make_uint4(hi[w], hi[w + 1], hi[w + 2], hi[w + 3]);
    }
}

// OUT: -1 plain bf16, else static_cast<int>(QuantFmt) of the gated form.
template <bool BYTES8, int OUT, bool WIDE, int SOLO>
__global__ void __launch_bounds__(512, 1)
    grouped_product(const __grid_constant__ GroupedArgs a, const __grid_constant__ GroupedMaps maps)
{
    using Cf = GroupedCfg<BYTES8, (OUT >= 0), WIDE, SOLO>;
    constexpr int G = Cf::G;
    constexpr bool GATED = OUT >= 0;
    constexpr int STAGES = Cf::STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    if (Cf::SLACK == 0 && (raw & 1023u)) {       // (never seen; see GroupedCfg)
        if (threadIdx.x == 0)
            atomicExch(&g_status, -5 /* MXFP4_ERR_CUDA */);
        return;
    }
    uint8_t *smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t *stage_out = smem + Cf::RING_BYTES;     // the plain epilogue's boxes
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cf::RING_BYTES + Cf::OUT_BYTES);
    uint64_t *empty = full + STAGES;
    uint64_t *sf_ready = empty + STAGES;            // the leader's are used
    uint64_t *acc_full = sf_ready + STAGES;
    uint64_t *acc_empty = acc_full + 1;             // the leader's is used
    uint64_t *drain = acc_empty + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *warp_sum = reinterpret_cast<int *>(tmem_slot + 2);
    static_assert((3 * STAGES + 3) * 8 + 8 + 64 <= Cf::BAR_BYTES, "barriers");
    int *tab_off = reinterpret_cast<int *>(smem + Cf::RING_BYTES + Cf::OUT_BYTES + Cf::BAR_BYTES);
    int *tab_base = tab_off + Cf::MAX_GROUPS + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = SOLO ? 0u : cluster_ctarank() & 1u;
    const bool leader = rank == 0;
    const int pair = blockIdx.x / (SOLO ? 1 : 2);
    const int pairs = gridDim.x / (SOLO ? 1 : 2);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 3);          // this CTA's three producers
            mbar_init(&empty[s], 1);         // the pair's MMA commit
            mbar_init(&sf_ready[s], SOLO ? 4 : 8);   // the scale writers of both CTAs
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, SOLO ? 8 : 16); // the epilogue warps of both CTAs
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 5) {
        if constexpr (SOLO) {
            tmem_alloc(tmem_slot, Cf::TMEM_COLS);
            tmem_relinquish();
        } else {
            tmem_alloc_pair(tmem_slot, Cf::TMEM_COLS);
            tmem_relinquish_pair();
        }
    }
    if (warp == 4 && lane == 0) {
        prefetch_tensormap(&maps.A);
        prefetch_tensormap(&maps.A32);
        prefetch_tensormap(&maps.SA);
        prefetch_tensormap(&maps.B);
        prefetch_tensormap(&maps.SB);
    }
    tc_fence_before();
    if constexpr (SOLO)
        __syncthreads();
    else
        cluster_sync();                      // barriers of both CTAs initialised
    tc_fence_after();
    const uint64_t keep = l2_policy_evict_last();
    const uint64_t once = l2_policy_evict_first();
    // Arguments that the first steps use are fetched before the wait.
    const int *const offsets = a.offsets;
    const int groups = a.groups, rows = a.rows, nt = a.nt;
    asm volatile("" ::"l"(offsets), "r"(groups), "r"(rows), "r"(nt), "r"(a.kt), "r"(a.N), "l"(a.wait_limit));
    // Offsets and weights may come from the work before this grid, like
    // everything else; with a.early only the rows and their scales do.  A role
    // that those keep waiting first waits for the grid before, which has no
    // limit: the limit is for this kernel's own work.
    if (!a.early)
        pdl_wait_prerequisites();
    build_tables<Cf::ROWS>(offsets, groups, rows, tab_off, tab_base, warp_sum);
    const uint32_t tmem = *tmem_slot;
    TileTable table{tab_off, tab_base, groups, nt};
    // With single CTAs, tiles that would leave half of them idle are halved (128
    // accumulator columns; tile_at then counts twice as many), which takes a
    // stage's MMAs less time to issue: one-token block of 3 experts, 544 x 1504,
    // 12.3 us, with whole tiles 13.7.  Halving the last of several rounds as well
    // keeps SMs from the next launch: 32 rows in 25 groups 24.4 against 23.3.
    const bool halves = SOLO && table.tiles() <= pairs / 2;
    if (halves)
        table.nt *= 2;
    const int tiles = table.tiles();
    if (threadIdx.x == 0)
        pdl_launch_dependents();

    if (warp < 4 || (warp >= 8 && warp < 12)) {
        take_registers();
        // ------------------------------------------------------ epilogue --
        if (a.early)
            pdl_wait_prerequisites();
        const int quarter = warp & 3;
        const int half = warp >> 3;
        const bool idle = halves && half != 0;
        const int row = static_cast<int>(rank) * 128 + quarter * 32 + lane;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
        const uint32_t lead_empty = SOLO ? 0u : map_to_rank(smem_addr(acc_empty), 0);
        uint32_t acc_phase = 0;
        for (int t = pair; t < tiles; t += pairs) {
            const Tile tl = tile_at<Cf::ROWS>(table, t);
            bool ok = mbar_wait(acc_full, acc_phase, abort_flag, a.wait_limit, &g_status);
            if (!__all_sync(kFull, ok))
                break;
            acc_phase ^= 1u;
            tc_fence_after();
            const int r = tl.row0 + row;
            const bool mine = r < tl.end && !idle;
            // All 128 columns of the lane to registers, then the accumulator is
            // released: the next tile's MMAs wait for the reads alone.
            uint32_t acc[4][32];
            if (__any_sync(kFull, mine)) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld_32x32b_x32(t_lane + 32 * c, acc[c]);
                tmem_ld_wait(acc[0], acc[1]);
                tmem_ld_wait(acc[2], acc[3]);
            }
            // (Nobody waits after the last tile, and an arrive in flight must not
            // outlive the leading CTA.)
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && t + pairs < tiles) {
                if (leader)
                    mbar_arrive(acc_empty);
                else
                    mbar_arrive_cluster_relaxed(lead_empty);
            }
            if constexpr (!GATED) {
                const int n0 = tl.q * (halves ? 128 : 256) + half * 128;
                const int first = r - lane;
                const int rows_here = idle ? 0 : min(32, tl.end - first);
                if (rows_here > 0 && (!a.vec_ok || rows_here == 32)) {
                    // Four boxes of 32 rows x 32 columns through shared memory.
                    // Whole ones leave by TMA: a thread's own 32-byte stores
                    // touch a line each, and 64 KB of them per tile hold up
                    // the MMA warp's barrier polls in the same queue (32768 rows,
                    // N = 4000, K = 2048: 109 us, with those stores 122).
                    uint8_t *buf = stage_out + (SOLO == 32 ? half : half * 4 + quarter) * kOutBoxBytes;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (n0 + 32 * c >= a.N)
                            break;
                        uint32_t out[16];
                        round_bf16(a, acc[c], out);
                        if (lane == 0)
                            bulk_wait_read();
                        __syncwarp();
                        fill_box(buf, lane, out);
                        if (a.vec_ok)
                            fence_proxy_async_smem();
                        __syncwarp();
                        if (!a.vec_ok) {
                            store_box(a, buf, lane, first, rows_here, n0 + 32 * c);
                        } else if (lane == 0) {
                            tma_store_2d(&maps.D, buf, n0 + 32 * c, first);
                            bulk_commit();
                        }
                    }
                } else if (mine) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        store_bf16(a, r, n0 + 32 * c, acc[c]);
                }
            } else if (mine) {
                const int64_t block = static_cast<int64_t>(tl.sfa + row / 128) * (sf_groups(a.N) * kSfAtomBytes);
                store_gated<static_cast<QuantFmt>(OUT)>(a, r, row & 127, block,
                                                        tl.q * (halves ? 64 : 128) + half * 64, acc[0], acc[1], acc[2],
                                                        acc[3]);
            }
        }
        if (!GATED && lane == 0)
            bulk_wait();
    } else {
        give_registers();
        if (warp == 4 || warp == 6 || warp == 7) {
            // ------------------------------------------------------ producers --
            if (lane == 0) {
                const int role = warp == 4 ? 0 : warp - 5;   // 0: A and its scales, 1: B, 2: B's scales
                if (role == 0 && a.early)
                    pdl_wait_prerequisites();
                int stage = 0;
                uint32_t phase = 0;
                int issued = 0;
                bool stop = false;
                for (int t = pair; t < tiles && !stop; t += pairs) {
                    const Tile tl = tile_at<Cf::ROWS>(table, t);
                    const int arow = tl.row0 + static_cast<int>(rank) * 128;
                    const bool rows_here = arow < tl.end;
                    // Rows of a decoding step: a quarter of A's box (32 rows in 26
                    // groups, N = K = 4096: 40.4 us, with whole boxes 54.1).
                    const bool few = SOLO == 32 || tl.end - arow <= 32;
                    // A group of one row tile reads its weights once (same product
                    // with everything kept: 110 us against 109; 26 groups of a
                    // decoding step 41.3 against 40.4).
                    const uint64_t pol_b = tl.single ? once : keep;
                    const uint32_t unit = role == 0   ? (!rows_here ? 0 : (few ? 32 * 128 : Cf::A_BYTES) + Cf::SFA_BYTES)
                                          : role == 1 ? (halves ? Cf::B_BYTES / 2 : Cf::B_BYTES)
                                                      : Cf::SFB_BYTES;
                    for (int kt = 0; kt < a.kt; ++kt) {
                        if (!mbar_try_wait(smem_addr(&empty[stage]), phase ^ 1u)) {
                            // B's loaders run ahead as far as the ring goes.  (Asked
                            // only where the slot is not free yet: a test of its own
                            // on every stage cost the 32768 rows' product 1 %.)
                            if (a.early)
                                pdl_wait_prerequisites();
                            if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.wait_limit, &g_status)) {
                                stop = true;
                                break;
                            }
                        }
                        uint8_t *st = smem + stage * Cf::STAGE_BYTES;
                        uint8_t *sf = st + Cf::A_BYTES + Cf::B_BYTES;
                        mbar_arrive_expect_tx(&full[stage], unit);
                        if (role == 0) {
                            if (rows_here) {
                                tma_load_2d(st, few ? &maps.A32 : &maps.A, &full[stage], kt * 128, arow, keep);
                                tma_load_3d(sf, &maps.SA, &full[stage], 0, G * kt, tl.sfa + static_cast<int>(rank), keep);
                            }
                        } else if (role == 1) {
                            // Plain: 128 rows of B.  Gated: 64 gate rows and the
                            // same 64 up rows (the map's third dimension).
                            const int unit_n = GATED ? 64 : 128;
                            const int n = (halves ? tl.q : 2 * tl.q + static_cast<int>(rank)) * unit_n;
                            tma_load_4d(st + Cf::A_BYTES, &maps.B, &full[stage], kt * 128, n, 0, tl.e, pol_b);
                            if (SOLO && !halves) // what the peer of a pair would load
                                tma_load_4d(st + Cf::A_BYTES + 128 * 128, &maps.B, &full[stage], kt * 128,
                                            n + unit_n, 0, tl.e, pol_b);
                        } else {
                            // Plain: two 128-row blocks of the expert.  Gated: the
                            // block of the gate rows and the block of the up rows.
                            tma_load_4d(sf + Cf::SFA_BYTES, &maps.SB, &full[stage], 0, G * kt,
                                        GATED == halves ? (GATED ? tl.q / 2 : 2 * tl.q) : tl.q,
                                        GATED ? 2 * tl.e : tl.e, pol_b);
                        }
                        ++issued;
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
                if (*abort_flag) {
                    // Let the copies already issued land before the CTA exits.
                    for (int i = max(0, issued - STAGES); i < issued; ++i)
                        mbar_wait_drain(&full[i % STAGES], (i / STAGES) & 1u, a.wait_limit);
                }
            }
        } else if (warp >= 12) {
            // -------------------------------------------- scale writers --
            // Line `lane` of an atom: rows lane, lane + 32, lane + 64, lane + 96 of
            // its 128-row block, a word of four scales each; the four warps write
            // the four lane quarters' replicas.
            const int quarter = warp & 3;
            const uint32_t t_q = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + Cf::ACC_COLS;
            const uint32_t lead_ready = SOLO ? 0u : map_to_rank(smem_addr(&sf_ready[0]), 0);
            const int my_tiles = pair < tiles ? (tiles - 1 - pair) / pairs + 1 : 0;
            const int total = my_tiles * a.kt;
            // The second half of a gated tile has the second half of either block.
            const bool upper = GATED && halves && total > 0 && (tile_at<Cf::ROWS>(table, pair).q & 1);
            int stage = 0;
            uint32_t phase = 0;
            if (a.early)
                pdl_wait_prerequisites();
            for (int i = 0; i < total; ++i) {
                bool ok = mbar_wait(&full[stage], phase, abort_flag, a.wait_limit, &g_status);
                if (!__all_sync(kFull, ok))
                    break;
                const uint8_t *sf = smem + stage * Cf::STAGE_BYTES + Cf::A_BYTES + Cf::B_BYTES;
                uint32_t wa[4 * G], wb[8 * G];
    #pragma unroll
                for (int g = 0; g < G; ++g) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(sf + g * kSfAtomBytes + 16 * lane);
                    const uint4 x = *reinterpret_cast<const uint4 *>(sf + Cf::SFA_BYTES + g * kSfAtomBytes + 16 * lane);
                    const uint4 y =
                        *reinterpret_cast<const uint4 *>(sf + Cf::SFA_BYTES + (G + g) * kSfAtomBytes + 16 * lane);
                    wa[4 * g] = v.x;
                    wa[4 * g + 1] = v.y;
                    wa[4 * g + 2] = v.z;
                    wa[4 * g + 3] = v.w;
                    // Word j of block b of atom g -> column 8 g + 4 b + j.  Plain:
                    // blocks x, y.  Gated: the tile's first 128 rows are gate rows
                    // 0-63 and up rows 0-63 (words 0, 1 of either block).
                    uint32_t *w = wb + 8 * g;
                    w[0] = x.x;
                    w[1] = x.y;
                    w[2] = GATED ? y.x : x.z;
                    w[3] = GATED ? y.y : x.w;
                    w[4] = GATED ? x.z : y.x;
                    w[5] = GATED ? x.w : y.y;
                    w[6] = y.z;
                    w[7] = y.w;
                    if (SOLO && GATED && upper) {
                        w[0] = x.z;
                        w[1] = x.w;
                        w[2] = y.z;
                        w[3] = y.w;
                    }
                }
                const uint32_t slot = t_q + stage * Cf::SF_COLS;
                if constexpr (G == 2) {
                    tmem_st_32x32b_x8(slot, wa);
                    tmem_st_32x32b_x16(slot + Cf::SF_COLS_A, wb);
                } else {
                    tmem_st_32x32b_x4(slot, wa);
                    tmem_st_32x32b_x8(slot + Cf::SF_COLS_A, wb);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader)
                        mbar_arrive(&sf_ready[stage]);
                    else
                        mbar_arrive_cluster_relaxed(lead_ready + static_cast<uint32_t>(stage * sizeof(uint64_t)));
                }
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        } else if (warp == 5) {
            // ------------------------------------------------ MMA (leader) --
            if (leader) {
                const uint32_t idesc = BYTES8 ? (!SOLO ? a.idesc8 : halves ? a.idesc8_half : a.idesc8_solo)
                                              : idesc_mxf4(SOLO ? 128 : 256, halves ? 128 : 256);
                int stage = 0;
                uint32_t phase = 0, acc_phase = 0;
                bool stop = false;
                if (a.early)
                    pdl_wait_prerequisites();
                for (int t = pair; t < tiles && !stop; t += pairs) {
                    if (!mbar_wait(acc_empty, acc_phase ^ 1u, abort_flag, a.wait_limit, &g_status))
                        break;
                    tc_fence_after();
                    for (int kt = 0; kt < a.kt; ++kt) {
                        // sf_ready completes after the scale writers of both CTAs
                        // saw the stage's bytes land.
                        if (!mbar_wait(&sf_ready[stage], phase, abort_flag, a.wait_limit, &g_status)) {
                            stop = true;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t sfa = tmem + Cf::ACC_COLS + stage * Cf::SF_COLS;
                        const uint32_t sfb = sfa + Cf::SF_COLS_A;
                        const uint32_t st = smem_addr(smem + stage * Cf::STAGE_BYTES);
                        const uint64_t adesc = sdesc_kmajor_sw128(st);
                        const uint64_t bdesc = sdesc_kmajor_sw128(st + Cf::A_BYTES);
                        const int left = a.K - kt * Cf::K_STAGE;      // K elements of this stage
    #pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (j * Cf::K_MMA >= left)
                                break;
                            const uint32_t acc = (kt > 0 || j > 0) ? 1u : 0u;
                            if constexpr (BYTES8) {
                                const uint32_t id = idesc_sf_ids(idesc, j, j);
                                if constexpr (SOLO)
                                    mma_mxf8_elect(tmem, adesc + 2 * j, bdesc + 2 * j, id, sfa, sfb, acc);
                                else
                                    mma_mxf8_pair_elect(tmem, adesc + 2 * j, bdesc + 2 * j, id, sfa, sfb, acc);
                            } else {
                                const uint32_t id = idesc_sf_ids(idesc, (j & 1) * 2, (j & 1) * 2);
                                if constexpr (SOLO)
                                    mma_mxf4_elect(tmem, adesc + 2 * j, bdesc + 2 * j, id, sfa + (j >> 1) * 4,
                                                   sfb + (j >> 1) * 8, acc);
                                else
                                    mma_mxf4_pair_elect(tmem, adesc + 2 * j, bdesc + 2 * j, id, sfa + (j >> 1) * 4,
                                                        sfb + (j >> 1) * 8, acc);
                            }
                        }
                        commit_elect<SOLO>(&empty[stage], static_cast<uint16_t>(3u));
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!stop)
                        commit_elect<SOLO>(acc_full, static_cast<uint16_t>(3u));
                    acc_phase ^= 1u;
                }
                if (*abort_flag) {
                    commit_elect<SOLO>(drain, static_cast<uint16_t>(1u));
                    mbar_wait_drain(drain, 0, a.wait_limit);
                }
            }
        }
    }

    tc_fence_before();
    // No CTA leaves while its peer may still signal it.
    if constexpr (SOLO)
        __syncthreads();
    else
        cluster_leave(warp < 4 || (warp >= 8 && warp < 12));
    if (warp == 5) {
        tc_fence_after();
        if constexpr (SOLO)
            tmem_dealloc(tmem, Cf::TMEM_COLS);
        else
            tmem_dealloc_pair(tmem, Cf::TMEM_COLS);
    }
}

template <bool BYTES8, int OUT, bool WIDE, int SOLO>
cudaError_t launch_one(const GroupedArgs &a, const GroupedMaps &m, cudaStream_t stream)
{
    using Cf = GroupedCfg<BYTES8, (OUT >= 0), WIDE, SOLO>;
    auto kern = grouped_product<BYTES8, OUT, WIDE, SOLO>;
    static std::atomic<int> max_clusters[64];   // per device; 0 = not yet queried
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(Cf::THREADS);
    cfg.dynamicSmemBytes = Cf::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SOLO ? 0 : 1;
    int limit = dev < 64 ? max_clusters[dev].load() : 0;
    if (limit == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM_BYTES);
        if (e != cudaSuccess)
            return e;
        // The register split needs the registers of a 128-register launch.
        cudaFuncAttributes attributes;
        e = cudaFuncGetAttributes(&attributes, kern);
        if (e != cudaSuccess)
            return e;
        if (attributes.numRegs <= 120)
            return cudaErrorInvalidConfiguration;
        // Persistent: a CTA, or a pair, for each slot.
        if (SOLO) {
            int per_sm = 0;
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, Cf::THREADS, Cf::SMEM_BYTES);
            if (e == cudaSuccess)
                e = cudaDeviceGetAttribute(&limit, cudaDevAttrMultiProcessorCount, dev);
            limit *= per_sm;
        } else {
            cfg.gridDim = dim3(2);
            e = cudaOccupancyMaxActiveClusters(&limit, kern, &cfg);
        }
        if (e != cudaSuccess)
            return e;
        if (limit <= 0)
            return cudaErrorInvalidConfiguration;
        if (dev < 64)
            max_clusters[dev] = limit;
    }
    // The host does not know the offsets: at most this many tiles.  (SMs beyond
    // them are left to the next launch, which may start early.)
    const int64_t row_tiles = static_cast<int64_t>(a.rows) / Cf::ROWS + (a.groups < a.rows ? a.groups : a.rows);
    int64_t most = row_tiles * a.nt;
    if (SOLO && 2 * most <= limit)
        most *= 2;                               // as halves
    const int pairs = most < limit ? static_cast<int>(most) : limit;
    cfg.gridDim = dim3(static_cast<unsigned>(SOLO ? pairs : 2 * pairs));
    cudaLaunchAttribute &dependent = attr[cfg.numAttrs++];
    dependent.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    dependent.val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, m);
}

template <bool WIDE, int SOLO>
cudaError_t launch_form(const GroupedArgs &a, const GroupedMaps &m, bool bytes8, int out, cudaStream_t stream)
{
    switch (out) {
    case -1:
        return bytes8 ? launch_one<true, -1, WIDE, SOLO>(a, m, stream) : launch_one<false, -1, WIDE, SOLO>(a, m, stream);
    case 0: return launch_one<false, 0, true, SOLO>(a, m, stream);     // (the gated forms have room for any table)
    case 1: return launch_one<true, 1, true, SOLO>(a, m, stream);
    default: return launch_one<true, 2, true, SOLO>(a, m, stream);
    }
}

}  // namespace

cudaError_t launch_grouped(const GroupedArgs &a, const GroupedMaps &m, bool bytes8, int out, cudaStream_t stream)
{
    if (out >= 0 && (out == 0) == bytes8)
        return cudaErrorInvalidValue;
    // Single CTAs while nearly all groups have 128 rows or fewer (the host knows
    // their average alone): twice as many tiles run together, and a group's last
    // one wastes half as much; a group of more reads B again.  4 tokens x 8 of 64
    // experts, N = K = 4096: 36.5 us, with pairs 41.3; 32 experts, 2048 x 2048, 64
    // rows on average: 16.3 and 19.8, 96: 17.8 and 20.3, 128: 21.2 and 20.4; gated
    // bytes, 16 experts, 96: 15.2 and 17.9, 128: 22.1 and 18.5.
    if (a.rows <= 32)                            // (one token x 4 experts: 9.2 us, with 128 rows of A 9.9)
        return launch_form<true, 32>(a, m, bytes8, out, stream);
    if (a.rows <= 112 * static_cast<int64_t>(a.groups) &&
        (out >= 0 || a.groups <= GroupedCfg<false, false, true, 128>::MAX_GROUPS))
        return launch_form<true, 128>(a, m, bytes8, out, stream);
    return a.groups > GroupedCfg<false, false, false, 0>::MAX_GROUPS ? launch_form<true, 0>(a, m, bytes8, out, stream)
                                                                     : launch_form<false, 0>(a, m, bytes8, out, stream);
}

cudaError_t read_grouped_status(int *status, int reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(status, g_status, sizeof(int));
    if (e != cudaSuccess || !reset)
        return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
}

}  // namespace mxfp4
