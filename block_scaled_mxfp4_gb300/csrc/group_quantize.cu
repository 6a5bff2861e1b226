// Grouped quantiser: bf16 rows to the operand of the grouped products.
#include <cuda_bf16.h>

#include "expert.h"
#include "launch.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace mxfp4 {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ------------------------------------------------------- grouped quantiser --
//
// One thread per 1x32 block of a source row: the block is read and rounded
// once and stored at each of the row's destinations.  The four threads of an
// atom's word (four consecutive blocks of a row) put their scale codes
// together and one of them stores the word.  Blocks move in 32-byte accesses,
// a whole sector per thread.  The destinations of four slots are looked up
// together, so that a row costs two dependent round trips (slot, then offset)
// and not two for each slot.
//
// Bound by HBM when there are many rows (one read and k writes of each): 8192
// rows of 8192, four E4M3 copies, 402 MB in 67 us, 6.0 TB/s or 90 % of a plain
// copy's rate; with 16-byte accesses instead it takes 77 us.  Bound by the launch
// when there are few: 64 rows of 2048, 3.0 us a call, an empty one's 2.9.

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

}  // namespace

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
    // Few blocks of work: small CTAs, so that they spread over the SMs (64 rows of
    // 2048, calls in a graph: 2.1 us, with 256 threads 2.6).
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

}  // namespace mxfp4
