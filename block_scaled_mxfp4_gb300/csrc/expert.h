// Internal launchers of the expert-layer operators: routing, grouped
// quantisation, grouped products, the gated join.  Arguments are checked in
// expert_api.cu; the ABI is in include/mxfp4_gemm.h.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "internal.h"

namespace mxfp4 {

// Shared with the GEMM entry points (api.cu).
int check_current_device(int *sms);             // MXFP4_OK, _ERR_ARCH or _ERR_CUDA
long long current_wait_limit();
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode_fn();

constexpr int kMaxGroups = 1024;                // experts of one call
constexpr int kMaxTopK = 16;

// Grouped scale layout: group e's rows start a 128-row block of their own,
// block offsets[e] / 128 + e.  Blocks never overlap: with o = 128 a + r and
// o' = 128 b + s the next offset, the group takes at most
// ceil((o' - o) / 128) <= b - a + 1 blocks, and the next group starts b - a + 1
// blocks on.  So no prefix sum over the groups is needed to find a block, and
// floor(rows / 128) + groups blocks hold them all.
__host__ __device__ inline int64_t group_sf_block(int offset, int e) { return offset / kSfRowBlock + e; }
inline int64_t group_sf_blocks(int rows, int groups) { return static_cast<int64_t>(rows) / kSfRowBlock + groups; }

// Byte of (row r of a 128-row block, 32-block kb) inside that block's atoms.
__host__ __device__ inline int64_t sf_byte(int r, int kb)
{
    return static_cast<int64_t>(kb >> 2) * kSfAtomBytes + 16 * (r & 31) + 4 * (r >> 5) + (kb & 3);
}

struct RouteArgs {
    const void *logits;         // bf16 or fp32 [T, ldl]
    int64_t ldl;
    int fp32;
    int vec;                    // rows allow loads of four logits
    const uint8_t *mask;        // [T] or null; 0: the token takes no expert
    int T, E, k, mode;
    float gate_scale;
    int *ids;                   // [T, k]
    float *gates;               // [T, k]
    int *offsets;               // [E + 1]
    int *row_token;             // [T k]
    int *slot_row;              // [T, k]
    uint16_t *counts;           // workspace: [blocks][E rounded up to 8]
    int blocks;
    int chunk;                  // tokens per block
};
int route_blocks(int T, int *chunk);
cudaError_t launch_route(const RouteArgs &a, int sms, cudaStream_t stream);

struct GroupQuantArgs {
    uint8_t *Q;
    int64_t ldq_bytes;
    uint8_t *S;
    const uint16_t *X;
    int64_t ldx;
    int T, K, k;
    const int *slot_row;        // [T, k] or null (row t stays row t)
    const int *ids;             // [T, k], with slot_row
    const int *offsets;
    int groups, rows;
    int fmt;                    // 0: packed E2M1, 1: E4M3, 2: E5M2
};
cudaError_t launch_group_quantize(const GroupQuantArgs &a, int sms, cudaStream_t stream);

struct CombineArgs {
    uint16_t *H;                // [T, ldh] or null
    int64_t ldh;
    uint16_t *Nrm;              // [T, ldn] or null
    int64_t ldn;
    const uint16_t *Y;          // [rows, ldy]
    int64_t ldy;
    int rows;
    const int *slot_row;        // [T, k] or null (k = 1, row t)
    const float *gates;         // [T, k] or null (all 1)
    int k;
    const uint16_t *resid;      // [T, ldr] or null
    int64_t ldr;
    const uint16_t *w_post, *w_pre;   // [N] or null
    float res_scale, out_scale, eps;
    int T, N;
    int width;                  // elements of the widest access that every row allows: 8, 4, 2, 1
    long long wait_limit;
    int early;                  // all but Y may be read before the preceding grid ends
};
cudaError_t read_expert_status(int *status, int reset);
cudaError_t launch_combine(const CombineArgs &a, int sms, cudaStream_t stream);

// Arguments of one grouped product (grouped.cu).
struct GroupedArgs {
    const int *offsets;         // [groups + 1], device
    int groups, rows;           // rows: capacity of A and of the output
    int N, K;                   // output columns (F for the gated form), reduction
    int kt;                     // stages of 128 bytes per row
    int nt;                     // column tiles: 256 columns, or 128 of the gated form
    float alpha;
    uint16_t *D;                // plain form: bf16 [rows, ldd]
    int64_t ldd;
    int vec32_ok, vec_ok;       // D (H) allows aligned 32- / 16-byte row stores
    uint8_t *H;                 // gated form: codes [rows, ldh bytes]
    int64_t ldh;
    uint8_t *SH;                // grouped scale layout over N
    // Byte formats, instruction descriptors: M x N = 256 x 256, 128 x 256, 128 x 128.
    uint32_t idesc8, idesc8_solo, idesc8_half;
    int early;                  // offsets, B and its scales may be read before the preceding
                                // grid ends: it is a kernel of the same call, which waited
                                // for the work before the call (one-token block of 3 x 544:
                                // 13.5 us, without 14.9)
    long long wait_limit;
};
struct GroupedMaps {
    CUtensorMap A, A32, SA, B, SB;   // A: boxes of 128 rows, A32: of 32
    CUtensorMap D;                   // plain form with vec_ok: boxes of 32 rows x 32 columns
};
// out: -1 plain (bf16), else the QuantFmt of the gated form's output.
cudaError_t launch_grouped(const GroupedArgs &a, const GroupedMaps &m, bool bytes8, int out, cudaStream_t stream);
cudaError_t read_grouped_status(int *status, int reset);

}  // namespace mxfp4
