// Internal launchers of the dense layer's operators: checkpoints in 8 bits, the
// activation's backward pass, layer norm and its gradients.  Arguments are
// checked in dense_api.cu; the ABI is in include/mxfp4_gemm.h.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace mxfp4 {

// One output of the transposing quantiser: codes (one per byte) and scales, both
// row-major; codes null: not wanted.
struct CodesOut {
    uint8_t *q;
    int64_t ldq;
    uint8_t *s;
    int64_t lds;
    int fmt;                    // 0: E4M3, 1: E5M2
};

struct CheckpointArgs {
    CodesOut by_row;            // [rows, cols], blocks along the row
    CodesOut by_col;            // [cols, rows], blocks along the column
    CodesOut act_by_col;        // backward: act(z), [cols, rows]
    uint16_t *dz;               // backward: bf16 [rows, lddz] or null
    int64_t lddz;
    float *sums;                // [cols] or null
    float *partials;            // [strips][cols], where strips > 1 and sums
    const uint16_t *x;          // bf16 [rows, ldx]: the rows, or dh
    int64_t ldx;
    const uint8_t *z, *sz;      // backward: 8-bit checkpoint of z
    int64_t ldz, ld_sz;
    int fmt_z;
    int rows, cols;
    int64_t strips, across;     // blocks below one another and side by side (checkpoint_shape)
    int steps;                  // tiles of a block
    int act;
    int vec_dz;                 // dz's rows allow 16-byte stores
    int wide_q, wide_qt;        // rows allow 32-byte stores (set at launch)
    long long wait_limit;
};
// A call's tiles, from rows and cols alone, so that the sums' order is too.
void checkpoint_shape(CheckpointArgs &a, bool backward);
// x in boxes of 64 columns x 128 rows, 128-byte swizzle.
cudaError_t launch_checkpoint(CheckpointArgs &a, const CUtensorMap &x, cudaStream_t stream);
// The backward pass's arrays, all in boxes of 64 x 64 with a 64-byte swizzle but x, whose is of 128
// bytes (those of an output that is not wanted: zeros).
struct BackwardMaps {
    CUtensorMap x, z, by_row, by_col, act_by_col;
};
cudaError_t launch_act_backward(const CheckpointArgs &a, const BackwardMaps &maps, cudaStream_t stream);
cudaError_t read_checkpoint_status(int *status, int reset);

// a[c] and b[c]: sums over the strips of partials[strip][na + nb], in a fixed order; zeros for
// no strips.  Either array may be null.
cudaError_t launch_sum_partials(float *a, int64_t na, float *b, int64_t nb, const float *partials, int strips, cudaStream_t stream);

struct NormArgs {
    const uint16_t *x;          // bf16 [T, ldx]
    int64_t ldx;
    const void *w, *b;          // [N] or null, bf16 or fp32
    int fp32;                   // type of w and b
    uint16_t *y;                // forward: bf16 [T, ldy]
    int64_t ldy;
    float *mean, *rstd;         // forward: [T] or null; backward: inputs
    float eps;
    const uint16_t *dy;         // backward
    int64_t lddy;
    const uint16_t *dres;       // backward: [T, ldr] or null
    int64_t ldr;
    uint16_t *dx;               // backward
    int64_t lddx;
    float *dw, *db;             // backward: [N], either may be null
    float *partials;            // backward: [blocks][2][N]
    int blocks;                 // backward: blocks that share the rows (at most, until it is launched)
    int T, N;
    int width;                  // elements of the widest access that every row allows (forward: and every
                                // parameter): 8, 4, 2, 1
    int single_w;               // backward: w does not allow accesses of that many
    long long wait_limit;
};
cudaError_t launch_layer_norm(const NormArgs &a, int sms, cudaStream_t stream);
int norm_backward_blocks(int T, int N);              // at most, by the sizes
cudaError_t launch_layer_norm_backward(NormArgs &a, cudaStream_t stream);
cudaError_t read_norm_status(int *status, int reset);

}  // namespace mxfp4
