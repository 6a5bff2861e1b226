// A grouped product that may start before the work ahead of it has ended, behind
// a kernel that lets it start and then keeps it waiting for its rows: what
// happens inside mxfp4_moe_ffn when a step ahead takes long.  Compiled and linked
// to the library by tests/test_gpu_wait_limit.py.
#include "../block_scaled_mxfp4_gb300/csrc/expert_api.cu"
#include "../block_scaled_mxfp4_gb300/csrc/launch.cuh"

__global__ void hold_kernel(long long cycles)
{
    pdl_launch_dependents();
    const long long t0 = clock64();
    while (clock64() - t0 < cycles) {
    }
}

// out: -1 bf16 rows into D, 0 packed codes into D with scales in S.
extern "C" int early_product(void *D, int64_t ldd, void *S, const void *A, int64_t lda, const void *SA, const void *B,
                             int64_t ldb, int64_t stride_b, const void *SB, const int *offsets, int groups, int rows,
                             int N, int K, int out, long long hold_cycles, void *stream)
{
    const Product p{D, ldd, S, A, lda, SA, B, ldb, stride_b, SB, offsets, groups, rows, N, K, 1.0f,
                    false, 0, 0, out, true};
    const int st = check_product(p);
    if (st != MXFP4_OK)
        return st;
    if (hold_cycles > 0)
        hold_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(hold_cycles);
    return run_product(p, static_cast<cudaStream_t>(stream));
}
