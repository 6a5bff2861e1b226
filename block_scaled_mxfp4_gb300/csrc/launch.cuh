// Launch helpers of the expert-layer and dense-layer kernels.
#pragma once

#include <atomic>
#include <cstddef>
#include <cuda_runtime.h>

namespace mxfp4 {

// Let kernel `Kern` use up to `Bytes` of dynamic shared memory, once per device.  `Bytes` is the most that
// any of its launches asks for, and not a launch's own: host threads that come here at
// once then all set the same limit, so that none takes another's away.
template <auto Kern, int Bytes>
cudaError_t opt_in()
{
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev].load(std::memory_order_relaxed)))
        return e;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Bytes);
    if (e == cudaSuccess && dev < 64)
        done[dev].store(true, std::memory_order_relaxed);
    return e;
}

// Launch as a programmatic dependent of the work before it on the stream: the
// kernel waits for that work (griddepcontrol.wait) before it reads anything.
template <typename Kern, typename... Args>
cudaError_t launch_dependent(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace mxfp4
