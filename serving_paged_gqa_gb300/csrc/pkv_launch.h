// Kernel launches that report their own error (and not one that an earlier call left behind).
#pragma once

#include <cuda_runtime.h>

namespace pkv {

template <typename... Args>
cudaError_t launch_kernel(void (*kernel)(Args...), int grid, int block, int smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The same on a grid of two dimensions; behind: its prologue may overlap the end of the kernel before it on the stream
// (programmatic dependent launch), which it waits for itself.
template <typename... Args>
cudaError_t launch_behind(void (*kernel)(Args...), dim3 grid, dim3 block, int smem, bool behind, cudaStream_t stream,
                          const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = behind ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pkv
