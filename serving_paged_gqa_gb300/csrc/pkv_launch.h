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

// The same on a grid of two dimensions, for a kernel whose beginning may overlap the end of the one before it on the stream
// (programmatic dependent launch): it executes griddepcontrol.wait before it reads or writes what another may write or read.
template <typename... Args>
cudaError_t launch_behind(void (*kernel)(Args...), dim3 grid, dim3 block, int smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pkv
