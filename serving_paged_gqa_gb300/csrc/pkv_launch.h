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

}  // namespace pkv
