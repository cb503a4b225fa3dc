// Launching the kernels of a decode step one behind the other.
#pragma once

#include "kda_common.cuh"

// Launches a kernel that begins with kda_grid_wait, so that its blocks are scheduled while the kernel
// ahead of it in the stream ends.
template <typename... Args>
inline cudaError_t kda_launch_chained(void (*kernel)(Args...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                                      const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
