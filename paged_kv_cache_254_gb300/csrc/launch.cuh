// A kernel launch that answers with its own status.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace pa {

// <<<grid, threads, smem, stream>>> with the launch's status.  cudaGetLastError()
// after a launch would also report an error that an earlier call of the thread left
// behind, for a kernel that did start.
template <class... Params, class... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace pa
