// Launches that overlap the end of the kernel in front of them.
#pragma once
#include <cuda_runtime.h>

namespace sgemm_gb300 {
namespace units {

// A launch that may start while the kernel in front of it on the stream ends:
// the kernels so launched wait for that one (griddep_wait) before they read
// or write anything it may touch, so that each is still complete only after
// all in front of it.
template <class Args>
cudaError_t launch_early(void (*kernel)(Args), dim3 grid, int threads, size_t smem, const Args &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace units
}  // namespace sgemm_gb300
