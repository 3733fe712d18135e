// Launch of the CUDA-core products with microscaled operands.
#include "mx_simple.cuh"
#include "mx_units.h"

namespace sgemm_gb300 {
namespace units {

cudaError_t mx_simple(const mx::SimpleArgs &a, cudaStream_t s) {
    mx::simple_kernel<<<dim3((unsigned)((a.m + 63) / 64), (unsigned)((a.n + 63) / 64)), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace units
}  // namespace sgemm_gb300
