// The launches of the gradients beside a matrix of BITS bits (one translation
// unit for each, compiled in parallel).
#pragma once
#include "mx_grad.cuh"
#include "mx_units.h"

namespace sgemm_gb300 {
namespace units {

template <int BN, int BITS, bool T, bool F32, bool PAIR>
cudaError_t grad_attr() {
    return cudaFuncSetAttribute(mx::grad_kernel<BN, BITS, T, F32, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, mx::g_smem_bytes(BN, PAIR, BITS, F32));
}

template <int BITS>
cudaError_t grad_setup() {
    cudaError_t (*const attrs[])() = {
        grad_attr<16, BITS, false, false, false>, grad_attr<64, BITS, false, false, false>, grad_attr<128, BITS, false, false, false>,
        grad_attr<256, BITS, false, false, true>, grad_attr<16, BITS, false, true, false>,
        grad_attr<64, BITS, false, true, false>,  grad_attr<64, BITS, false, true, true>,   grad_attr<128, BITS, false, true, true>,  grad_attr<64, BITS, true, false, false>,
        grad_attr<128, BITS, true, false, false>, grad_attr<256, BITS, true, false, true>,
        grad_attr<64, BITS, true, true, false>,   grad_attr<128, BITS, true, true, true>};
    for (auto f : attrs)
        if (const cudaError_t e = f()) return e;
    return cudaSuccess;
}

template <int BITS>
cudaError_t grad_launch(const cudaLaunchConfig_t &cfg, const MxPlan &p, bool transposed, bool f32, const CUtensorMap *m, const mx::GradArgs &a) {
    using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, mx::GradArgs);
    Kernel k;
    if (p.bn == 16) k = f32 ? mx::grad_kernel<16, BITS, false, true, false> : mx::grad_kernel<16, BITS, false, false, false>;
    else if (p.bn == 64 && p.pair) k = mx::grad_kernel<64, BITS, false, true, true>;
    else if (p.bn == 64 && !transposed) k = f32 ? mx::grad_kernel<64, BITS, false, true, false> : mx::grad_kernel<64, BITS, false, false, false>;
    else if (p.bn == 64) k = f32 ? mx::grad_kernel<64, BITS, true, true, false> : mx::grad_kernel<64, BITS, true, false, false>;
    else if (p.bn == 128 && !transposed) k = f32 ? mx::grad_kernel<128, BITS, false, true, true> : mx::grad_kernel<128, BITS, false, false, false>;
    else if (p.bn == 128) k = f32 ? mx::grad_kernel<128, BITS, true, true, true> : mx::grad_kernel<128, BITS, true, false, false>;
    else k = transposed ? mx::grad_kernel<256, BITS, true, false, true> : mx::grad_kernel<256, BITS, false, false, true>;
    return cudaLaunchKernelEx(&cfg, k, m[0], m[1], m[2], a);
}

}  // namespace units
}  // namespace sgemm_gb300
