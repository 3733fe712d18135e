// Wrappers of the 5th-generation tensor core for 4-bit operands with a scale
// per 32 values (kind::mxf4): MMA issue, the copies of scales from shared to
// tensor memory, and their descriptors.
#pragma once
#include <cstdint>

#include "tcgen05_f16.cuh"

namespace sgemm_gb300 {
namespace tc {

// D[tmem] (+)= A[smem] * B[smem]^T over 64 e2m1 values, each 32 of a row of A
// and of B times 2^(scale - 127), issued by one thread (of the even CTA of a
// PAIR, where A's and B's rows are split between the two).
template <bool PAIR>
__device__ __forceinline__ void mma_mx4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t a_scales,
                                        uint32_t b_scales, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
            "}\n" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n"
            ".reg .pred p;\n"
            "setp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n"
            "}\n" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate)
            : "memory");
}

// Instruction descriptor of kind::mxf4 with e2m1 operands and e8m0 scales:
// [4,6) and [29,31) the first of the two bytes that B's and A's scales take of
// their 32-bit column (0 or 2), [7,10) and [10,12) A and B format (1 = E2M1),
// [17,23) N >> 3, 23 the scales' format (1 = E8M0), [24,29) M >> 4.
__host__ __device__ constexpr uint32_t idesc_mx4(int m, int n, int scale_byte) {
    return (uint32_t(scale_byte) << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (1u << 23) | (uint32_t(m >> 4) << 24) |
           (uint32_t(scale_byte) << 29);
}

// 32 lines of 16 bytes from shared memory (512 contiguous bytes) into four
// columns of tensor memory, the same 32 lanes in each quarter of it: the
// scales of 128 rows, row 32 c + l at lane l, column c.  In the order of the
// issuing thread's MMAs.  PAIR: of both CTAs, each from its own shared memory.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(tmem), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(tmem), "l"(desc) : "memory");
}

// Its source: no swizzle, groups of 8 lines 128 bytes apart.
__device__ __forceinline__ uint64_t desc_scales(uint32_t smem_addr) {
    uint64_t d = (uint64_t)((smem_addr >> 4) & 0x3FFFu);
    d |= (uint64_t)(128u >> 4) << 16;
    d |= (uint64_t)(128u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    return d;
}

}  // namespace tc
}  // namespace sgemm_gb300
