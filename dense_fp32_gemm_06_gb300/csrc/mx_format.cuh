// The microscaled format: blocks of 32 values with one power of two.
#pragma once
#include <cstdint>

#include "elem.cuh"

namespace sgemm_gb300 {
namespace mx {

constexpr int BLOCK = 32;
__host__ __device__ __forceinline__ int blocks(int cols) { return cols / BLOCK + (cols % BLOCK != 0); }
__host__ __device__ __forceinline__ constexpr int block_bytes(int bits) { return bits * 4; }

constexpr uint32_t NOT_FINITE = 255;   // the scale byte of a block that holds an infinity or NaN
__host__ __device__ constexpr uint32_t largest_byte(int bits) { return bits == 4 ? 125 + 127 : 121 + 127; }

// The scale byte of a block whose largest magnitude has these FP32 bits.  With
// amax = 1.f 2^(E - 127) and M = 1.5 2^2 (6) or 1.984375 2^6 (127), the least
// power of two that holds it is 2^(E - 127) / 2^2 (2^6), or twice that where
// 1.f is above M's own fraction; byte = exponent + 127.  The largest byte keeps
// a rounded-up magnitude below 2^128.
template <int BITS>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    constexpr int shift = BITS == 4 ? 2 : 6, most = (int)largest_byte(BITS);
    constexpr uint32_t fraction = BITS == 4 ? 0x400000u : 0x7e0000u;
    if (amax >= 0x7f800000u) return NOT_FINITE;
    const int b = (int)(amax >> 23) - shift + ((amax & 0x7fffffu) > fraction);
    return (uint32_t)min(max(b, 0), most);
}

// 2^(127 - byte), which brings a block's values to their codes' range (byte at most 252).
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^(byte - 127); byte 0 is a subnormal, 255 NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == NOT_FINITE ? 0x7fc00000u : byte << 23);
}

// Eight values as 4-bit codes, the first in the low bits: to nearest, ties to
// the even code, magnitudes above 6 to 6 (those occur at the largest scale alone).
__device__ __forceinline__ uint32_t codes4(const float (&f)[8]) {
    uint32_t w;
    asm("{\n"
        ".reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "mov.b32 %0, {a, b, c, d};\n"
        "}\n"
        : "=r"(w)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return w;
}

// Eight values times `inv` as 8-bit codes, the same: 1.5 2^23 + v has the
// rounded v in its low bits.  At the largest scale v may be above 127.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv, bool largest) {
    constexpr float magic = 12582912.f;
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = fmaf(f[i], inv, magic);
    if (largest) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = fminf(fmaxf(c[i], magic - 127.f), magic + 127.f);
    }
    auto four = [&](int i) {
        const uint32_t a = __float_as_uint(c[i]), b = __float_as_uint(c[i + 1]), d = __float_as_uint(c[i + 2]), e = __float_as_uint(c[i + 3]);
        return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(d, e, 0x0040), 0x5410);
    };
    return make_uint2(four(0), four(4));
}

// NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The values of eight 4-bit codes, without their scale.
__device__ __forceinline__ void values4(uint32_t w, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("{\n"
            ".reg .b8 a, b, c, d;\n"
            "mov.b32 {a, b, c, d}, %1;\n"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n"
            "}\n"
            : "=r"(h)
            : "r"(w >> (8 * i)));
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

__device__ __forceinline__ void values8(uint32_t w, float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
}

}  // namespace mx
}  // namespace sgemm_gb300
