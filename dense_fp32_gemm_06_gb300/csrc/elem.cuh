// The element types of the adapter and loss operators: FP32, bfloat16 and
// FP16 values read into and rounded (once, to nearest) from FP32.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace sgemm_gb300 {
namespace elem {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <class T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// One 32-bit word of two 16-bit values (or one FP32 value) as floats.
template <class T> struct Word;
template <> struct Word<float> {
    static constexpr int N = 1;
    static __device__ __forceinline__ void unpack(uint32_t w, float *f) { f[0] = __uint_as_float(w); }
    static __device__ __forceinline__ uint32_t pack(const float *f) { return __float_as_uint(f[0]); }
};
template <> struct Word<__nv_bfloat16> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void unpack(uint32_t w, float *f) {
        f[0] = __uint_as_float(w << 16);   // a bfloat16 is the upper half of its FP32 value
        f[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t pack(const float *f) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[0], f[1]);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <> struct Word<__half> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void unpack(uint32_t w, float *f) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        f[0] = v.x;
        f[1] = v.y;
    }
    static __device__ __forceinline__ uint32_t pack(const float *f) {
        const __half2 v = __floats2half2_rn(f[0], f[1]);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

// The values of a 16-byte vector.
template <class T>
__device__ __forceinline__ void unpack16(const uint4 &w, float *f) {
    constexpr int N = Word<T>::N;
    Word<T>::unpack(w.x, f);
    Word<T>::unpack(w.y, f + N);
    Word<T>::unpack(w.z, f + 2 * N);
    Word<T>::unpack(w.w, f + 3 * N);
}

// Up to four consecutive elements from p on as floats, `n` of which exist (the
// others read as zero), without a branch between loads, so that several stay
// on their way.  VEC: p is aligned to four elements, and four exist or none.
template <class T, bool VEC>
__device__ __forceinline__ float4 fetch4(const T *p, int n) {
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (VEC && sizeof(T) == 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n > 0) v = *reinterpret_cast<const float4 *>(p);
        return v;
    } else if constexpr (VEC) {
        uint2 w = make_uint2(0, 0);
        if (n > 0) w = *reinterpret_cast<const uint2 *>(p);
        Word<T>::unpack(w.x, f);
        Word<T>::unpack(w.y, f + 2);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) f[i] = to_f32(p[i]);
    }
    return make_float4(f[0], f[1], f[2], f[3]);
}

template <class T>
__device__ __forceinline__ void store4(T *p, float4 v, int n, bool vec) {
    const float f[4] = {v.x, v.y, v.z, v.w};
    if (vec && n >= 4) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4 *>(p) = v;
        } else {
            *reinterpret_cast<uint2 *>(p) = make_uint2(Word<T>::pack(f), Word<T>::pack(f + 2));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[i] = from_f32<T>(f[i]);
    }
}

// v as two bfloat16 parts hi + lo, within 2^-16 of it.  What is not finite is
// hi alone (an infinity less itself would be NaN); what is above bfloat16's
// largest value is that and the rest.
__device__ __forceinline__ void parts(float v, __nv_bfloat16 &hi, __nv_bfloat16 &lo) {
    constexpr float top = 3.38953139e38f;   // 0x7f7f
    const bool finite = fabsf(v) < INFINITY;
    hi = __float2bfloat16_rn(finite ? fminf(fmaxf(v, -top), top) : v);
    lo = __float2bfloat16_rn(finite ? v - __bfloat162float(hi) : 0.f);
}

// The parts of eight values, each eight packed.
__device__ __forceinline__ void parts8(const float *v, uint4 &hi, uint4 &lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 a, b;
        parts(v[2 * i], a.x, b.x);
        parts(v[2 * i + 1], a.y, b.y);
        h[i] = *reinterpret_cast<const uint32_t *>(&a);
        l[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// 2^x in the special-function unit (within 2 units in the last place over
// the normal range; -inf gives 0).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// The same with subnormal results: for values that are scaled up afterwards.
__device__ __forceinline__ float exp2_tiny(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace elem
}  // namespace sgemm_gb300
