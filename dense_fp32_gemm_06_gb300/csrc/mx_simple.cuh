// Products with microscaled operands on the CUDA cores, for any sizes:
// out[p][q] (+)= sum_r A[p][r] B[r][q], 64 x 64 outputs a CTA.
#pragma once
#include "mx_format.cuh"

namespace sgemm_gb300 {
namespace mx {

// An operand as a matrix of rows x cols: real (FP32, bfloat16) or coded, as
// stored or transposed.
struct SimpleOperand {
    const void *p;
    const uint8_t *scales;
    long long ld, lds;
    int kind;          // 0 FP32, 1 bfloat16, 4 or 8 bits
    bool transposed;   // element (i, j) is stored at (j, i)
    __device__ __forceinline__ float at(long long i, long long j) const {
        if (transposed) {
            const long long h = i;
            i = j;
            j = h;
        }
        if (kind == 0) return static_cast<const float *>(p)[i * ld + j];
        if (kind == 1) return elem::to_f32(static_cast<const __nv_bfloat16 *>(p)[i * ld + j]);
        const float s = scale_value(scales[i * lds + j / BLOCK]);
        if (kind == 8) return (float)static_cast<const int8_t *>(p)[i * ld + j] * s;
        float f[8];
        values4(static_cast<const uint8_t *>(p)[i * ld + j / 2] >> (4 * (j & 1)), f);
        return f[0] * s;
    }
};

struct SimpleArgs {
    SimpleOperand a, b;
    void *out;
    long long ld;
    int m, n, k;
    bool bf16, accumulate;
};

static __global__ void __launch_bounds__(256) simple_kernel(const SimpleArgs g) {
    __shared__ float sa[16][65], sb[16][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long m0 = (long long)blockIdx.x * 64, n0 = (long long)blockIdx.y * 64;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < g.k; k0 += 16) {
        for (int q = threadIdx.x; q < 1024; q += 256) {
            const int i = q >> 4, k = q & 15;
            sa[k][i] = m0 + i < g.m && k0 + k < g.k ? g.a.at(m0 + i, k0 + k) : 0.f;
            sb[k][i] = n0 + i < g.n && k0 + k < g.k ? g.b.at(k0 + k, n0 + i) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < 16; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long p = m0 + ty * 4 + i, q = n0 + tx + 16 * j;
            if (p >= g.m || q >= g.n) continue;
            const long long o = p * g.ld + q;
            if (g.bf16) {
                __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(g.out) + o;
                *y = __float2bfloat16_rn(acc[i][j] + (g.accumulate ? elem::to_f32(*y) : 0.f));
            } else {
                float *y = static_cast<float *>(g.out) + o;
                *y = acc[i][j] + (g.accumulate ? *y : 0.f);
            }
        }
}

}  // namespace mx
}  // namespace sgemm_gb300
