// Matrices into codes and scales, and back.
#pragma once
#include "mx_format.cuh"

namespace sgemm_gb300 {
namespace mx {

struct QuantArgs {
    const void *x;
    long long ldx;        // of the stored matrix
    uint8_t *codes, *scales;
    long long ldc, lds;
    int rows, cols;
    bool vec;             // rows of x: eight values at a time, 16-byte aligned
};

struct DequantArgs {
    const uint8_t *codes, *scales;
    long long ldc, lds;
    void *y;
    long long ldy;
    int rows, cols;
    bool vec;
};

constexpr int STORE_THREADS = 256;

// Eight consecutive values from column c of a row on; those from `cols` on are 0.
template <class T>
__device__ __forceinline__ void load8(const T *row, int c, int cols, bool vec, float (&f)[8]) {
    if (vec && c <= cols - 8) {
        constexpr int N = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) elem::unpack16<T>(*reinterpret_cast<const uint4 *>(row + c + i * N), f + i * N);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < cols - c ? elem::to_f32(row[c + i]) : 0.f;
    }
}

// The magnitudes' bits: as whole numbers they order as the values do, and NaN lies above infinity.
__device__ __forceinline__ uint32_t largest8(const float (&f)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    return m;
}

// Row-major: four lanes a block, eight values each; a warp takes 256 columns
// of a row.  Bound by memory.
template <class T, int BITS>
__global__ void __launch_bounds__(STORE_THREADS) quantize_kernel(const QuantArgs a) {
    const int lane = threadIdx.x & 31;
    const int nb = blocks(a.cols), segs = (nb + 7) / 8;
    const long long units = (long long)a.rows * segs, step = (long long)gridDim.x * (STORE_THREADS / 32);
    for (long long u = (long long)blockIdx.x * (STORE_THREADS / 32) + (threadIdx.x >> 5); u < units; u += step) {
        const long long row = u / segs;
        const int c = (int)(u - row * segs) * 256 + lane * 8, b = c / BLOCK;
        float f[8];
        load8(static_cast<const T *>(a.x) + row * a.ldx, c, a.cols, a.vec, f);
        uint32_t m = largest8(f);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t s = scale_byte<BITS>(m);
        const float inv = s == NOT_FINITE ? 0.f : inverse_scale(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = s == NOT_FINITE ? 0.f : f[i] * inv;
        if (b >= nb) continue;
        uint8_t *codes = a.codes + row * a.ldc + (long long)c * BITS / 8;
        if (SG_IN(row < a.rows && (b + 1ll) * block_bytes(BITS) <= a.ldc && b < a.lds)) {
            if constexpr (BITS == 4) *reinterpret_cast<uint32_t *>(codes) = codes4(f);
            else *reinterpret_cast<uint2 *>(codes) = make_uint2(codes8(f[0], f[1], f[2], f[3]), codes8(f[4], f[5], f[6], f[7]));
            if ((lane & 3) == 0) a.scales[row * a.lds + b] = (uint8_t)s;
        }
    }
}

// X stored cols x rows: a thread takes a whole block, the lanes of a warp 32
// rows, so that its 32 loads are of whole lines; the codes of eight blocks of
// those rows meet in shared memory, so that they leave as whole lines too.
template <class T, int BITS>
__global__ void __launch_bounds__(STORE_THREADS) quantize_t_kernel(const QuantArgs a) {
    constexpr int BYTES = block_bytes(BITS), LINE = 8 * BYTES, PITCH = LINE + 16;
    __shared__ __align__(16) uint8_t lines[32 * PITCH];
    __shared__ uint8_t scales[32 * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nb = blocks(a.cols), segs = (nb + 7) / 8;
    const long long tiles = (long long)((a.rows + 31) / 32) * segs;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const long long r0 = tile / segs * 32;
        const int b0 = (int)(tile % segs) * 8, b = b0 + warp;
        const T *x = static_cast<const T *>(a.x) + r0 + lane;
        float f[BLOCK];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < BLOCK; ++i) {
            const long long c = (long long)b * BLOCK + i;
            f[i] = r0 + lane < a.rows && c < a.cols ? elem::to_f32(x[c * a.ldx]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < BLOCK; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
        const uint32_t s = scale_byte<BITS>(m);
        const float inv = s == NOT_FINITE ? 0.f : inverse_scale(s);
#pragma unroll
        for (int i = 0; i < BLOCK; ++i) f[i] = s == NOT_FINITE ? 0.f : f[i] * inv;
        uint4 *line = reinterpret_cast<uint4 *>(lines + lane * PITCH + warp * BYTES);
        if constexpr (BITS == 4) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float g[8] = {f[8 * i], f[8 * i + 1], f[8 * i + 2], f[8 * i + 3], f[8 * i + 4], f[8 * i + 5], f[8 * i + 6], f[8 * i + 7]};
                w[i] = codes4(g);
            }
            *line = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = codes8(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
            line[0] = make_uint4(w[0], w[1], w[2], w[3]);
            line[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        scales[lane * 8 + warp] = (uint8_t)s;
        __syncthreads();
        const int in_line = min(8, nb - b0) * BYTES / 16;   // 16-byte chunks of a row
        for (int q = threadIdx.x; q < 32 * (LINE / 16); q += STORE_THREADS) {
            const int row = q / (LINE / 16), ch = q % (LINE / 16);
            if (ch < in_line && r0 + row < a.rows && SG_IN((long long)b0 * BYTES + (ch + 1) * 16 <= a.ldc))
                *reinterpret_cast<uint4 *>(a.codes + (r0 + row) * a.ldc + (long long)b0 * BYTES + ch * 16) =
                    *reinterpret_cast<const uint4 *>(lines + row * PITCH + ch * 16);
        }
        const int row = threadIdx.x / 8, i = threadIdx.x % 8;
        if (b0 + i < nb && r0 + row < a.rows && SG_IN(b0 + i < a.lds)) a.scales[(r0 + row) * a.lds + b0 + i] = scales[row * 8 + i];
        __syncthreads();
    }
}

template <class T, int BITS>
__global__ void __launch_bounds__(STORE_THREADS) dequantize_kernel(const DequantArgs a) {
    const int lane = threadIdx.x & 31;
    const int segs = (blocks(a.cols) + 7) / 8;
    const long long units = (long long)a.rows * segs, step = (long long)gridDim.x * (STORE_THREADS / 32);
    for (long long u = (long long)blockIdx.x * (STORE_THREADS / 32) + (threadIdx.x >> 5); u < units; u += step) {
        const long long row = u / segs;
        const int c = (int)(u - row * segs) * 256 + lane * 8;
        if (c >= a.cols) continue;
        const uint8_t *codes = a.codes + row * a.ldc + (long long)c * BITS / 8;
        float f[8];
        if constexpr (BITS == 4) {
            values4(*reinterpret_cast<const uint32_t *>(codes), f);
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(codes);
            values8(w.x, f);
            values8(w.y, f + 4);
        }
        const float s = scale_value(a.scales[row * a.lds + c / BLOCK]);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= s;
        T *y = static_cast<T *>(a.y) + row * a.ldy + c;
        if (!SG_IN(row < a.rows && c < a.cols)) continue;
        elem::store4(y, make_float4(f[0], f[1], f[2], f[3]), a.cols - c, a.vec);
        elem::store4(y + 4, make_float4(f[4], f[5], f[6], f[7]), a.cols - c - 4, a.vec);
    }
}

}  // namespace mx
}  // namespace sgemm_gb300
