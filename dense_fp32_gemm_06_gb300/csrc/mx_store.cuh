// Matrices into codes and scales, and back.
#pragma once
#include "mx_format.cuh"

namespace sgemm_gb300 {
namespace mx {

// A matrix that is read: `vec` where its rows start at multiples of 16 bytes.
template <class T>
struct Source {
    const T *x;
    long long ld;
    int rows, cols;
    bool vec;
    __device__ __forceinline__ const T *row(long long r) const { return x + r * ld; }
    __device__ __forceinline__ bool has(const T *p, int n) const { return in_matrix(p, n, x, ld, rows, cols); }
};

struct QuantArgs {
    const void *x;
    long long ldx;        // of the stored matrix
    uint8_t *codes, *scales;
    long long ldc, lds;
    int rows, cols;
    bool vec;             // rows of x start at multiples of 16 bytes
};

template <class T>
__device__ __forceinline__ Source<T> source(const QuantArgs &a) {
    return {static_cast<const T *>(a.x), a.ldx, a.rows, a.cols, a.vec};
}

struct DequantArgs {
    const uint8_t *codes, *scales;
    long long ldc, lds;
    void *y;
    long long ldy;
    int rows, cols;
    bool vec;             // the same of y
};

constexpr int STORE_THREADS = 256;

// A warp's runs of a matrix, `runs` of them a row, taken in turn with a step: the
// place of each from that of the one before it (a division a run was a quarter
// of the quantiser's instructions).
struct Runs {
    long long row, row_step;
    int run, run_step, runs;
    __device__ __forceinline__ Runs(int runs_, int warps) : runs(runs_) {
        const long long u = (long long)blockIdx.x * warps + (threadIdx.x >> 5), step = (long long)gridDim.x * warps;
        row = u / runs;
        run = (int)(u - row * runs);
        row_step = step / runs;
        run_step = (int)(step - row_step * runs);
    }
    __device__ __forceinline__ void next() {
        row += row_step;
        run += run_step;
        if (run >= runs) {
            run -= runs;
            ++row;
        }
    }
};

// Eight consecutive values from column c of a row on; those behind the row are 0.
template <class T>
__device__ __forceinline__ void load8(const Source<T> &m, long long r, int c, float (&f)[8]) {
    const T *row = m.row(r);
    if (m.vec && c <= m.cols - 8 && SG_IN(m.has(row + c, 8))) {
        constexpr int N = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < 8 / N; ++i) elem::unpack16<T>(*reinterpret_cast<const uint4 *>(row + c + i * N), f + i * N);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < m.cols - c && SG_IN(m.has(row + c + i, 1)) ? elem::to_f32(row[c + i]) : 0.f;
    }
}

// 256 values of a row from column c0 on, eight consecutive ones to each lane, by
// way of `lines` (a warp's 256 floats of shared memory): rows that start anywhere
// are read and written a whole warp's run at a time.  Those behind the row are 0
// (load) and left (store).
template <class T>
__device__ __forceinline__ void load_run(const Source<T> &m, long long r, int c0, T (&v)[8]) {
    const int lane = threadIdx.x & 31;
    const T *row = m.row(r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = lane + 32 * i < m.cols - c0 && SG_IN(m.has(row + c0 + lane + 32 * i, 1)) ? row[c0 + lane + 32 * i] : elem::from_f32<T>(0.f);
}
template <class T>
__device__ __forceinline__ void turn_run(const T (&v)[8], float *lines, float (&f)[8]) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) lines[lane + 32 * i] = elem::to_f32(v[i]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<float4 *>(f + 4 * i) = *reinterpret_cast<const float4 *>(lines + lane * 8 + 4 * i);
}
template <class T>
__device__ __forceinline__ void store_run(T *row, int c0, int cols, float *lines, const float (&f)[8]) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<float4 *>(lines + lane * 8 + 4 * i) = *reinterpret_cast<const float4 *>(f + 4 * i);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (lane + 32 * i < cols - c0) row[c0 + lane + 32 * i] = elem::from_f32<T>(lines[lane + 32 * i]);
}

// The largest magnitude's bits of a block's values; NaN's lie above infinity's.
template <int N>
__device__ __forceinline__ uint32_t largest_bits(const float (&f)[N]) {
    float m = fabsf(f[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) m = max_nan(m, fabsf(f[i]));
    return __float_as_uint(m);
}

// Eight values as codes of a block with this scale byte: 4 bits in .x alone.
template <int BITS>
__device__ __forceinline__ uint2 codes_of(const float (&f)[8], uint32_t s) {
    if (s == NOT_FINITE) return make_uint2(0, 0);
    const float inv = inverse_scale(s);
    if constexpr (BITS == 8) {
        return codes8(f, inv, s == largest_byte(8));
    } else {
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = f[i] * inv;
        return make_uint2(codes4(g), 0);
    }
}

// Eight values as they are stored.
template <class T>
struct Raw {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) elem::unpack16<T>(w[i], f + i * 16 / sizeof(T));
    }
};

// Row-major: four lanes a block, eight values each; a warp takes runs of 256 U
// columns of a row.  Aligned rows: a whole run's loads on their way together, and
// the next run's beside this one's arithmetic.  Bound by memory: 8192 x 8192
// bfloat16 values into 8 bits take 31.6 us (6.4 TB/s), into 4 bits 28.2 (6.0); with
// two values' loads together 34.5 and 31.3.
template <class T>
__host__ __device__ constexpr int quant_unroll() { return sizeof(T) == 2 ? 4 : 2; }

template <class T, int BITS>
__device__ __forceinline__ void quantize_eight(const QuantArgs &a, const float (&f)[8], long long row, int c) {
    const int b = c / BLOCK;
    uint32_t m = largest_bits(f);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t s = scale_byte<BITS>(m);
    const uint2 w = codes_of<BITS>(f, s);
    if (b < blocks(a.cols) && SG_IN(row < a.rows && (b + 1ll) * block_bytes(BITS) <= a.ldc && b < a.lds)) {
        uint8_t *codes = a.codes + row * a.ldc + (long long)c * BITS / 8;
        if constexpr (BITS == 4) *reinterpret_cast<uint32_t *>(codes) = w.x;
        else *reinterpret_cast<uint2 *>(codes) = w;
        if ((threadIdx.x & 3) == 0) a.scales[row * a.lds + b] = (uint8_t)s;
    }
}

template <class T, int BITS>
__global__ void __launch_bounds__(STORE_THREADS, 4) quantize_kernel(const QuantArgs a) {
    constexpr int U = quant_unroll<T>();
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int runs = (blocks(a.cols) + 8 * U - 1) / (8 * U), whole = a.cols / (256 * U);   // of a row
    const Source<T> m = source<T>(a);
    Raw<T> next[U];
    auto fetch = [&](const Runs &at) {
        const int c = at.run * (256 * U) + lane * 8;
        if (at.row < a.rows && at.run < whole) {
            const T *x = m.row(at.row) + c;
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (SG_IN(m.has(x + i * 256, 8))) next[i].load(x + i * 256);
        }
    };
    Runs at(runs, STORE_THREADS / 32);
    fetch(at);
    while (at.row < a.rows) {
        const long long row = at.row;
        const int c = at.run * (256 * U) + lane * 8;
        const bool ahead = at.run < whole;
        float f[8];
        Raw<T> now[U];
#pragma unroll
        for (int i = 0; i < U; ++i) now[i] = next[i];
        at.next();
        fetch(at);
        if (ahead) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                now[i].unpack(f);
                quantize_eight<T, BITS>(a, f, row, c + i * 256);
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < U; ++i) {
                load8(m, row, c + i * 256, f);
                quantize_eight<T, BITS>(a, f, row, c + i * 256);
            }
        }
    }
}

// Rows that start anywhere, the next run's loads beside this one's arithmetic as
// well: 8191 x 8191 bfloat16 values into 8 bits 45.9 us, into 4 bits 43.7, FP32 into 8
// bits 52.5 (47.4, 45.0 and 58.9 without; with four values' loads together 54.2 and 52.1).
constexpr int QUANT_ANY_UNROLL = 2;

template <class T, int BITS>
__global__ void __launch_bounds__(STORE_THREADS) quantize_any_kernel(const QuantArgs a) {
    constexpr int U = QUANT_ANY_UNROLL;
    __shared__ __align__(16) float lines[STORE_THREADS / 32][256];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const Source<T> m = source<T>(a);
    T next[U][8];
    auto fetch = [&](const Runs &at) {
        if (at.row >= a.rows) return;
#pragma unroll
        for (int i = 0; i < U; ++i) load_run(m, at.row, at.run * (256 * U) + i * 256, next[i]);
    };
    Runs at((blocks(a.cols) + 8 * U - 1) / (8 * U), STORE_THREADS / 32);
    fetch(at);
    while (at.row < a.rows) {
        const long long row = at.row;
        const int c0 = at.run * (256 * U);
        T v[U][8];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = next[i][j];
        at.next();
        fetch(at);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            __align__(16) float f[8];
            turn_run(v[i], lines[threadIdx.x >> 5], f);
            quantize_eight<T, BITS>(a, f, row, c0 + i * 256 + lane * 8);
        }
    }
}

// X stored cols x rows: a thread takes a whole block of ROWS rows (1, or 2 of 16-bit
// values, whose pairs are then aligned), the lanes of a warp 32 ROWS rows, so that
// its 32 loads are of whole lines; the codes of eight blocks of those rows meet in
// shared memory, so that they leave as whole lines too.  Bound by memory once
// whole blocks are loaded without a test at each load: 8192 x 8192 bfloat16 values
// into 4 bits 30.7 us (5.5 TB/s; with the tests 42.1), into 8 bits 35.2 (46.9), FP32
// 55.2 and 57.7 (69.1 and 63.6); single rows of bfloat16 (8191 x 8190) 40.5 (71.0).
template <class T, int BITS, int ROWS>
__global__ void __launch_bounds__(STORE_THREADS) quantize_t_kernel(const QuantArgs a) {
    static_assert(ROWS == 1 || sizeof(T) == 2, "pairs of 16-bit values");
    constexpr int BYTES = block_bytes(BITS), LINE = 8 * BYTES, PITCH = LINE + 16, TILE = 32 * ROWS;
    __shared__ __align__(16) uint8_t lines[TILE * PITCH];
    __shared__ uint8_t scales[TILE * 8];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nb = blocks(a.cols), segs = (nb + 7) / 8;
    const long long tiles = (long long)(a.rows / TILE + (a.rows % TILE != 0)) * segs;
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const long long r0 = tile / segs * TILE;
        const int b0 = (int)(tile % segs) * 8, b = b0 + warp, mine = lane * ROWS;
        const Source<T> m = {static_cast<const T *>(a.x), a.ldx, a.cols, a.rows, false};   // as stored
        const T *x = m.x + r0 + mine;
        uint32_t raw[BLOCK];
        auto load = [&](const T *at, bool pair) -> uint32_t {
            if (!SG_IN(m.has(at, pair ? ROWS : 1))) return 0;
            if constexpr (sizeof(T) == 4) return __float_as_uint(*at);
            else return ROWS == 2 && pair ? *reinterpret_cast<const uint32_t *>(at) : *reinterpret_cast<const uint16_t *>(at);
        };
        if (b < a.cols / BLOCK && r0 + TILE <= a.rows) {   // a whole block of whole rows: nothing to test at each load
            const T *at = x + (long long)b * BLOCK * a.ldx;
#pragma unroll
            for (int i = 0; i < BLOCK; ++i, at += a.ldx) raw[i] = load(at, true);
        } else {
            const bool both = r0 + mine + ROWS <= a.rows;
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) {
                const long long c = (long long)b * BLOCK + i;
                raw[i] = c < a.cols && r0 + mine < a.rows ? load(x + c * a.ldx, both) : 0;
            }
        }
#pragma unroll
        for (int h = 0; h < ROWS; ++h) {
            float f[BLOCK];
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) f[i] = __uint_as_float(sizeof(T) == 4 ? raw[i] : h == 0 ? raw[i] << 16 : raw[i] & 0xffff0000u);
            const uint32_t s = scale_byte<BITS>(largest_bits(f));
            uint2 *line = reinterpret_cast<uint2 *>(lines + (mine + h) * PITCH + warp * BYTES);
            uint2 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float g[8] = {f[8 * i], f[8 * i + 1], f[8 * i + 2], f[8 * i + 3], f[8 * i + 4], f[8 * i + 5], f[8 * i + 6], f[8 * i + 7]};
                w[i] = codes_of<BITS>(g, s);
            }
            if constexpr (BITS == 4) {
                line[0] = make_uint2(w[0].x, w[1].x);
                line[1] = make_uint2(w[2].x, w[3].x);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) line[i] = w[i];
            }
            scales[(mine + h) * 8 + warp] = (uint8_t)s;
        }
        __syncthreads();
        const int in_line = min(8, nb - b0) * BYTES / 16;   // 16-byte chunks of a row
        for (int q = threadIdx.x; q < TILE * (LINE / 16); q += STORE_THREADS) {
            const int row = q / (LINE / 16), ch = q % (LINE / 16);
            if (ch < in_line && r0 + row < a.rows && SG_IN((long long)b0 * BYTES + (ch + 1) * 16 <= a.ldc))
                *reinterpret_cast<uint4 *>(a.codes + (r0 + row) * a.ldc + (long long)b0 * BYTES + ch * 16) =
                    *reinterpret_cast<const uint4 *>(lines + row * PITCH + ch * 16);
        }
        for (int q = threadIdx.x; q < TILE * 8; q += STORE_THREADS) {
            const int row = q / 8, i = q % 8;
            if (b0 + i < nb && r0 + row < a.rows && SG_IN(b0 + i < a.lds)) a.scales[(r0 + row) * a.lds + b0 + i] = scales[q];
        }
        __syncthreads();
    }
}

// The same way back: 8192 x 8192 values of 8 bits into bfloat16 32.8 us (6.2 TB/s),
// of 4 bits 28.8.
template <class T, int BITS>
__global__ void __launch_bounds__(STORE_THREADS) dequantize_kernel(const DequantArgs a) {
    constexpr int U = quant_unroll<T>();
    __shared__ __align__(16) float lines[STORE_THREADS / 32][256];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31;
    for (Runs at((blocks(a.cols) + 8 * U - 1) / (8 * U), STORE_THREADS / 32); at.row < a.rows; at.next()) {
        const long long row = at.row;
        const int c0 = at.run * (256 * U) + lane * 8;
        const uint8_t *codes = a.codes + row * a.ldc, *scales = a.scales + row * a.lds;
        T *y = static_cast<T *>(a.y) + row * a.ldy;
        uint2 w[U];
        uint32_t byte[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = c0 + i * 256;
            w[i] = make_uint2(0, 0);
            byte[i] = 0;
            if (c < a.cols && SG_IN(c / BLOCK < a.lds && (c / BLOCK + 1ll) * block_bytes(BITS) <= a.ldc)) {
                if constexpr (BITS == 4) w[i].x = *reinterpret_cast<const uint32_t *>(codes + (long long)c / 2);
                else w[i] = *reinterpret_cast<const uint2 *>(codes + c);
                byte[i] = scales[c / BLOCK];
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = c0 + i * 256;
            __align__(16) float f[8];
            if constexpr (BITS == 4) {
                values4(w[i].x, f);
            } else {
                values8(w[i].x, f);
                values8(w[i].y, f + 4);
            }
            const float s = scale_value(byte[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= s;
            if (a.vec && c - lane * 8 <= a.cols - 256) {   // the warp's run: 16 bytes a lane at a time
                const bool in = SG_IN(row < a.rows && c <= a.cols - 8);
                if constexpr (sizeof(T) == 2) {
                    if (in) *reinterpret_cast<uint4 *>(y + c) = make_uint4(elem::Word<T>::pack(f), elem::Word<T>::pack(f + 2), elem::Word<T>::pack(f + 4), elem::Word<T>::pack(f + 6));
                } else {   // by way of shared memory, so that a store's lanes follow one another
                           // (with half a sector a lane 8192 x 8192 took 70.9 us, 57.7 so)
                    float *line = lines[threadIdx.x >> 5];
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 2; ++j) *reinterpret_cast<float4 *>(line + lane * 8 + 4 * j) = *reinterpret_cast<const float4 *>(f + 4 * j);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (in) *reinterpret_cast<float4 *>(y + c - lane * 8 + j * 128 + lane * 4) = *reinterpret_cast<const float4 *>(line + j * 128 + lane * 4);
                }
            } else if (c - lane * 8 < a.cols && SG_IN(row < a.rows)) {
                store_run(y, c - lane * 8, a.cols, lines[threadIdx.x >> 5], f);
            }
        }
    }
}

}  // namespace mx
}  // namespace sgemm_gb300
