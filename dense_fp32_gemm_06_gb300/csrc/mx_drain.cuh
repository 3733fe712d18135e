// What the tensor-core products with microscaled operands share: the output's
// tile, 128 features (the MMA's M, the tensor memory's lanes) by BN rows (its
// N, the columns), out of tensor memory and into rows of consecutive features.
#pragma once
#include "mx_format.cuh"
#include "raster.cuh"
#include "tcgen05_f16.cuh"

namespace sgemm_gb300 {
namespace mx {

constexpr int TC_M = 128;

struct Out {
    void *y;
    long long ldy;
    int rows, cols;     // of Y
    bool accumulate;
};

// mbar_arrive_cluster without its fence at cluster scope, which takes 1000 to
// 2000 cycles: for a thread whose writes before it are to its own CTA's shared
// memory, and have been made visible to the async proxy (fence_proxy_async_smem)
// that alone reads them there, or are to its tensor memory, as its reads may be
// (tcgen05 fences order those with the MMA).
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(bar_cluster) : "memory");
}

// The same lane of a whole warp each time.  The warp that issues MMAs and
// copies runs its loops as a whole and elects the issuing lane around each
// batch, so that descriptors and addresses stay in uniform registers: from a loop
// of one lane a scaled MMA or copy took ~100 cycles to issue, where an MMA of 256
// columns takes 128.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "elect.sync _|p, 0xffffffff;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(p));
    return p != 0;
}

template <class T>
__device__ __forceinline__ float before(const Out &o, long long row, int f) {
    return o.accumulate && row < o.rows && f < o.cols && SG_IN(row >= 0 && f >= 0 && f < o.ldy) ? elem::to_f32(static_cast<const T *>(o.y)[row * o.ldy + f]) : 0.f;
}

// A lane's NC rows of feature f from row t0 on, as pairs of bfloat16 values.
// The lane that has feature f ^ 1 is lane ^ SWAP; the two swap halves, so that
// each stores two features of every second row.
template <int NC, int SWAP>
__device__ __forceinline__ void store_tile(const Out &o, const uint32_t (&p)[NC / 2], long long t0, int f) {
    const long long rows = o.rows - t0;
    __nv_bfloat16 *const y = static_cast<__nv_bfloat16 *>(o.y);
    const bool odd = f & 1;
    // every feature of the warp exists and pairs of them are aligned
    if ((f | 31) < o.cols && o.ldy % 2 == 0 && (reinterpret_cast<uintptr_t>(y) & 3) == 0) {
        __nv_bfloat16 *at = y + (t0 + odd) * o.ldy + (f & ~1);
#pragma unroll
        for (int j = 0; j < NC; j += 2) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, p[j / 2], SWAP);
            const uint32_t v = odd ? __byte_perm(got, p[j / 2], 0x7632) : __byte_perm(p[j / 2], got, 0x5410);
            if (j + odd < rows && SG_IN(t0 + j + odd < o.rows && f < o.cols)) *reinterpret_cast<uint32_t *>(at) = v;
            at += 2 * o.ldy;
        }
    } else if (f < o.cols) {
        __nv_bfloat16 *at = y + t0 * o.ldy + f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const uint32_t v = j & 1 ? p[j / 2] >> 16 : p[j / 2];
            if (j < rows && SG_IN(t0 + j < o.rows)) *at = __ushort_as_bfloat16((unsigned short)v);
            at += o.ldy;
        }
    }
}

template <int NC>
__device__ __forceinline__ void store_tile(const Out &o, const float (&v)[NC], long long t0, int f) {
    const long long rows = o.rows - t0;
    if (f >= o.cols) return;
    float *at = static_cast<float *>(o.y) + t0 * o.ldy + f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        if (j < rows && SG_IN(t0 + j < o.rows)) *at = v[j];
        at += o.ldy;
    }
}

// NC columns of this warp's quarter of the tensor memory, up to MOST at a time.
template <int NC, int MOST, class F>
__device__ __forceinline__ void read_columns(uint32_t at, F &&use) {
    constexpr int STEP = NC % 32 == 0 && MOST >= 32 ? 32 : NC % 16 == 0 && MOST >= 16 ? 16 : 8;
    static_assert(NC % STEP == 0, "columns");
#pragma unroll
    for (int c = 0; c < NC; c += STEP) {
        uint32_t v[STEP];
        if constexpr (STEP == 8) tc::ld_32x32b_x8(at + c, v);
        else if constexpr (STEP == 16) tc::ld_32x32b_x16(at + c, v);
        else tc::ld_32x32b_x32(at + c, v);
        tc::wait_ld();
#pragma unroll
        for (int j = 0; j < STEP; ++j) use(c + j, __uint_as_float(v[j]));
    }
}

// The tensor core truncates its sum once per MMA, a loss that grows with the
// contraction: bfloat16 gradients of 262144 tokens (16384 MMAs), all of one sign,
// were 0.14 % too small in the mean, those of 2^20 0.6 %, where bfloat16 rounds by
// up to 0.39 %.  So no accumulator takes more than this many: less than 2^-12 of
// its sum is lost, and of random signs' 8192 tokens (512 MMAs) 0.1 % of the results
// round the other way.
constexpr int MOST_MMAS = 1024;

// Floats of `sums` that the CTAs of such a launch need.
__host__ __device__ constexpr size_t sums_of(long long ctas, int bn) { return (size_t)ctas * bn * TC_M; }

// A draining warp's part of a tile: NC columns (rows of Y from t0 on) of its
// 32 lanes (feature f of this lane), in `segs` accumulators that it acquires
// and releases one after the other (FP32: their sum; else one).  Into Y, or
// (split) as floats into `stage`, where this lane's feature of row j is at
// j * TC_M.  The accumulators are released before the stores: the next tile's
// MMAs start while this one's are on their way.  ADDS: what Y holds may count.
template <int NC, bool F32, int SWAP, bool ADDS, class Acquire, class Release>
__device__ __forceinline__ bool drain(const Out &o, int segs, bool split, float *stage, long long t0, int f, Acquire &&acquire, Release &&release) {
    uint32_t at;
    if constexpr (F32) {
        // 64 sums leave registers for 8 more columns (with 32, sums were spilt: gradients
        // of 2048^3 42.4 us, 39.9 so, the weights' of 256 tokens 31.3 and 24.8)
        float v[NC];
#pragma unroll
        for (int j = 0; j < NC; ++j) v[j] = 0.f;
        for (int i = 0; i < segs; ++i) {
            if (!acquire(at)) return false;
            read_columns<NC, NC >= 64 ? 8 : 32>(at, [&](int j, float x) { v[j] += x; });
            release();
        }
        if (split) {
#pragma unroll
            for (int j = 0; j < NC; ++j) stage[j * TC_M] = v[j];
            return true;
        }
        if (ADDS && o.accumulate)
#pragma unroll
            for (int j = 0; j < NC; ++j) v[j] += before<float>(o, t0 + j, f);
        store_tile<NC>(o, v, t0, f);
    } else {
        if (!acquire(at)) return false;
        if (split) {
            read_columns<NC, 32>(at, [&](int j, float x) { stage[j * TC_M] = x; });
            release();
            return true;
        }
        uint32_t p[NC / 2];
        float even = 0.f;
        read_columns<NC, 32>(at, [&](int j, float x) {
            if (ADDS && o.accumulate) x += before<__nv_bfloat16>(o, t0 + j, f);
            if (j % 2 == 0) {
                even = x;
            } else {
                const float pair[2] = {even, x};
                p[j / 2] = elem::Word<__nv_bfloat16>::pack(pair);
            }
        });
        release();
        store_tile<NC, SWAP>(o, p, t0, f);
    }
    return true;
}

// The same of bfloat16 results whose sum is of several accumulators: kept in `sums`,
// this lane's part of row j at j * TC_M.  Such calls take milliseconds: values are
// stored one by one.  (As a branch of drain it cost registers there: 512 x 4096 x 4096
// in 8 bits 20.8 us, 21.8 so.)
template <int NC, bool ADDS, class Acquire, class Release>
__device__ __forceinline__ bool drain_deep(const Out &o, int segs, bool split, float *stage, float *sums, long long t0, int f, Acquire &&acquire, Release &&release) {
#pragma unroll 1
    for (int i = 0; i < segs; ++i) {
        uint32_t at;
        if (!acquire(at)) return false;
#pragma unroll 1
        for (int c = 0; c < NC; c += 8) {
            float *const part = sums + c * TC_M;
            uint32_t v[8];
            float x[8];
            __syncwarp();
            tc::ld_32x32b_x8(at + c, v);
            tc::wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = i > 0 ? part[j * TC_M] + __uint_as_float(v[j]) : __uint_as_float(v[j]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const long long row = t0 + c + j;
                if (i < segs - 1) {
                    part[j * TC_M] = x[j];
                } else if (split) {
                    stage[(c + j) * TC_M] = x[j];
                } else if (row < o.rows && f < o.cols && SG_IN(row >= 0 && f >= 0 && f < o.ldy)) {
                    if (ADDS) x[j] += before<__nv_bfloat16>(o, row, f);
                    static_cast<__nv_bfloat16 *>(o.y)[row * o.ldy + f] = elem::from_f32<__nv_bfloat16>(x[j]);
                }
            }
        }
        release();
    }
    return true;
}

// The accumulators of a cluster's CTAs, which lie as [row][TC_M] floats at
// `stage` in each, added in rank order: each CTA writes every nsplit-th row.
// All threads of the cluster.
template <class T, int THREADS>
__device__ __forceinline__ void join_split(const Out &o, uint32_t stage, int bn, long long t0, int f0, int rank, int nsplit) {
    tc::cluster_sync();
    const int rows = (int)min((long long)bn, o.rows - t0);
    T *const y = static_cast<T *>(o.y);
    const bool vec = (reinterpret_cast<uintptr_t>(y) & (4 * sizeof(T) - 1)) == 0 && o.ldy % 4 == 0;
    for (int q = threadIdx.x;; q += THREADS) {
        const int row = rank + (q >> 5) * nsplit, f = (q & 31) * 4;
        if (row >= rows) break;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t at = stage + (uint32_t)(row * TC_M + f) * 4;
        float4 u[8];   // their loads on their way together
#pragma unroll
        for (int p = 0; p < 8; ++p)
            if (p < nsplit) u[p] = tc::ld_cluster_v4(tc::map_shared_rank(at, (uint32_t)p));
#pragma unroll
        for (int p = 0; p < 8; ++p)
            if (p < nsplit) {
                v.x += u[p].x;
                v.y += u[p].y;
                v.z += u[p].z;
                v.w += u[p].w;
            }
        if (f0 + f >= o.cols) continue;
        v.x += before<T>(o, t0 + row, f0 + f);
        v.y += before<T>(o, t0 + row, f0 + f + 1);
        v.z += before<T>(o, t0 + row, f0 + f + 2);
        v.w += before<T>(o, t0 + row, f0 + f + 3);
        if (SG_IN(t0 + row < o.rows)) elem::store4(y + (t0 + row) * o.ldy + f0 + f, v, o.cols - f0 - f, vec);
    }
    // no CTA leaves while another reads its shared memory
    __syncwarp();
    tc::cluster_arrive_relaxed();
    tc::cluster_wait();
}

}  // namespace mx
}  // namespace sgemm_gb300
