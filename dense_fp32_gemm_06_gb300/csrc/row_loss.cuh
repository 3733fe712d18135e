// Losses over rows of logits with their gradients by the logits: distillation
// from a teacher's top logits, and the clipped policy loss with a KL term.
//
// Mathematics.  Both need, per row z of V logits (divided by the temperature,
// 1 for the policy loss), only M = max z, S = sum exp((z - M) / tau) and the
// logits at a few named places; the gradient is then
//     distill:  tau w (p_v - q_v)          policy:  d (1[v = label] - p_v)
// with p_v = exp((z_v - M) / tau) / S, q the teacher's softmax over its
// usable places (zero elsewhere) and d the loss's derivative by
// lp = (z_label - M) / tau - ln S.  Exponentials are powers of two of
// z c - M c, c = log2 e / tau, one FMA each: the rounding of M c is the same
// in every term and in S, so it leaves the quotients.  Past |M c| = 2^24 that
// rounding alone could overflow the power (a row of the type's lowest value):
// such a row is summed again with the difference first, (z - M) c.
//
// What bounds it.  The row has to come from memory once and its gradient go
// back once: 2 V sizeof(T) bytes, against two exponentials (16 a cycle and
// SM) and ~4 other instructions per element and pass, which for 16-bit types
// is within a factor of 1.4 of the memory's time.  So a row is read once into
// registers by a cluster of 1 to 8 CTAs (NV 16-byte vectors per thread), the
// CTAs exchange one (M, S) pair through distributed shared memory, and the
// gradient is written from the registers; several small CTAs per SM keep
// loads in flight while others reduce or write, and pairs of elements go
// through packed FP32 instructions.  Rows longer than a cluster's registers
// are read a second time (CACHED = false).
//
// Rows start at any element: the vectors lie on the row's own 16-byte
// boundaries, the up to 2 (VE - 1) elements in front of and behind them go
// one each to the first threads of the cluster's first CTA.
//
// One GB300's times: policy 4096 x 131072 bfloat16 335 us (6.4 TB/s of the
// bytes it needs, a plain copy moves 6.8), 1000 x 50021 FP32 68 (5.8 TB/s; a
// row's parts end unevenly); distill 4096 x 32768 bfloat16 110 (4.9 TB/s:
// barriers around the keeper of the places).  Short batches are bound by the
// launch: policy 32 x 32768 4.0.
#pragma once
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "elem.cuh"
#include "tcgen05.cuh"

namespace sgemm_gb300 {
namespace rowloss {

constexpr int MAX_TOP = 1024;
constexpr int MAX_CLUSTER = 8;

enum Kind { DISTILL = 0, POLICY = 1 };

struct Args {
    const void *z;
    void *grad;          // NULL: none; may be z
    long long ldz, ldg;  // in elements
    int t, v;
    float c;             // log2(e) / tau
    const float *weight; // NULL: 1
    float *loss;
    // distill
    const float *teacher;
    const int *index;
    int top;
    float tau;
    // policy
    const int *label;
    const float *old_logp, *adv, *ref;
    float clip_low, clip_high, kl;
    float *logp;
};

// The statistics of a part of a row: its maximum m and s, the sum of
// exp2(z c - m c).  A part without a logit above -inf has m = -inf, s = 0.
struct Stat {
    float m, s;
};

// m c as every power is taken against it: a product that is rounded, and not
// contracted with the sum it goes into.
__device__ __forceinline__ float scaled(float m, float c) { return __fmul_rn(m, c); }

__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, a.s + b.s};   // both sums are 0, or NaN
    // the powers' arguments are differences of the rounded m c, as the sums' are
    // (contracted into one FMA they left each part's sum off by the rounding of
    // its m c, up to a factor of 2^(2^-7) at an offset of 1e5)
    const float sa = a.m == m ? a.s : a.s * elem::exp2_fast(scaled(a.m, c) - scaled(m, c));
    const float sb = b.m == m ? b.s : b.s * elem::exp2_fast(scaled(b.m, c) - scaled(m, c));
    return {m, sa + sb};
}

constexpr float WIDE_FROM = 16777216.f;   // 2^24

// The maximum that a part's powers are taken against: 0 for one so low that
// every power is 0 beside any row that is not summed again.
__device__ __forceinline__ float against(float m, float c) { return m * c < -WIDE_FROM ? 0.f : m; }

__device__ __forceinline__ uint4 ld_once(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_cluster_v2(uint32_t addr, float a, float b) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};\n" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

// Pairs of FP32 values in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n.reg .b64 a, b, c, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
        "fma.rn.f32x2 d, a, b, c;\nmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmul.rn.f32x2 d, a, b;\nmov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The pairs of a 16-byte vector: 2 of FP32, 4 of 16-bit values.
template <class T>
__device__ __forceinline__ void unpack16(const uint4 &w, float2 *f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 4) {
        f[0] = make_float2(__uint_as_float(u[0]), __uint_as_float(u[1]));
        f[1] = make_float2(__uint_as_float(u[2]), __uint_as_float(u[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[2];
            elem::Word<T>::unpack(u[i], x);
            f[i] = make_float2(x[0], x[1]);
        }
    }
}

template <class T>
__device__ __forceinline__ uint4 pack16(const float2 *f) {
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x[2] = {f[i].x, f[i].y};
            u[i] = elem::Word<T>::pack(x);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// The largest element of a vector (NaN only where all are).
template <class T>
__device__ __forceinline__ float max16(const uint4 &w) {
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)), fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
    } else if constexpr (std::is_same<T, __half>::value) {
        const __half2 *h = reinterpret_cast<const __half2 *>(&w);
        const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&w);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
}

// sum of exp2(z c - mc) over a vector, or with the difference first.
template <class T, bool WIDE>
__device__ __forceinline__ float2 sum16(const uint4 &w, float c, float m, float2 s) {
    constexpr int P = 8 / sizeof(T);
    float2 f[P];
    unpack16<T>(w, f);
    const float2 c2 = make_float2(c, c), n2 = make_float2(-scaled(m, c), -scaled(m, c));
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float2 x = WIDE ? make_float2((f[i].x - m) * c, (f[i].y - m) * c) : fma2(f[i], c2, n2);
        s = add2(s, make_float2(elem::exp2_fast(x.x), elem::exp2_fast(x.y)));
    }
    return s;
}

// What turns a logit into its gradient off the named places: k exp2(z c - mc).
// (k in the exponent, as log2|k| - mc, would bring a rounding that S has not:
// 4 % of the result at |mc| of 1e6.)  FP32 rows keep powers below 2^-126, 16-bit
// ones do not need them while k is at most FAST_K; with a larger k they take the
// wide form, k exp2((z - m) c), which keeps them.
constexpr float FAST_K = 2.f;
struct Slope {
    float c, m, k;
};

__device__ __forceinline__ float slope_at(float z, const Slope &q, bool wide) {
    return elem::exp2_tiny(wide ? (z - q.m) * q.c : fmaf(z, q.c, -scaled(q.m, q.c))) * q.k;
}

template <class T, bool WIDE>
__device__ __forceinline__ uint4 give16(const uint4 &w, const Slope &q) {
    constexpr int P = 8 / sizeof(T);
    float2 f[P];
    unpack16<T>(w, f);
    [[maybe_unused]] const float2 c2 = make_float2(q.c, q.c), k2 = make_float2(q.k, q.k),
                                  n2 = make_float2(-scaled(q.m, q.c), -scaled(q.m, q.c));
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if constexpr (WIDE) {
            f[i] = make_float2(slope_at(f[i].x, q, true), slope_at(f[i].y, q, true));
        } else {
            const float2 x = fma2(f[i], c2, n2);
            f[i] = mul2(sizeof(T) == 4 ? make_float2(elem::exp2_tiny(x.x), elem::exp2_tiny(x.y))
                                       : make_float2(elem::exp2_fast(x.x), elem::exp2_fast(x.y)), k2);
        }
    }
    return pack16<T>(f);
}

template <class T>
__device__ __forceinline__ void put16(T *g, const uint4 &w, bool vec) {
    if (vec) {
        __stcs(reinterpret_cast<uint4 *>(g), w);
    } else {
        constexpr int P = 8 / sizeof(T);
        float2 f[P];
        unpack16<T>(w, f);   // exact: the values are T's
#pragma unroll
        for (int i = 0; i < P; ++i) {
            g[2 * i] = elem::from_f32<T>(f[i].x);
            g[2 * i + 1] = elem::from_f32<T>(f[i].y);
        }
    }
}

// A warp's statistics from its lanes': one maximum, one rescaling, one sum.
__device__ __forceinline__ Stat join_warp(Stat st, float c) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(m) : "f"(st.m));
    float s = st.m == m ? st.s : st.s * elem::exp2_fast(scaled(st.m, c) - scaled(m, c));
    if (st.m == -INFINITY) s = st.s;   // 0, or NaN
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return {m, s};
}

// A bulk copy of `bytes` (a multiple of 16) from global to shared memory, its
// bytes counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

constexpr int kWaitRow = 0x221;

// Eight bytes into a peer's shared memory, counted on the peer's barrier.
__device__ __forceinline__ void send_stat(uint32_t addr, Stat st, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];\n" ::"r"(addr),
                 "f"(st.m), "f"(st.s), "r"(bar)
                 : "memory");
}

constexpr int kWaitPeers = 0x222;

// Where a row's vectors and edges lie, and this CTA's part of them (a row's
// cluster has 2^lg CTAs).
template <class T>
struct Part {
    static constexpr int VE = 16 / sizeof(T);
    const T *z;
    int head, nv, tail, v0, n;   // n vectors from v0 on
    __device__ __forceinline__ Part(const Args &a, long long row, uint32_t rank, int lg) {
        z = static_cast<const T *>(a.z) + row * a.ldz;
        head = (int)((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / (int)sizeof(T);
        if (head > a.v) head = a.v;
        nv = (a.v - head) / VE;
        tail = a.v - head - nv * VE;
        const int per = (nv + (1 << lg) - 1) >> lg;
        v0 = min(nv, (int)rank * per);
        n = min(nv, v0 + per) - v0;
    }
    __device__ __forceinline__ const uint4 *vectors() const { return reinterpret_cast<const uint4 *>(z + head) + v0; }
    // the element that a thread of the first CTA takes beside its vectors, -1: none
    __device__ __forceinline__ int edge(uint32_t rank, int v) const {
        const int tid = threadIdx.x;
        if (rank != 0 || tid >= head + tail) return -1;
        return tid < head ? tid : v - tail + (tid - head);
    }
    // whether an element belongs to this CTA's part
    __device__ __forceinline__ bool mine(int at, uint32_t rank) const {
        const int v = at < head ? -1 : (at - head) / VE;
        return v < 0 || v >= nv ? rank == 0 : v >= v0 && v < v0 + n;
    }
};

// The scalars of a row, loaded two rows ahead.
template <Kind KIND>
struct Ahead {
    float w, old, adv, ref;
    int label;
    __device__ __forceinline__ void load(const Args &a, long long row) {
        w = a.weight ? a.weight[row] : 1.f;
        if constexpr (KIND == POLICY) {
            label = a.label[row];
            if (label >= a.v) label = -1;
            old = a.old_logp[row];
            adv = a.adv[row];
            ref = a.kl != 0.f ? a.ref[row] : 0.f;
        }
    }
    // the row counts for nothing and nothing is asked of it, or it has no label
    __device__ __forceinline__ bool skip(const Args &a) const {
        return (w == 0.f && (KIND == DISTILL || a.logp == nullptr)) || (KIND == POLICY && label < 0);
    }
};

// What warp 0 makes of a row for the others: its maximum and log2 of its sum,
// the gradient's factors, and what the label's place gets (policy).
struct __align__(16) RowOut {
    float m, ls, k;
    float at_label;
    int wide, dead;   // wide: differences first
};

// The named places of a row of distill, kept by the last warp: the index (-1: not
// usable), the student's logit there, q and log2 q, and the q of all places
// that name the index (in the first of them; -1 in the others).
struct Places {
    int *at;
    float *z, *q, *lq, *sum, *raw;
    uint32_t *bits;
    int n;
    __device__ __forceinline__ Places(uint8_t *p, int top) : n((top + 3) & ~3) {
        at = reinterpret_cast<int *>(p);
        z = reinterpret_cast<float *>(at + n);
        q = z + n;
        lq = q + n;
        sum = lq + n;
        raw = sum + n;   // two rows' logits and indexes as stored, the second on its way
        bits = reinterpret_cast<uint32_t *>(raw + 4 * n);   // 4 n words of zeros between rows
    }
    // One of the 128 n bits: two rounds of a multiplication by 2^32 over the
    // golden ratio, so that regular strides of indexes spread too.
    __device__ __forceinline__ uint32_t hash(int i) const {
        uint32_t h = (uint32_t)i * 2654435769u;
        h = (h ^ (h >> 15)) * 2654435769u;
        return __umulhi(h, 128u * (uint32_t)n);
    }
    // Two rows ahead: while the memory is busy a load takes ~3 us.
    __device__ __forceinline__ void fetch(const Args &a, long long row, int half, int lane) const {
        if (row < a.t) {
            float *to = raw + 2 * n * half;
            for (int j = lane; j < a.top; j += 32) {
                cp_async_4(smem_u32(to + j), a.teacher + row * a.top + j, 4);
                cp_async_4(smem_u32(to + n + j), a.index + row * a.top + j, 4);
            }
        }
        cp_async_commit();
    }
    // Looks the fetched values over and (`go`) sets out for the student's
    // logits of the first 64 places; whether any place is usable.  Whole warp.
    template <class T>
    __device__ __forceinline__ bool begin(const Args &a, const T *row, int half, bool go, int lane, T *ahead) const {
        const float *tl = raw + 2 * n * half;
        const int *idx = reinterpret_cast<const int *>(tl + n);
        cp_async_wait<1>();
        __syncwarp();
        bool any = false;
        for (int j = lane; j < a.top; j += 32) {
            const int i = idx[j];
            const bool ok = i >= 0 && i < a.v && !(tl[j] == -INFINITY);
            at[j] = ok ? i : -1;
            any = any || ok;
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int j = lane + 32 * g;
            if (go && j < a.top && at[j] >= 0) ahead[g] = row[at[j]];
        }
        return __any_sync(0xffffffffu, any);
    }
    // The student's logits: those set out for, or out of the row in shared
    // memory (`vec`: its `count` elements from `head` on).
    template <class T>
    __device__ __forceinline__ void land(const Args &a, const T *row, int lane, const T *ahead, const T *vec, int head,
                                         int count) const {
        if (vec != nullptr) {
            for (int j = lane; j < a.top; j += 32) {
                const int i = at[j] - head;
                z[j] = at[j] < 0 ? 0.f : elem::to_f32(i >= 0 && i < count ? vec[i] : row[at[j]]);
            }
            return;
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int j = lane + 32 * g;
            if (j < a.top) z[j] = at[j] >= 0 ? elem::to_f32(ahead[g]) : 0.f;
        }
#pragma unroll 4
        for (int j = lane + 64; j < a.top; j += 32) z[j] = at[j] >= 0 ? elem::to_f32(row[at[j]]) : 0.f;
    }
    // Everything else.  Equal indexes are found by a bit per hashed index (128
    // bits a place): who meets a set bit compares with all places.  Whole warp.
    __device__ __forceinline__ void finish(const Args &a, int half, int lane) const {
        const float *tl = raw + 2 * n * half;
        float m = -INFINITY;
        for (int j = lane; j < a.top; j += 32)
            if (at[j] >= 0) m = fmaxf(m, tl[j]);
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(m) : "f"(m));
        if (m == -INFINITY) m = 0.f;
        float s = 0.f;
        for (int j = lane; j < a.top; j += 32) {
            const float x = (tl[j] - m) * a.c, e = at[j] >= 0 ? elem::exp2_fast(x) : 0.f;
            lq[j] = x;
            q[j] = e;
            s += e;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const float is = 1.f / s, ls = log2f(s);
        for (int j = lane; j < a.top; j += 32) {
            lq[j] -= ls;
            q[j] *= is;
            sum[j] = q[j];
        }
        __syncwarp();
        for (int j0 = 0; j0 < a.top; j0 += 32) {
            const int j = j0 + lane, i = j < a.top ? at[j] : -1;
            const uint32_t h = hash(i);
            const bool met = i >= 0 && (atomicOr(&bits[h >> 5], 1u << (h & 31)) >> (h & 31) & 1) != 0;
            for (uint32_t todo = __ballot_sync(0xffffffffu, met); todo != 0; todo &= todo - 1) {
                const int k = __shfl_sync(0xffffffffu, i, __ffs(todo) - 1);
                // all places of index k, in order: the first takes the sum
                int first = -1;
                float total = 0.f;
                for (int g0 = 0; g0 < a.top; g0 += 32) {
                    const int g = g0 + lane;
                    const bool same = g < a.top && at[g] == k;
                    for (uint32_t in = __ballot_sync(0xffffffffu, same); in != 0; in &= in - 1) {
                        const int f = g0 + __ffs(in) - 1;
                        if (first < 0) first = f;
                        total += q[f];
                    }
                    if (same) sum[g] = -1.f;
                }
                __syncwarp();
                if (lane == 0) sum[first] = total;
                __syncwarp();
            }
        }
        for (int j = lane; j < a.top; j += 32) {
            if (at[j] >= 0) bits[hash(at[j]) >> 5] = 0;
        }
        __syncwarp();
    }
};
__host__ __device__ constexpr int places_bytes(int top) { return 13 * ((top + 3) & ~3) * 4; }

__device__ __forceinline__ void barrier_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void barrier_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// A cluster of 2^lg CTAs takes rows c, c + clusters, c + 2 clusters, ...  The
// first comes straight into registers; every later one is copied into shared
// memory while the row before it is in work, its named places and scalars
// too, so that no memory latency stands between rows.  Per row: every warp
// reduces its part; warp 0 joins them, exchanges with the cluster's other
// CTAs and makes the row's scalars; every warp writes the gradient.  Distill
// leaves its last warp without vectors: it keeps the places, writes them once
// the others have written, then makes the next row's while it is on its way.  (With the
// places shared out over all warps 4096 rows of 32768 bfloat16 logits took
// 133 us, with one warp keeping them beside its vectors 124, so 111.)
template <class T, Kind KIND, int THREADS, int NV, bool CACHED>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) row_loss_kernel(const Args a) {
    constexpr int VE = 16 / sizeof(T);
    constexpr int WARPS = THREADS / 32;
    constexpr int DATA = KIND == DISTILL ? THREADS - 32 : THREADS;   // threads with vectors
    extern __shared__ __align__(128) uint8_t s_dyn[];   // the lists, then DATA * NV vectors (more than one row per cluster)
    __shared__ uint64_t s_bar, s_peers[2];
    __shared__ Stat s_warp[WARPS];
    __shared__ Stat s_cta[2][MAX_CLUSTER];
    __shared__ RowOut s_out;
    __shared__ int s_places;   // distill: whether the row has any

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = tc::cluster_ctarank(), nrank = tc::cluster_nctarank();
    const int lg = __ffs(nrank) - 1;
    const long long clusters = gridDim.x >> lg, first = blockIdx.x >> lg;
    const int V = a.v;
    const float c = a.c;
    const uint32_t bar = smem_u32(&s_bar);
    const Places list(s_dyn, KIND == DISTILL ? a.top : 0);
    uint4 *s_row = reinterpret_cast<uint4 *>(s_dyn + (KIND == DISTILL ? (places_bytes(a.top) + 127) / 128 * 128 : 0));

    const bool keeper = KIND == DISTILL && warp == WARPS - 1;

    griddep_wait();   // this kernel starts while the one in front of it ends
    Ahead<KIND> now, next;
    now.load(a, first);
    T at_places[2];   // keeper: the student's logits at the first places, on their way
    if (keeper) {
        list.fetch(a, first, 0, lane);
        list.fetch(a, first + clusters, 1, lane);
        for (int i = lane; i < 4 * list.n; i += 32) list.bits[i] = 0;
        const bool any = list.begin(a, static_cast<const T *>(a.z) + first * a.ldz, 0, !now.skip(a), lane, at_places);
        if (lane == 0) s_places = any;
        __syncwarp();
        list.finish(a, 0, lane);
    }
    if (first + clusters < a.t) next.load(a, first + clusters);
    if (tid == 0) {
        mbar_init(bar, 1);
        mbar_init(smem_u32(&s_peers[0]), 1);
        mbar_init(smem_u32(&s_peers[1]), 1);
        fence_mbar_init();
    }
    if (nrank > 1) tc::cluster_sync();   // peers' barriers exist
    else __syncthreads();
    uint32_t loads = 0, exchanges = 0;
    bool from_smem = false;
    int half = 0;   // the row's half of the fetched places
    const uint32_t none = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;   // -inf

    for (long long row = first; row < a.t; row += clusters) {
        const Part<T> part(a, row, rank, lg);
        T *g = a.grad ? static_cast<T *>(a.grad) + row * a.ldg : nullptr;
        const int ei = part.edge(rank, V), n = keeper ? 0 : part.n;
        const bool skip = now.skip(a);

        Stat st = {-INFINITY, 0.f};
        uint4 keep[CACHED ? NV : 1];
        float ev = -INFINITY, zl = 0.f;
        if (!skip) {
            // every load of the row in flight before the first is used
            if (CACHED && !from_smem) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int v = i * DATA + tid;
                    keep[i] = make_uint4(none, none, none, none);
                    if (v < n && SG_IN(part.head + (part.v0 + v + 1) * VE <= V)) keep[i] = ld_once(part.vectors() + v);
                }
            }
            if (ei >= 0 && SG_IN(ei < V)) ev = elem::to_f32(part.z[ei]);
            if (KIND == POLICY && warp == 0) zl = elem::to_f32(part.z[now.label]);
        }
        if (CACHED && from_smem) {
            if (!skip) {
                mbar_wait(bar, loads & 1, kWaitRow);
                ++loads;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int v = i * DATA + tid;
                    keep[i] = make_uint4(none, none, none, none);
                    if (v < n) keep[i] = s_row[v];
                }
            }
        }
        const bool was_smem = from_smem;
        const Ahead<KIND> mine = now;
        now = next;
        const bool more = row + clusters < a.t;
        // what comes along with the rows after this one
        if (row + 2 * clusters < a.t) next.load(a, row + 2 * clusters);

        if (keeper) {
            if (!skip)
                list.land(a, part.z, lane, at_places, CACHED && was_smem && nrank == 1 ? reinterpret_cast<const T *>(s_row) : nullptr,
                          part.head, part.n * VE);
            list.fetch(a, row + 2 * clusters, half, lane);
            half ^= 1;
            if (lane == 0) s_warp[warp] = st;
        } else if (!skip) {
            st.m = ev;
            if constexpr (CACHED) {
#pragma unroll
                for (int i = 0; i < NV; ++i) st.m = fmaxf(st.m, max16<T>(keep[i]));
                const float m = against(st.m, c);
                float2 s = make_float2(elem::exp2_fast(fmaf(ev, c, -scaled(m, c))), 0.f);
#pragma unroll
                for (int i = 0; i < NV; ++i) s = sum16<T, false>(keep[i], c, m, s);
                st.s = s.x + s.y;
            } else {
                if (ei >= 0) st.s = elem::exp2_fast(fmaf(ev, c, -scaled(against(ev, c), c)));
                for (int v = tid; v < n; v += DATA) {
                    const uint4 x = SG_IN(part.head + (part.v0 + v + 1) * VE <= V) ? ld_once(part.vectors() + v)
                                                                                   : make_uint4(none, none, none, none);
                    Stat one = {max16<T>(x), 0.f};
                    const float m = against(one.m, c);
                    const float2 s = sum16<T, false>(x, c, m, make_float2(0.f, 0.f));
                    one.s = s.x + s.y;
                    st = join(st, one, c);
                }
            }
            st = join_warp(st, c);
            if (lane == 0) s_warp[warp] = st;
        }
        __syncthreads();   // the warps' statistics; the buffer is free
        from_smem = more;
        if (more) {
            if (CACHED && tid == DATA - 32 && !now.skip(a)) {
                const Part<T> ahead(a, row + clusters, rank, lg);
                const uint32_t bytes = (uint32_t)ahead.n * 16;
                mbar_arrive_expect_tx(bar, bytes);
                if (bytes > 0) {
                    tc::fence_proxy_async_smem();
                    bulk_load(smem_u32(s_row), ahead.vectors(), bytes, bar);
                }
            }
        }
        // warp 0: the row's statistics from the warps', the cluster's from the
        // CTAs'.  A peer's statistics also say that it has read its part and
        // the named places, on which this CTA's gradient may lie.
        auto join_row = [&]() {
            const Stat x = join_warp(lane < WARPS ? s_warp[lane] : Stat{-INFINITY, 0.f}, c);
            if (nrank == 1) return x;
            const int b = exchanges & 1;
            const uint32_t pb = smem_u32(&s_peers[b]);
            if (lane == 0) mbar_arrive_expect_tx(pb, nrank * 8);
            uint32_t zero = __float_as_uint(zl);   // 0 once the label's logit has arrived
            asm volatile("and.b32 %0, %0, 0;\n" : "+r"(zero));
            if (lane < (int)nrank)
                send_stat(tc::map_shared_rank(smem_u32(&s_cta[b][rank]) + zero, lane), x, tc::map_shared_rank(pb, lane));
            mbar_wait_cluster(pb, (exchanges >> 1) & 1, kWaitPeers);
            ++exchanges;
            __syncwarp();
            return join_warp(lane < (int)nrank ? s_cta[b][lane] : Stat{-INFINITY, 0.f}, c);
        };
        auto is_wide = [&](float m) { return fabsf(m * c) > WIDE_FROM && fabsf(m) != INFINITY; };
        // warp 0: everything else that is the row's own
        auto scalars = [&](Stat x) {
            RowOut o = {};
            o.m = x.m;
            o.ls = log2f(x.s);
            o.wide = is_wide(x.m);
            o.dead = skip || (KIND == DISTILL && !s_places) || mine.w == 0.f || (x.m == -INFINITY && x.s == 0.f);
            if constexpr (KIND == POLICY) {
                const bool empty = x.m == -INFINITY && x.s == 0.f;
                const float below = o.wide ? (zl - x.m) * c : fmaf(zl, c, -scaled(x.m, c));   // of base 2
                const float lp = (below - o.ls) * 0.693147180559945309f;
                float loss = 0.f, d = 0.f;
                if (!o.dead) {
                    const float r = expf(lp - mine.old);
                    const float u = r * mine.adv, b = fminf(fmaxf(r, 1.f - a.clip_low), 1.f + a.clip_high) * mine.adv;
                    loss = -fminf(u, b);
                    d = u <= b ? -u : 0.f;
                    // fminf and fmaxf leave out a NaN: of r, of the advantage, or of an infinite r times 0
                    if (r != r || u != u || b != b) loss = d = r + u + b;
                    if (a.kl != 0.f) {
                        const float y = mine.ref - lp, e = expf(y);
                        loss += a.kl * (e - y - 1.f);
                        d += a.kl * (1.f - e);
                    }
                    loss *= mine.w;
                    d *= mine.w;
                }
                if (rank == 0 && lane == 0) {
                    a.loss[row] = loss;
                    if (a.logp) a.logp[row] = skip ? 0.f : empty ? -INFINITY : lp;
                }
                o.k = -d / x.s;
                o.at_label = d - d * (elem::exp2_fast(below) / x.s);
            } else {
                o.k = mine.w * a.tau / x.s;
            }
            if (lane == 0) s_out = o;
        };
        if (warp == 0) scalars(skip ? Stat{-INFINITY, 0.f} : join_row());
        __syncthreads();
        RowOut o = s_out;
        if (o.wide && !skip) {   // (a skipped row's maximum is -inf)
            float2 s = make_float2(ei >= 0 ? elem::exp2_fast((ev - o.m) * c) : 0.f, 0.f);
            if constexpr (CACHED) {
#pragma unroll
                for (int i = 0; i < NV; ++i) s = sum16<T, true>(keep[i], c, o.m, s);
            } else {
                for (int v = tid; v < n; v += DATA)
                    if (SG_IN(part.head + (part.v0 + v + 1) * VE <= V)) s = sum16<T, true>(ld_once(part.vectors() + v), c, o.m, s);
            }
            st = join_warp({o.m, keeper ? 0.f : s.x + s.y}, c);
            if (lane == 0) s_warp[warp] = st;
            __syncthreads();
            if (warp == 0) scalars(join_row());
            __syncthreads();
            o = s_out;
        }
        if (sizeof(T) == 2 && !o.wide && fabsf(o.k) > FAST_K) {
            // S has the rounding of m c in every term, the wide form's powers have not
            const float d = fmaf(o.m, c, -scaled(o.m, c));
            o.ls -= d;
            o.k *= elem::exp2_fast(d);
            o.wide = 1;
        }

        auto below = [&](float x) { return o.wide ? (x - o.m) * c : fmaf(x, c, -scaled(o.m, c)); };
        if constexpr (KIND == DISTILL) {
            if (rank == 0 && keeper) {   // the loss
                float sum = 0.f;
                if (!o.dead) {
                    for (int j = lane; j < a.top; j += 32) {
                        const float qj = list.q[j];
                        if (qj != 0.f) sum += qj * (list.lq[j] - (below(list.z[j]) - o.ls));
                    }
#pragma unroll
                    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
                }
                if (lane == 0) a.loss[row] = o.dead ? 0.f : mine.w * a.tau * a.tau * (sum * 0.693147180559945309f);
            }
        }
        auto places_of_next = [&]() {
            if (keeper && more) {
                const bool any = list.begin(a, static_cast<const T *>(a.z) + (row + clusters) * a.ldz, half, !now.skip(a) && (nrank > 1 || !CACHED),
                                             lane, at_places);
                if (lane == 0) s_places = any;
                __syncwarp();
                list.finish(a, half, lane);   // (nothing but the student's logits is left for the row's own time)
            }
        };
        if (g == nullptr) {
            places_of_next();
            continue;
        }

        T *gv = g + part.head + (long long)part.v0 * VE;
        const bool gvec = (reinterpret_cast<uintptr_t>(gv) & 15) == 0;
        if (o.dead) {
            for (int v = tid; v < n; v += DATA)
                if (SG_IN(part.head + (part.v0 + v + 1) * VE <= V)) put16<T>(gv + (long long)v * VE, make_uint4(0, 0, 0, 0), gvec);
            if (ei >= 0 && SG_IN(ei < V)) g[ei] = elem::from_f32<T>(0.f);
            places_of_next();
            continue;
        }
        const Slope q = {c, o.m, o.k};
        if (CACHED && gvec && !o.wide) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * DATA + tid;
                const uint4 x = give16<T, false>(keep[i], q);
                if (v < n && SG_IN(part.head + (part.v0 + v + 1) * VE <= V)) __stcs(reinterpret_cast<uint4 *>(gv) + v, x);
            }
        } else if constexpr (CACHED) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = i * DATA + tid;
                if (v < n && SG_IN(part.head + (part.v0 + v + 1) * VE <= V))
                    put16<T>(gv + (long long)v * VE, o.wide ? give16<T, true>(keep[i], q) : give16<T, false>(keep[i], q), gvec);
            }
        } else {
            for (int v = tid; v < n; v += DATA)
                if (SG_IN(part.head + (part.v0 + v + 1) * VE <= V)) {
                    const uint4 x = ld_once(part.vectors() + v);
                    put16<T>(gv + (long long)v * VE, o.wide ? give16<T, true>(x, q) : give16<T, false>(x, q), gvec);
                }
        }
        if (ei >= 0 && SG_IN(ei < V)) g[ei] = elem::from_f32<T>(slope_at(ev, q, o.wide));
        // the named places again, after their vectors
        if constexpr (KIND == POLICY) {
            // by the thread that has written the vector (or the edge)
            const int at = mine.label, v = at < part.head ? -1 : (at - part.head) / VE;
            const bool owner = v >= 0 && v < part.nv ? v >= part.v0 && v < part.v0 + part.n && ((v - part.v0) & (THREADS - 1)) == tid
                                                     : ei == at;
            if (owner && SG_IN(at >= 0 && at < V)) g[at] = elem::from_f32<T>(o.at_label);
        } else {
            if (!keeper) {
                barrier_arrive(1, THREADS);
                continue;
            }
            barrier_sync(1, THREADS);
            const float wt = mine.w * a.tau;
            for (int j = lane; j < a.top; j += 32) {
                const int at = list.at[j];
                const float sum = list.sum[j];
                if (at >= 0 && !(sum < 0.f) && part.mine(at, rank) && SG_IN(at < V))
                    g[at] = elem::from_f32<T>(wt * (elem::exp2_fast(below(list.z[j]) - o.ls) - sum));
            }
            places_of_next();
        }
    }
}

}  // namespace rowloss
}  // namespace sgemm_gb300
