// Losses over rows of logits with their gradients by the logits: distillation
// from a teacher's top logits, and the clipped policy loss with a KL term.
//
// Mathematics.  Both need, per row z of V logits (divided by the temperature,
// 1 for the policy loss), only M = max z, S = sum exp((z - M) / tau) and the
// logits at a few named places; the gradient is then
//     distill:  tau w (p_v - q_v)          policy:  d (1[v = label] - p_v)
// with p_v = exp((z_v - M) / tau) / S, q the teacher's softmax over its
// usable places (zero elsewhere) and d the loss's derivative by
// lp = (z_label - M) - ln S.  Exponentials are taken to base 2 of
// (z - M) * (log2 e / tau), the difference first: a row of the type's lowest
// value then gives differences of zero, not an overflow.
//
// What bounds it.  The row has to come from memory once and its gradient go
// back once: 2 V sizeof(T) bytes, against ~10 operations per element.  So a
// row is read once into registers by a cluster of 1 to 8 CTAs (NV 16-byte
// vectors per thread), each thread keeps a maximum and a sum of its own, the
// CTAs exchange one (M, S) pair through distributed shared memory, and the
// gradient is written from the registers.  Rows longer than a cluster's
// registers (8 x 64 KB) are read a second time (CACHED = false).
//
// Rows start at any element: the vectors lie on the row's own 16-byte
// boundaries, the up to 2 (VE - 1) elements in front of and behind them go
// one each to the first threads of the cluster's first CTA.
#pragma once
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "elem.cuh"
#include "tcgen05.cuh"

namespace sgemm_gb300 {
namespace rowloss {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
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

// The statistics of a part of a row: its maximum and the sum of
// exp2((z - max) c).  A part without a logit above -inf has m = -inf, s = 0.
struct Stat {
    float m, s;
};

__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, a.s + b.s};   // both sums are 0, or NaN
    const float sa = a.m == m ? a.s : a.s * elem::exp2_fast((a.m - m) * c);
    const float sb = b.m == m ? b.s : b.s * elem::exp2_fast((b.m - m) * c);
    return {m, sa + sb};
}

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

template <class T>
__device__ __forceinline__ void unpack16(const uint4 &w, float *f) {
    constexpr int N = elem::Word<T>::N;
    elem::Word<T>::unpack(w.x, f);
    elem::Word<T>::unpack(w.y, f + N);
    elem::Word<T>::unpack(w.z, f + 2 * N);
    elem::Word<T>::unpack(w.w, f + 3 * N);
}

template <class T>
__device__ __forceinline__ uint4 pack16(const float *f) {
    constexpr int N = elem::Word<T>::N;
    return make_uint4(elem::Word<T>::pack(f), elem::Word<T>::pack(f + N), elem::Word<T>::pack(f + 2 * N),
                      elem::Word<T>::pack(f + 3 * N));
}

// A vector's elements joined to the thread's running statistics: one
// rescaling of the sum per vector at most.
template <class T>
__device__ __forceinline__ void take(Stat &st, const uint4 &w, float c) {
    constexpr int VE = 16 / sizeof(T);
    float f[VE];
    unpack16<T>(w, f);
    float m = f[0];
#pragma unroll
    for (int j = 1; j < VE; ++j) m = fmaxf(m, f[j]);
    if (m > st.m) {
        st.s = st.m == -INFINITY ? st.s : st.s * elem::exp2_fast((st.m - m) * c);
        st.m = m;
    }
    const float mm = st.m == -INFINITY ? 0.f : st.m;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VE; ++j) s += elem::exp2_fast((f[j] - mm) * c);
    st.s += s;
}

template <class T>
__device__ __forceinline__ void give(uint4 w, Stat st, float c, float k, T *g, bool vec) {
    constexpr int VE = 16 / sizeof(T);
    float f[VE];
    unpack16<T>(w, f);
#pragma unroll
    for (int j = 0; j < VE; ++j) f[j] = elem::exp2_tiny((f[j] - st.m) * c) * k;
    if (vec) {
        __stcs(reinterpret_cast<uint4 *>(g), pack16<T>(f));
    } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) g[j] = elem::from_f32<T>(f[j]);
    }
}

// A cluster of gridDim.x / t CTAs per row.
template <class T, Kind KIND, int NV, bool CACHED>
__global__ void __launch_bounds__(THREADS, NV >= 8 ? 2 : NV >= 4 ? 2 : 3) row_loss_kernel(const Args a) {
    constexpr int VE = 16 / sizeof(T);
    __shared__ Stat s_warp[WARPS];
    __shared__ Stat s_cta[MAX_CLUSTER];
    __shared__ float s_q[KIND == DISTILL ? MAX_TOP : 1];    // the teacher's logits, then q
    __shared__ float s_z[KIND == DISTILL ? MAX_TOP : 1];    // the student's logits there
    __shared__ int s_at[KIND == DISTILL ? MAX_TOP : 1];     // the places, -1 where not usable

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = tc::cluster_ctarank(), nrank = tc::cluster_nctarank();
    const long long row = blockIdx.x / nrank;
    const T *z = static_cast<const T *>(a.z) + row * a.ldz;
    T *g = a.grad ? static_cast<T *>(a.grad) + row * a.ldg : nullptr;
    const int V = a.v;

    // the row's vectors and edges, and this CTA's part of them
    int head = (int)((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / (int)sizeof(T);
    if (head > V) head = V;
    const int nv = (V - head) / VE, tail = V - head - nv * VE;
    const int per = (nv + (int)nrank - 1) / (int)nrank;
    const int v0 = min(nv, (int)rank * per), v1 = min(nv, v0 + per);
    const uint4 *zv = reinterpret_cast<const uint4 *>(z + head);
    const bool gvec = g && ((reinterpret_cast<uintptr_t>(g + head) & 15) == 0);
    const bool edge = rank == 0 && tid < head + tail;
    const int ei = tid < head ? tid : V - tail + (tid - head);

    const float w = a.weight ? a.weight[row] : 1.f;
    int label = -1;
    bool skip = w == 0.f;
    if constexpr (KIND == POLICY) {
        label = a.label[row];
        const bool ok = label >= 0 && label < V;
        skip = (skip && a.logp == nullptr) || !ok;
    }

    Stat st = {-INFINITY, 0.f};
    uint4 keep[CACHED ? NV : 1];
    float ev = -INFINITY, zl = 0.f;
    bool dead = skip;
    if (!skip) {
        // every load of the row in flight before the first is used
        if constexpr (CACHED) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = v0 + i * THREADS + tid;
                if (v < v1 && SG_IN(head + (v + 1) * VE <= V)) keep[i] = ld_once(zv + v);
            }
        }
        if (edge && SG_IN(ei >= 0 && ei < V)) ev = elem::to_f32(z[ei]);
        if constexpr (KIND == POLICY) zl = elem::to_f32(z[label]);
        if constexpr (KIND == DISTILL) {
            for (int j = tid; j < a.top; j += THREADS) {
                const float tv = a.teacher[row * a.top + j];
                const int at = a.index[row * a.top + j];
                const bool ok = at >= 0 && at < V && !(tv == -INFINITY);
                s_q[j] = ok ? tv : -INFINITY;
                s_z[j] = ok ? elem::to_f32(z[at]) : 0.f;
                s_at[j] = ok ? at : -1;
            }
        }
        if (edge) {
            st.m = ev;
            st.s = ev == -INFINITY ? 0.f : elem::exp2_fast((ev - ev) * a.c);   // 1, or NaN
        }
        if constexpr (CACHED) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (v0 + i * THREADS + tid < v1) take<T>(st, keep[i], a.c);
        } else {
            for (int v = v0 + tid; v < v1; v += THREADS)
                if (SG_IN(head + (v + 1) * VE <= V)) take<T>(st, ld_once(zv + v), a.c);
        }
        // the warp, the CTA, the cluster
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            st = join(st, {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o)}, a.c);
        if (lane == 0) s_warp[warp] = st;
        __syncthreads();
        st = s_warp[lane & (WARPS - 1)];
#pragma unroll
        for (int o = WARPS / 2; o > 0; o >>= 1)
            st = join(st, {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o)}, a.c);
        if (nrank > 1) {
            if (tid < (int)nrank) st_cluster_v2(tc::map_shared_rank(smem_u32(&s_cta[rank]), tid), st.m, st.s);
            // no CTA writes a gradient (which may lie on the logits) before
            // every CTA has read its part and the named places
            tc::cluster_sync();
            st = s_cta[0];
            for (uint32_t i = 1; i < nrank; ++i) st = join(st, s_cta[i], a.c);
        } else {
            __syncthreads();   // the same within the CTA
        }
        dead = st.m == -INFINITY && st.s == 0.f;
    }

    const float lns = logf(st.s);
    float k = 0.f;      // p_v's factor: the gradient is k exp2((z_v - M) c) off the named places
    float d = 0.f;      // policy: the loss's derivative by lp
    float tm = -INFINITY, ts = 0.f;
    if constexpr (KIND == POLICY) {
        const float lp = (zl - st.m) - lns;
        float loss = 0.f;
        if (!dead && w != 0.f) {
            const float adv = a.adv[row];
            const float r = expf(lp - a.old_logp[row]);
            const float u = r * adv, b = fminf(fmaxf(r, 1.f - a.clip_low), 1.f + a.clip_high) * adv;
            loss = -fminf(u, b);
            d = u <= b ? -u : 0.f;
            if (r != r) loss = d = r;
            if (a.kl != 0.f) {
                const float x = a.ref[row] - lp, e = expf(x);
                loss += a.kl * (e - x - 1.f);
                d += a.kl * (1.f - e);
            }
            loss *= w;
            d *= w;
        }
        if (rank == 0 && tid == 0) {
            a.loss[row] = loss;
            if (a.logp) a.logp[row] = skip ? 0.f : dead ? -INFINITY : lp;
        }
        if (w == 0.f) dead = true;
        k = -d / st.s;
    } else {
        if (!skip) {
            // every warp sums the teacher's softmax for itself
            for (int j = lane; j < a.top; j += 32) tm = fmaxf(tm, s_q[j]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
            const float tmm = tm == -INFINITY ? 0.f : tm;
            for (int j = lane; j < a.top; j += 32) ts += elem::exp2_fast((s_q[j] - tmm) * a.c);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ts += __shfl_xor_sync(0xffffffffu, ts, o);
            if (ts == 0.f) dead = true;
            tm = tmm;
        }
        if (rank == 0 && warp == 0) {
            float sum = 0.f;
            if (!dead) {
                const float it = 1.f / a.tau, lnt = logf(ts);
                for (int j = lane; j < a.top; j += 32) {
                    const float q = elem::exp2_fast((s_q[j] - tm) * a.c) / ts;
                    if (q != 0.f) sum += q * (((s_q[j] - tm) * it - lnt) - ((s_z[j] - st.m) * it - lns));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            if (lane == 0) a.loss[row] = dead ? 0.f : w * a.tau * a.tau * sum;
        }
        k = w * a.tau / st.s;
    }
    if (g == nullptr) return;

    if (dead) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int v = v0 + tid; v < v1; v += THREADS) {
            T *p = g + head + (long long)v * VE;
            if (gvec) {
                __stcs(reinterpret_cast<uint4 *>(p), zero);
            } else {
#pragma unroll
                for (int j = 0; j < VE; ++j) p[j] = elem::from_f32<T>(0.f);
            }
        }
        if (edge) g[ei] = elem::from_f32<T>(0.f);
        return;
    }
    if constexpr (CACHED) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = v0 + i * THREADS + tid;
            if (v < v1 && SG_IN(head + (v + 1) * VE <= V)) give<T>(keep[i], st, a.c, k, g + head + (long long)v * VE, gvec);
        }
    } else {
        for (int v = v0 + tid; v < v1; v += THREADS)
            if (SG_IN(head + (v + 1) * VE <= V)) give<T>(ld_once(zv + v), st, a.c, k, g + head + (long long)v * VE, gvec);
    }
    if (edge && SG_IN(ei >= 0 && ei < V)) g[ei] = elem::from_f32<T>(elem::exp2_tiny((ev - st.m) * a.c) * k);
    __syncthreads();   // the named places are written again, after their vectors

    auto mine = [&](int at) {
        const int v = at < head ? -1 : (at - head) / VE;
        return v < 0 || v >= nv ? rank == 0 : v >= v0 && v < v1;
    };
    if constexpr (KIND == POLICY) {
        if (tid == 0 && mine(label)) {
            const float p = elem::exp2_fast((zl - st.m) * a.c) / st.s;
            g[label] = elem::from_f32<T>(d - d * p);
        }
    } else {
        for (int j = tid; j < a.top; j += THREADS) {
            const int at = s_at[j];
            if (at < 0 || !mine(at)) continue;
            float q = 0.f;
            bool first = true;
            for (int i = 0; i < a.top; ++i) {   // places that name the same index add up, written by the first
                if (s_at[i] != at) continue;
                first = first && i >= j;
                q += elem::exp2_fast((s_q[i] - tm) * a.c) / ts;
            }
            if (!first) continue;
            const float p = elem::exp2_fast((s_z[j] - st.m) * a.c) / st.s;
            g[at] = elem::from_f32<T>(w * a.tau * (p - q));
        }
    }
}

}  // namespace rowloss
}  // namespace sgemm_gb300
