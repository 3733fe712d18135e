// The adapters' skinny products on the CUDA cores: shrink (H = s X S_a^T) of
// FP32 matrices and of few bfloat16 rows, and of FP32 matrices expand
// (Y += H E_a) and the gradients of an adapter (G_a = sum_t P_t^T X_t).
//
// A stack S holds l adapters of r rows of `cols` consecutive elements.  A
// row t of X belongs to adapter ids[t]; an id outside 0 .. l-1 is none.
#pragma once
#include <cstdint>

#include "elem.cuh"
#include "tcgen05_f16.cuh"

namespace sgemm_gb300 {
namespace lora {

struct ShrinkArgs {
    const void *x;
    long long ldx;
    const void *s;        // l x r rows of k
    long long lds;
    const int *ids;
    const float *scale;   // NULL: 1
    float *h;             // t x r
    int t, k, l, r;
    bool vec;             // k and rows of x and s are whole vectors of four elements
};

struct ExpandArgs {
    const float *h;       // t x r
    const float *e;       // l x r x n
    const int *ids;
    float *y;
    long long ldy;
    int t, n, l, r;
    bool vec;             // n and rows of e and y are whole vectors of four
};

// One gradient of a launch; a backward pass has two, over the same rows.
struct GradProblem {
    const float *p;       // t x r
    const float *x;
    long long ldx;
    float *g;             // l x r x k
    float *ws;            // splits x l x r x k partial sums (splits > 1)
    int k;                // 0: none
};
struct GradArgs {
    GradProblem of[2];
    bool vec;             // k and rows of x and g are whole vectors of four, of both
    const int *ids;
    int t, l, r, splits;
};

__device__ __forceinline__ float warp_sum_all(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c))));
}

// ---------------------------------------------------------------- shrink

constexpr int SHRINK_THREADS = 256;

// One row and four ranks per CTA (grid: t x ceil(r / 4)), its eight warps
// side by side along k: few rows are bound by the latency of their loads, so
// a thread's are wide, independent and all on their way at once (the row's
// before its adapter is known).  64 rows of 4096, rank 16, take 6.1 us under
// the profiler, with 5 MB read: latency.  VEC: rows of x and of the stack
// 16-byte aligned.
template <class T, bool VEC>
__global__ void __launch_bounds__(SHRINK_THREADS) shrink_row_kernel(const ShrinkArgs a) {
    griddep_wait();                // this kernel starts while the one in front of it ends
    griddep_launch_dependents();   // the projection's loop does not wait for H
    constexpr int VE = VEC ? 16 / (int)sizeof(T) : 1;
    constexpr int UN = 2;
    __shared__ float s_part[SHRINK_THREADS / 32][4];
    const int t = blockIdx.x, r0 = blockIdx.y * 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int id = a.ids[t];
    const bool has = id >= 0 && id < a.l;
    const T *x = static_cast<const T *>(a.x) + (long long)t * a.ldx;
    const int nr = min(4, a.r - r0), whole = a.k / VE;   // whole vectors of a row
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (has) {
        const T *s = static_cast<const T *>(a.s) + ((long long)id * a.r + r0) * a.lds;
        const T *row[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) row[q] = s + (long long)min(q, nr - 1) * a.lds;   // (a rank past r repeats the last)
        for (int v0 = tid; v0 < whole; v0 += SHRINK_THREADS * UN) {
            if constexpr (VEC) {
                uint4 xv[UN], sv[UN][4];
#pragma unroll
                for (int u = 0; u < UN; ++u) {
                    const int v = min(v0 + u * SHRINK_THREADS, whole - 1);
                    xv[u] = *reinterpret_cast<const uint4 *>(x + (long long)v * VE);
#pragma unroll
                    for (int q = 0; q < 4; ++q) sv[u][q] = *reinterpret_cast<const uint4 *>(row[q] + (long long)v * VE);
                }
#pragma unroll
                for (int u = 0; u < UN; ++u) {
                    if (v0 + u * SHRINK_THREADS >= whole) continue;
                    float xf[VE], sf[VE];
                    elem::unpack16<T>(xv[u], xf);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        elem::unpack16<T>(sv[u][q], sf);
#pragma unroll
                        for (int i = 0; i < VE; ++i) acc[q] = fmaf(xf[i], sf[i], acc[q]);
                    }
                }
            } else {
#pragma unroll
                for (int u = 0; u < UN; ++u) {
                    const int v = v0 + u * SHRINK_THREADS;
                    if (v >= whole) continue;
                    const float xf = elem::to_f32(x[v]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[q] = fmaf(xf, elem::to_f32(row[q][v]), acc[q]);
                }
            }
        }
        const int v = whole * VE + tid;   // what is behind the whole vectors
        if (VEC && v < a.k) {
            const float xf = elem::to_f32(x[v]);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[q] = fmaf(xf, elem::to_f32(row[q][v]), acc[q]);
        }
    }
    const float sc = has && a.scale ? a.scale[id] : 1.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float v = warp_sum_all(acc[q]);
        if (lane == 0) s_part[warp][q] = v;
    }
    __syncthreads();
    if (tid < 4 && r0 + tid < a.r) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < SHRINK_THREADS / 32; ++w) v += s_part[w][tid];
        if (SG_IN(t < a.t)) a.h[(long long)t * a.r + r0 + tid] = has ? v * sc : 0.f;
    }
}

// Eight rows per CTA: each load of an adapter's values serves every row of
// the tile's run of that adapter, each load of the rows' (from shared
// memory) four ranks.  KS warps share a group of four ranks along k.  Eight
// loads per thread are on their way at a time: with a branch around each the
// kernel took 24 us at 2048 x 2048, rank 16, against 18 without.
constexpr int SHRINK_ROWS = 8;
constexpr int SHRINK_CHUNK = 1024;

template <class T, int KS, bool VEC>
__global__ void __launch_bounds__(SHRINK_THREADS, 2) shrink_tile_kernel(const ShrinkArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int GPW = 8 / KS;   // groups of four ranks in work at a time
    constexpr int UN = 2;
    __shared__ float4 s_x[SHRINK_ROWS][SHRINK_CHUNK / 4];
    __shared__ float s_part[8][SHRINK_ROWS][4];
    __shared__ int s_id[SHRINK_ROWS];
    const long long t0 = (long long)blockIdx.x * SHRINK_ROWS;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rows = (int)min((long long)SHRINK_ROWS, a.t - t0);
    if (tid < SHRINK_ROWS) {
        const int id = tid < rows ? a.ids[t0 + tid] : -1;
        s_id[tid] = id >= 0 && id < a.l ? id : -1;
    }
    __syncthreads();
    const T *x = static_cast<const T *>(a.x) + t0 * a.ldx;
    const int groups = (a.r + 3) / 4;
    for (int i0 = 0; i0 < rows;) {
        const int id = s_id[i0];
        int i1 = i0 + 1;
        while (i1 < rows && s_id[i1] == id) ++i1;
        if (id < 0) {
            for (int i = tid; i < (i1 - i0) * a.r; i += SHRINK_THREADS) a.h[(t0 + i0) * a.r + i] = 0.f;
            i0 = i1;
            continue;
        }
        const float sc = a.scale ? a.scale[id] : 1.f;
        for (int gb = 0; gb < groups; gb += GPW) {
            const int grp = gb + warp / KS, part = warp % KS;
            const int nr = min(4, a.r - grp * 4);   // <= 0: no group
            const T *s = static_cast<const T *>(a.s) + ((long long)id * a.r + grp * 4) * a.lds;
            float acc[SHRINK_ROWS][4];
#pragma unroll
            for (int i = 0; i < SHRINK_ROWS; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[i][q] = 0.f;
            for (int k0 = 0; k0 < a.k; k0 += SHRINK_CHUNK) {
                const int kn = min(SHRINK_CHUNK, a.k - k0), nf = (kn + 3) / 4;
                float4 xv[SHRINK_ROWS];
#pragma unroll
                for (int i = 0; i < SHRINK_ROWS; ++i)
                    xv[i] = elem::fetch4<T, VEC>(x + i * a.ldx + k0 + tid * 4, i >= i0 && i < i1 ? kn - tid * 4 : 0);
                __syncthreads();   // the chunk before is used up
#pragma unroll
                for (int i = 0; i < SHRINK_ROWS; ++i) s_x[i][tid] = xv[i];
                __syncthreads();
                for (int f0 = part * 32 + lane; f0 < nf && nr > 0; f0 += KS * 32 * UN) {
                    float4 sv[UN][4];
#pragma unroll
                    for (int u = 0; u < UN; ++u) {
                        const int f = f0 + u * KS * 32;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            sv[u][q] = elem::fetch4<T, VEC>(s + q * a.lds + k0 + f * 4, q < nr ? kn - f * 4 : 0);
                    }
#pragma unroll
                    for (int u = 0; u < UN; ++u) {
                        const int f = min(f0 + u * KS * 32, SHRINK_CHUNK / 4 - 1);   // (past the chunk sv is 0)
#pragma unroll
                        for (int i = 0; i < SHRINK_ROWS; ++i) {
                            if (i < i0 || i >= i1) continue;
                            const float4 v = s_x[i][f];
#pragma unroll
                            for (int q = 0; q < 4; ++q) acc[i][q] = f0 + u * KS * 32 < nf ? dot4(v, sv[u][q], acc[i][q]) : acc[i][q];
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < SHRINK_ROWS; ++i) {
                if (i < i0 || i >= i1) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float v = warp_sum_all(acc[i][q]);
                    if (lane == 0) s_part[warp][i][q] = v;
                }
            }
            __syncthreads();
            for (int e = tid; e < GPW * (i1 - i0) * 4; e += SHRINK_THREADS) {
                const int q = e & 3, i = i0 + (e >> 2) % (i1 - i0), gw = (e >> 2) / (i1 - i0);
                const int r = (gb + gw) * 4 + q;
                if (r < a.r) {
                    float v = 0.f;
#pragma unroll
                    for (int p = 0; p < KS; ++p) v += s_part[gw * KS + p][i][q];
                    if (SG_IN(t0 + i < a.t)) a.h[(t0 + i) * a.r + r] = v * sc;
                }
            }
        }
        i0 = i1;
    }
}

// ---------------------------------------------------------------- expand

constexpr int EXPAND_THREADS = 128;
constexpr int EXPAND_ROWS = 8;
constexpr int EXPAND_MAX_R = 256;

// Y += H E_a, eight rows by 512 columns per CTA; a row without an adapter is
// left alone.  The rows' H is one stretch of memory; Y and eight ranks of E per
// thread are on their way at a time.  16 us under the profiler at 2048 x 2048,
// rank 16, where Y, read and written, needs 5: short CTAs, whose loads' latency
// shows.
template <bool VEC>
__global__ void __launch_bounds__(EXPAND_THREADS) expand_kernel(const ExpandArgs a) {
    constexpr int UN = 8;
    griddep_wait();
    __shared__ float s_h[EXPAND_ROWS * EXPAND_MAX_R];
    __shared__ int s_id[EXPAND_ROWS];
    const long long t0 = (long long)blockIdx.x * EXPAND_ROWS;
    const int tid = threadIdx.x;
    const int rows = (int)min((long long)EXPAND_ROWS, a.t - t0);
    if (tid < EXPAND_ROWS) {
        const int id = tid < rows ? a.ids[t0 + tid] : -1;
        s_id[tid] = id >= 0 && id < a.l ? id : -1;
    }
#pragma unroll 4
    for (int i = tid; i < rows * a.r; i += EXPAND_THREADS) s_h[i] = a.h[t0 * a.r + i];
    __syncthreads();
    const int c = (blockIdx.y * EXPAND_THREADS + tid) * 4, left = a.n - c;
    if (left <= 0) return;
    for (int i0 = 0; i0 < rows;) {
        const int id = s_id[i0];
        int i1 = i0 + 1;
        while (i1 < rows && s_id[i1] == id) ++i1;
        if (id < 0) {
            i0 = i1;
            continue;
        }
        float4 acc[EXPAND_ROWS];
#pragma unroll
        for (int i = 0; i < EXPAND_ROWS; ++i)
            acc[i] = elem::fetch4<float, VEC>(a.y + (t0 + i) * a.ldy + c, i >= i0 && i < i1 && SG_IN(t0 + i < a.t && c < a.n) ? left : 0);
        {
            const float *e = a.e + (long long)id * a.r * a.n + c;
            for (int r0 = 0; r0 < a.r; r0 += UN) {
                float4 ev[UN];
#pragma unroll
                for (int u = 0; u < UN; ++u) ev[u] = elem::fetch4<float, VEC>(e + (long long)(r0 + u) * a.n, r0 + u < a.r ? left : 0);
#pragma unroll
                for (int u = 0; u < UN; ++u) {
                    if (r0 + u >= a.r) continue;
#pragma unroll
                    for (int i = 0; i < EXPAND_ROWS; ++i) {
                        if (i < i0 || i >= i1) continue;
                        const float h = s_h[i * a.r + r0 + u];
                        acc[i].x = fmaf(h, ev[u].x, acc[i].x);
                        acc[i].y = fmaf(h, ev[u].y, acc[i].y);
                        acc[i].z = fmaf(h, ev[u].z, acc[i].z);
                        acc[i].w = fmaf(h, ev[u].w, acc[i].w);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < EXPAND_ROWS; ++i) {
            if (i < i0 || i >= i1) continue;
            if (SG_IN(t0 + i < a.t && c < a.n)) elem::store4(a.y + (t0 + i) * a.ldy + c, acc[i], left, VEC);
        }
        i0 = i1;
    }
}

// ---------------------------------------------------------------- gradients of the adapters

constexpr int GRAD_THREADS = 256;
constexpr int GRAD_COLS = 64;
constexpr int GRAD_RANKS = 16;
constexpr int GRAD_CHUNK = 64;
constexpr int GRAD_WINDOW = 1024;

// 64 columns and 16 ranks of one adapter's gradient per CTA (grid: (adapters'
// rank blocks, for each of the column blocks of both problems in turn) x splits
// of the rows: a grid's other axes end at 65535, 4 million columns).  The
// CTA lists the rows of its part that belong to its adapter, a window of 1024
// at a time, and sums over them in 16 lanes of rows, 64 rows to a step: their
// P in shared memory, and a thread's four loads of X and four of P for the
// next step on their way meanwhile.  The lanes are added in a fixed order.
// Both gradients of 2048 rows x 2048, rank 16, take 27 us.
template <bool VEC>
__global__ void __launch_bounds__(GRAD_THREADS, 2) grad_kernel(const GradArgs a) {
    griddep_wait();
    __shared__ int s_row[GRAD_WINDOW];
    __shared__ int s_cnt[GRAD_THREADS / 32];
    __shared__ union {
        float4 p[GRAD_CHUNK][GRAD_RANKS / 4];
        float4 sum[GRAD_THREADS / 32][GRAD_RANKS][GRAD_COLS / 4];
    } s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c4 = tid & 15, tl = tid >> 4;
    const int rblocks = (a.r + GRAD_RANKS - 1) / GRAD_RANKS;
    const int lr = a.l * rblocks, block = (int)(blockIdx.x / lr), of_l = (int)(blockIdx.x % lr);
    const int id = of_l / rblocks, r0 = (of_l % rblocks) * GRAD_RANKS;
    const int blocks0 = (a.of[0].k + GRAD_COLS - 1) / GRAD_COLS;
    const GradProblem &pr = a.of[block >= blocks0];
    const int c = (block - (block >= blocks0 ? blocks0 : 0)) * GRAD_COLS + c4 * 4;
    const int nr = min(GRAD_RANKS, a.r - r0), left = pr.k - c;
    const long long per = ((long long)a.t + a.splits - 1) / a.splits;
    const int tb = (int)min((long long)a.t, per * blockIdx.y), te = (int)min((long long)a.t, tb + per);
    const float *x = pr.x + c;
    float4 acc[GRAD_RANKS];
#pragma unroll
    for (int r = 0; r < GRAD_RANKS; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w0 = tb; w0 < te; w0 += GRAD_WINDOW) {
        // the window's rows of the adapter in order, an eighth per warp, in two passes
        const int qb = w0 + warp * (GRAD_WINDOW / 8), qe = min(te, qb + GRAD_WINDOW / 8);
        uint32_t in[GRAD_WINDOW / 256];
        int n = 0;
#pragma unroll
        for (int i = 0; i < GRAD_WINDOW / 256; ++i) {
            const int t = qb + i * 32 + lane;
            in[i] = __ballot_sync(0xffffffffu, t < qe && a.ids[t] == id);
            n += __popc(in[i]);
        }
        __syncthreads();   // the list before is used up
        if (lane == 0) s_cnt[warp] = n;
        __syncthreads();
        int at = 0, cnt = 0;
#pragma unroll
        for (int w = 0; w < GRAD_THREADS / 32; ++w) {
            if (w < warp) at += s_cnt[w];
            cnt += s_cnt[w];
        }
#pragma unroll
        for (int i = 0; i < GRAD_WINDOW / 256; ++i) {
            if (in[i] >> lane & 1) s_row[at + __popc(in[i] & ((1u << lane) - 1))] = qb + i * 32 + lane;
            at += __popc(in[i]);
        }
        __syncthreads();   // the list
        constexpr int UX = GRAD_CHUNK / 16, UP = GRAD_CHUNK * GRAD_RANKS / GRAD_THREADS;
        float4 nx[UX];
        float np[UP];
        auto fetch = [&](int j0) {
#pragma unroll
            for (int u = 0; u < UX; ++u) {
                const int j = j0 + tl + 16 * u;
                nx[u] = elem::fetch4<float, VEC>(x + (j < cnt ? s_row[j] * pr.ldx : 0), j < cnt ? left : 0);
            }
#pragma unroll
            for (int u = 0; u < UP; ++u) {
                const int j = j0 + u * (GRAD_THREADS / GRAD_RANKS) + tl, r = c4;   // 16 ranks of 16 rows a time
                np[u] = j < cnt && r < nr ? pr.p[(long long)s_row[j] * a.r + r0 + r] : 0.f;
            }
        };
        fetch(0);
        for (int j0 = 0; j0 < cnt; j0 += GRAD_CHUNK) {
            float4 xv[UX];
#pragma unroll
            for (int u = 0; u < UX; ++u) xv[u] = nx[u];
            __syncthreads();   // the chunk before is used up
#pragma unroll
            for (int u = 0; u < UP; ++u) reinterpret_cast<float *>(s.p)[(u * 16 + tl) * GRAD_RANKS + c4] = np[u];
            __syncthreads();
            fetch(j0 + GRAD_CHUNK);
#pragma unroll
            for (int u = 0; u < GRAD_CHUNK / 16; ++u) {
#pragma unroll
                for (int q = 0; q < GRAD_RANKS / 4; ++q) {
                    const float4 p = s.p[tl + 16 * u][q];
                    const float pf[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float4 &v = acc[4 * q + i];
                        v.x = fmaf(pf[i], xv[u].x, v.x);
                        v.y = fmaf(pf[i], xv[u].y, v.y);
                        v.z = fmaf(pf[i], xv[u].z, v.z);
                        v.w = fmaf(pf[i], xv[u].w, v.w);
                    }
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < GRAD_RANKS; ++r) {
        float4 v = acc[r];
        v.x += __shfl_xor_sync(0xffffffffu, v.x, 16);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, 16);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, 16);
        v.w += __shfl_xor_sync(0xffffffffu, v.w, 16);
        if (lane < 16) s.sum[warp][r][lane] = v;
    }
    __syncthreads();
    const int r = tid >> 4;
    if (r < nr && left > 0) {
        float4 v = s.sum[0][r][c4];
#pragma unroll
        for (int w = 1; w < GRAD_THREADS / 32; ++w) {
            const float4 u = s.sum[w][r][c4];
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
        }
        const long long row = (long long)id * a.r + r0 + r;
        if (SG_IN(id < a.l && r0 + r < a.r)) {
            if (a.splits > 1)
                elem::store4(pr.ws + ((long long)blockIdx.y * a.l * a.r + row) * pr.k + c, v, left, VEC);
            else
                elem::store4(pr.g + row * pr.k + c, v, left, VEC);
        }
    }
}

// G = the sum of `splits` partial gradients of `count` values, in order, for
// both problems.
template <class T>
struct GradSumArgs {
    const float *ws[2];
    T *g[2];
    long long count[2];
    int splits;
};

template <class T>
__global__ void __launch_bounds__(256) grad_sum_kernel(const GradSumArgs<T> a) {
    griddep_wait();
    long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int o = i >= a.count[0];
    if (o) i -= a.count[0];
    if (i >= a.count[o]) return;
    float v = 0.f;
    for (int s = 0; s < a.splits; ++s) v += a.ws[o][s * a.count[o] + i];
    a.g[o][i] = elem::from_f32<T>(v);
}

// ---------------------------------------------------------------- few FP32 rows

// Y = X op(W) + H E_a for few FP32 rows, W read once: 64 features by ROWS rows
// per CTA, W (and X) through a ring of asynchronous copies 32 deep in k, four
// groups of threads side by side along k, a cluster of CTAs too.  One thread
// has one feature: four of its W from shared memory meet four k of each row
// (a broadcast), 4 ROWS FMAs.  The sums over groups and CTAs are added in a
// fixed order, every product is an FP32 FMA.
//
// Bound by W: 64 MB, 10 us, at 4096 x 4096.  For one row there a call with
// the library's sgemm, made for tiles of 128 rows, takes 56 us, with this
// kernel 16.7; at 16 rows, where the FMAs and the broadcasts of X count as
// much as W, 74 and 37.
struct FewArgs {
    const float *x, *w, *e;
    long long ldx, ldw;
    const float *h;
    const int *ids;
    float *y;
    long long ldy;
    int t, k, n, l, r;    // l or r 0: no adapters
    bool vec;             // rows of w 16-byte aligned
};

constexpr int FEW_THREADS = 256;
constexpr int FEW_COLS = 64;
constexpr int FEW_K = 32;
constexpr int FEW_STAGES = 6;
constexpr int FEW_W = FEW_COLS * (FEW_K + 4);   // floats of a stage's W: pitch 36 (k inside) or 72 (features inside, 32 lines)

template <int ROWS, bool W_MN>
__global__ void __launch_bounds__(FEW_THREADS, 2) few_rows_kernel(const FewArgs a) {
    constexpr int PITCH = W_MN ? FEW_COLS + 8 : FEW_K + 4;
    extern __shared__ __align__(16) float s_few[];   // stages of W, then of X
    float *s_w = s_few, *s_x = s_few + FEW_STAGES * FEW_W;
    const int tid = threadIdx.x, f = tid & (FEW_COLS - 1), grp = tid >> 6;
    const int rank = (int)tc::cluster_ctarank(), split = (int)tc::cluster_nctarank();
    const int n0 = (int)(blockIdx.x / split) * FEW_COLS;
    const long long t0 = (long long)blockIdx.y * ROWS;
    const int rows = (int)min((long long)ROWS, a.t - t0);
    const int nk_all = (a.k + FEW_K - 1) / FEW_K;
    const int kb = (int)((long long)nk_all * rank / split), nk = (int)((long long)nk_all * (rank + 1) / split) - kb;

    auto load = [&](int c) {
        if (c < nk) {
            const int k0 = (kb + c) * FEW_K, s = c % FEW_STAGES;
            float *w = s_w + s * FEW_W;
            constexpr int LINES = W_MN ? FEW_K : FEW_COLS, WIDE = W_MN ? FEW_COLS : FEW_K;
            // (lines: rows of W as stored, WIDE values of each)
            const int line_end = W_MN ? a.k - k0 : a.n - n0, wide_end = W_MN ? a.n - n0 : a.k - k0;
            const float *src = W_MN ? a.w + (long long)k0 * a.ldw + n0 : a.w + (long long)n0 * a.ldw + k0;
            if (a.vec) {
#pragma unroll
                for (int e = tid; e < LINES * WIDE / 4; e += FEW_THREADS) {
                    const int line = e / (WIDE / 4), c4 = e % (WIDE / 4) * 4;
                    const int bytes = line < line_end ? max(0, min(16, (wide_end - c4) * 4)) : 0;
                    cp_async_16(smem_u32(w + line * PITCH + c4), bytes > 0 ? src + line * a.ldw + c4 : a.w, (uint32_t)bytes);
                }
            } else {
#pragma unroll
                for (int e = tid; e < LINES * WIDE; e += FEW_THREADS) {
                    const int line = e / WIDE, c1 = e % WIDE;
                    const bool in = line < line_end && c1 < wide_end;
                    cp_async_4(smem_u32(w + line * PITCH + c1), in ? src + line * a.ldw + c1 : a.w, in ? 4u : 0u);
                }
            }
#pragma unroll
            for (int e = tid; e < ROWS * FEW_K; e += FEW_THREADS) {
                const int row = e / FEW_K, k = e % FEW_K;
                const bool in = row < rows && k0 + k < a.k;
                cp_async_4(smem_u32(s_x + (s * ROWS + row) * FEW_K + k), in ? a.x + (t0 + row) * a.ldx + k0 + k : a.x, in ? 4u : 0u);
            }
        }
        cp_async_commit();
    };

    float acc[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) acc[i] = 0.f;
    for (int c = 0; c < FEW_STAGES - 1; ++c) load(c);
    for (int c = 0; c < nk; ++c) {
        cp_async_wait<FEW_STAGES - 2>();
        __syncthreads();   // stage c is here; the one before it is used up
        load(c + FEW_STAGES - 1);
        const int s = c % FEW_STAGES;
        const float *w = s_w + s * FEW_W;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int k = grp * 8 + q * 4;
            float4 wv;
            if (W_MN)
                wv = make_float4(w[k * PITCH + f], w[(k + 1) * PITCH + f], w[(k + 2) * PITCH + f], w[(k + 3) * PITCH + f]);
            else
                wv = *reinterpret_cast<const float4 *>(w + f * PITCH + k);
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                acc[i] = dot4(*reinterpret_cast<const float4 *>(s_x + (s * ROWS + i) * FEW_K + k), wv, acc[i]);
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    // the groups' sums meet in group 0's place, then the CTAs'
    float *s_sum = s_few;   // [4][ROWS][FEW_COLS]
#pragma unroll
    for (int i = 0; i < ROWS; ++i) s_sum[(grp * ROWS + i) * FEW_COLS + f] = acc[i];
    __syncthreads();
    for (int i = grp; i < ROWS; i += 4) {
        float v = s_sum[i * FEW_COLS + f];
#pragma unroll
        for (int g = 1; g < 4; ++g) v += s_sum[(g * ROWS + i) * FEW_COLS + f];
        s_sum[i * FEW_COLS + f] = v;
    }
    griddep_wait();   // H may come from the kernel in front of this one
    if (split > 1) tc::cluster_sync();
    else __syncthreads();
    const bool adapters = a.l > 0 && a.r > 0;
    for (int i = rank + grp * split; i < rows; i += 4 * split) {
        float v = 0.f;
        if (split > 1) {
            const uint32_t at = smem_u32(s_sum + i * FEW_COLS + f);
            for (int p = 0; p < split; ++p) v += tc::ld_cluster_f32(tc::map_shared_rank(at, (uint32_t)p));
        } else {
            v = s_sum[i * FEW_COLS + f];
        }
        if (n0 + f >= a.n) continue;
        const int id = adapters ? a.ids[t0 + i] : -1;
        if (id >= 0 && id < a.l) {
            const float *h = a.h + (t0 + i) * a.r, *e = a.e + (long long)id * a.r * a.n + n0 + f;
            float sum = 0.f;
#pragma unroll 8
            for (int r = 0; r < a.r; ++r) sum = fmaf(h[r], e[(long long)r * a.n], sum);
            v += sum;
        }
        if (SG_IN(t0 + i < a.t)) a.y[(t0 + i) * a.ldy + n0 + f] = v;
    }
    if (split > 1) tc::cluster_sync();   // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------- rows TMA can read

// Copies of 16-bit matrices whose rows TMA cannot read, with rows 16 bytes
// apart: a warp per row, eight values a lane, read as widely as the row's
// alignment allows (`step` values at a time).
struct PadJob {
    const uint16_t *src;
    uint16_t *dst;
    long long lds, ldd, rows;
    int cols, step;
};
constexpr int PAD_JOBS = 5;
struct PadArgs {
    PadJob job[PAD_JOBS];
    int jobs;
};

static __global__ void __launch_bounds__(256) pad_rows_kernel(const PadArgs a) {
    griddep_wait();
    for (int i = 0; i < a.jobs; ++i) {
        const PadJob &b = a.job[i];
        for (long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); row < b.rows; row += (long long)gridDim.x * 8) {
            const uint16_t *s = b.src + row * b.lds;
            uint16_t *d = b.dst + row * b.ldd;
            for (int c = (threadIdx.x & 31) * 8; c < b.cols; c += 256) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (c + 8 <= b.cols && b.step == 4) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(s + c), y = *reinterpret_cast<const uint2 *>(s + c + 4);
                    v = make_uint4(x.x, x.y, y.x, y.y);
                } else if (c + 8 <= b.cols && b.step == 2) {
                    const uint32_t *w = reinterpret_cast<const uint32_t *>(s + c);
                    v = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    uint32_t u[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) u[q] = c + q < b.cols ? s[c + q] : 0u;
                    v = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
                }
                if (SG_IN(c + 8 <= b.ldd)) *reinterpret_cast<uint4 *>(d + c) = v;
            }
        }
    }
}

}  // namespace lora
}  // namespace sgemm_gb300
