// The adapters' skinny products of bfloat16 matrices on the tensor cores
// (FP32 accumulators):
//
//     shrink    H[t][r] = s_a sum_k X[t][k] S[a][r][k],   a = ids[t]
//     gradient  G[a][r][f] = sum over the rows t of adapter a of P[t][r] X[t][f]
//
// Both are bound by reading X once: at rank r they do 2 r operations per
// value of X, 16 to 128 FLOP/byte for ranks 16 to 128, which the CUDA cores
// cannot follow above rank ~8 (80 TFLOP/s against 6.8 TB/s) and the tensor
// cores hardly notice.  At 8192 rows of 4096, rank 64, a shrink takes 23 us (10
// for X's bytes; every tile of 64 rows loads its adapters' rows again, out of L2
// as many bytes as X's own there, and the rest is the latency of loads), both
// gradients 54 (20).
#pragma once
#include <cstdint>

#include <cuda.h>

#include "elem.cuh"
#include "lora_simt.cuh"
#include "lora_tc.cuh"
#include "tcgen05_f16.cuh"

namespace sgemm_gb300 {
namespace lora {

constexpr int kWaitShrink = 0x216, kWaitShrinkMma = 0x217, kWaitShrinkAcc = 0x218, kWaitGrad = 0x219, kWaitGradMma = 0x21a,
              kWaitGradAcc = 0x21b;

// ---------------------------------------------------------------- the parts of H
//
// The gradient reads H (or U) as two bfloat16 parts hi + lo: t rows of
// gr_blocks(r) blocks of gr_ranks(r) hi, then as many lo.

constexpr int GR_RANKS = 64;
__host__ __device__ constexpr int gr_ranks(int r) { return r >= GR_RANKS ? GR_RANKS : (r + 7) / 8 * 8; }   // ranks of a block
__host__ __device__ constexpr int gr_blocks(int r) { return (r + GR_RANKS - 1) / GR_RANKS; }

// Where the two parts of a rank of row t are, and what they are.
__device__ __forceinline__ void put_parts(__nv_bfloat16 *parts, long long row, int rank, int r, float v) {
    const int n = gr_ranks(r), b = rank / GR_RANKS;
    __nv_bfloat16 *d = parts + (row * gr_blocks(r) + b) * 2 * n + rank - b * GR_RANKS;
    elem::parts(v, d[0], d[n]);
}

// ---------------------------------------------------------------- shrink
//
// A tile of SH_BN rows of X is the operand N, the listed adapters' rows of S
// the operand M: 128 / (r rounded up to 8) adapters at a time, each brought by
// a TMA box of its own, k in stages of 64.  Of an accumulator column only its
// own adapter's lanes are kept, so what other adapters hold (NaN too) does
// not reach a row.  A tile whose rows name more adapters takes further
// passes.  Few tiles are cut along k into the CTAs of a cluster.

constexpr int SH_BN = 64;
constexpr int SH_STAGES = 4;
constexpr int SH_STAGE = TC_M_BYTES + SH_BN * TC_K * 2;
constexpr int SH_THREADS = 192;   // warp 0: TMA, warp 1: MMA, warps 2-5: the list, and the accumulator

struct ShrinkShared {
    uint64_t full[SH_STAGES], empty[SH_STAGES], acc;
    uint32_t tmem;
    int count;
    int wsum[4];
    int list[SH_BN];
    short slot[SH_BN];
};
constexpr int SH_SMEM = 1024 + SH_STAGES * SH_STAGE + (int)sizeof(ShrinkShared);
static_assert(SH_STAGES * SH_STAGE >= SH_BN * TC_M * 4, "the ring holds an accumulator");

struct ShrinkTcArgs {
    int t, k, l, r;
    const int *ids;
    const float *scale;   // NULL: 1
    float *h;
    __nv_bfloat16 *parts;   // NULL, or where the gradient wants H too
};

static __global__ void __launch_bounds__(SH_THREADS, 2)
    shrink_tc_kernel(const __grid_constant__ CUtensorMap map_s, const __grid_constant__ CUtensorMap map_x, const ShrinkTcArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
    ShrinkShared &sh = *reinterpret_cast<ShrinkShared *>(ring_ptr + SH_STAGES * SH_STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)tc::cluster_ctarank(), nsplit = (int)tc::cluster_nctarank();
    const int nk_all = (a.k + TC_K - 1) / TC_K;
    const int kb = (int)((long long)nk_all * rank / nsplit), nk = (int)((long long)nk_all * (rank + 1) / nsplit) - kb;
    const long long t0 = (long long)(blockIdx.x / nsplit) * SH_BN;
    const int rchunks = (a.r + 127) / 128;                       // passes of 128 ranks
    const int rows = a.r >= 128 ? 128 : (a.r + 7) / 8 * 8;       // lanes of an adapter
    const int per = 128 / rows;                                  // adapters of a pass

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&map_s);
        tma_prefetch_desc(&map_x);
        for (int i = 0; i < SH_STAGES; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        mbar_init(smem_u32(&sh.acc), 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(smem_u32(&sh.tmem), SH_BN);
        tc::tmem_relinquish();
    }
    griddep_wait();                // this kernel starts while the one in front of it ends
    griddep_launch_dependents();   // the projection's loop does not wait for H
    if (warp >= 2) {
        const int tid = threadIdx.x - 64;
        const int count = list_adapters<SH_BN>(a.ids, a.l, t0, a.t, sh.list, sh.slot, sh.wsum, tid);
        if (tid == 0) sh.count = count;
        if (rank == 0 && blockIdx.y == 0 && tid < SH_BN && t0 + tid < a.t && sh.slot[tid] < 0)   // (the thread's own entry)
            for (int r = 0; r < a.r; ++r) a.h[(t0 + tid) * a.r + r] = 0.f;   // (in no gradient's list)
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const int count = sh.count, passes = (count + per - 1) / per * rchunks;

    uint32_t it = 0, done = 0;
    bool ok = true;
    for (int p = blockIdx.y; p < passes; p += gridDim.y, ++done) {
        const int j0 = rchunks > 1 ? p / rchunks : p * per;      // the pass's first adapter
        const int nj = rchunks > 1 ? 1 : min(per, count - j0);
        const int r0 = rchunks > 1 ? p % rchunks * 128 : 0;
        if (warp == 0) {
            if (lane == 0) {
                for (int k = 0; k < nk && ok; ++k, ++it) {
                    const uint32_t s = it % SH_STAGES, st = ring + s * SH_STAGE, bar = smem_u32(&sh.full[s]);
                    if (!(ok = mbar_wait(smem_u32(&sh.empty[s]), ((it / SH_STAGES) & 1) ^ 1, kWaitShrink))) break;
                    mbar_arrive_expect_tx(bar, (uint32_t)(nj * rows * 128 + SH_BN * 128));
                    for (int j = 0; j < nj; ++j)
                        tma_load_3d(st + j * rows * 128, &map_s, (kb + k) * TC_K, r0, sh.list[j0 + j], bar);
                    tma_load_2d(st + TC_M_BYTES, &map_x, (kb + k) * TC_K, (int)t0, bar);
                }
            }
        } else if (warp == 1) {
            if (lane == 0) {
                uint32_t acc = 0;
                for (int k = 0; k < nk && ok; ++k, ++it) {
                    const uint32_t s = it % SH_STAGES, st = ring + s * SH_STAGE;
                    if (!(ok = mbar_wait(smem_u32(&sh.full[s]), (it / SH_STAGES) & 1, kWaitShrinkMma))) break;
                    tc::fence_after_sync();
                    const uint64_t ds = tc::desc_kmajor_sw128(st), dx = tc::desc_kmajor_sw128(st + TC_M_BYTES);
#pragma unroll
                    for (int q = 0; q < TC_K / 16; ++q) {
                        tc::mma_bf16(tmem, ds + (uint64_t)(q * 2), dx + (uint64_t)(q * 2),
                                     tc::idesc_bf16(TC_M, SH_BN, false, false), acc);
                        acc = 1;
                    }
                    tc::commit(smem_u32(&sh.empty[s]));
                }
                tc::commit(smem_u32(&sh.acc));
            }
        } else {
            ok = mbar_wait(smem_u32(&sh.acc), done & 1, kWaitShrinkAcc);
            tc::fence_after_sync();
            const int quad = warp & 3, row = quad * 32 + lane;
            const int j = row / rows, r = r0 + row - j * rows;   // this lane's adapter of the pass, its rank
            const bool mine = j < nj && r < a.r;
            const float sc = mine && a.scale ? a.scale[sh.list[j0 + j]] : 1.f;
#pragma unroll
            for (int c = 0; c < SH_BN; c += 32) {
                uint32_t v[32];
                __syncwarp();
                tc::ld_32x32b_x32(tmem + c + ((uint32_t)(quad * 32) << 16), v);
                tc::wait_ld();
                if (nsplit > 1) {
                    float *stage = reinterpret_cast<float *>(ring_ptr);
#pragma unroll
                    for (int i = 0; i < 32; ++i) stage[(c + i) * TC_M + row] = __uint_as_float(v[i]) * sc;
                } else if (mine) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (sh.slot[c + i] != j0 + j || !SG_IN(t0 + c + i < a.t)) continue;
                        const float x = __uint_as_float(v[i]) * sc;
                        a.h[(t0 + c + i) * a.r + r] = x;
                        if (a.parts) put_parts(a.parts, t0 + c + i, r, a.r, x);
                    }
                }
            }
            tc::fence_before_sync();
        }
        __syncwarp();
        if (nsplit > 1) {
            // the ranks' accumulators in rank order; every nsplit-th row of the tile is this rank's
            tc::cluster_sync();
            const int take = min(rows, a.r - r0);
            for (int q = threadIdx.x; q < SH_BN / nsplit * 128 + 128; q += SH_THREADS) {
                const int c = rank + q / 128 * nsplit, row = q & 127;
                if (c >= SH_BN) break;
                const int j = row / rows, r = row - j * rows;
                if (j < nj && r < take && sh.slot[c] == j0 + j) {
                    const uint32_t at = ring + (uint32_t)(c * TC_M + row) * 4;
                    float v = 0.f;
                    for (int u = 0; u < nsplit; ++u) v += tc::ld_cluster_f32(tc::map_shared_rank(at, (uint32_t)u));
                    if (!SG_IN(t0 + c < a.t)) continue;
                    a.h[(t0 + c) * a.r + r0 + r] = v;
                    if (a.parts) put_parts(a.parts, t0 + c, r0 + r, a.r, v);
                }
            }
            tc::cluster_sync();
            // (the next pass's TMA writes where these threads have read)
            tc::fence_proxy_async_smem();
            __syncthreads();
        } else {
            __syncthreads();   // the accumulator is drained
        }
        tc::fence_after_sync();
    }
    if (nsplit > 1) tc::cluster_sync();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, SH_BN);
    }
}

// ---------------------------------------------------------------- gradients of the adapters
//
// 128 features and up to 64 ranks of one adapter per CTA.  The CTA lists the
// rows of its part that belong to its adapter; 64 of them make a stage: the
// operand M is their values of X, the operand N their P as two bfloat16 parts
// hi + lo side by side (their sum keeps 16 bits of P; the two halves of the
// accumulator are added at the end), both MN-major, fetched row by row with
// 16-byte copies, so that a row of another adapter is never read.  Rows are
// cut into `splits` parts where adapters and features alone do not occupy the
// device; the parts' sums are added in order by a second kernel.
//
// The parts of P are made once per call, by the shrink or `parts_kernel`:
// splitting P in the loop, from plain loads, took 270 us at 8192 rows x 4096,
// rank 64.  One launch has both gradients of a backward pass.

constexpr int GR_WINDOW = 2048;   // rows that are listed at a time
constexpr int GR_WARPS = 8;       // list, load, drain; one more issues the MMAs (four loading took 62 us where eight take 54)
constexpr int GR_LOADERS = 32 * GR_WARPS;
constexpr int GR_THREADS = GR_LOADERS + 32;
constexpr int GR_AHEAD = 2;       // stages of copies in flight behind the one being written

__host__ __device__ constexpr int gr_stages(int r) { return r > 32 ? 3 : 4; }   // two CTAs to an SM
// (a line of the operand N is 128 bytes a 64 columns, used or not)
__host__ __device__ constexpr int gr_stage(int r) { return TC_M_BYTES + (r > 32 ? 2 : 1) * TC_M_BYTES / 2; }

struct GradShared {
    uint64_t full[4], empty[4], acc;
    uint32_t tmem;
    int wsum[GR_WARPS];
    int list[GR_WINDOW];
};
__host__ __device__ constexpr int gr_smem(int r) { return 1024 + gr_stages(r) * gr_stage(r) + (int)sizeof(GradShared); }

// One gradient of a launch; a backward pass has two, over the same rows.
struct GradTcProblem {
    const __nv_bfloat16 *parts;
    const __nv_bfloat16 *x;
    long long ldx;
    __nv_bfloat16 *g;             // l x r x k
    float *ws;                    // splits x l x r x k partial sums (splits > 1)
    int k;                        // 0: none
};
struct GradTcArgs {
    GradTcProblem of[2];
    const int *ids;
    int t, l, r, splits;
};

// The parts of an FP32 P of t x r (ranks past r: zeros).
struct PartsArgs {
    const float *p;
    __nv_bfloat16 *parts;
    int t, r;
};

static __global__ void __launch_bounds__(256) parts_kernel(const PartsArgs a) {
    griddep_wait();
    const float *p = a.p;
    __nv_bfloat16 *parts = a.parts;
    const int t = a.t, r = a.r;
    const int n = gr_ranks(r), width = gr_blocks(r) * n;
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
    if (e >= (long long)t * width) return;
    const long long row = e / width;
    const int rank = (int)(e - row * width);   // blocks but the last are whole: a rank is its place
    put_parts(parts, row, rank, r, rank < r ? p[row * r + rank] : 0.f);
}

static __global__ void __launch_bounds__(GR_THREADS, 2) grad_tc_kernel(const GradTcArgs a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
    const int nrank = gr_ranks(a.r), rblocks = gr_blocks(a.r), stage_bytes = gr_stage(a.r);
    const uint32_t nst = (uint32_t)gr_stages(a.r);
    GradShared &sh = *reinterpret_cast<GradShared *>(ring_ptr + nst * stage_bytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lr = a.l * rblocks, tile = (int)(blockIdx.x / lr), of_l = (int)(blockIdx.x % lr);
    const int id = of_l / rblocks, rb = of_l % rblocks, r0 = rb * GR_RANKS;
    const int tiles0 = (a.of[0].k + TC_M - 1) / TC_M;
    const GradTcProblem &pr = a.of[tile >= tiles0];
    const int f0 = (tile - (tile >= tiles0 ? tiles0 : 0)) * TC_M;
    const int nr = min(nrank, a.r - r0);
    const long long part = ((long long)a.t + a.splits - 1) / a.splits;
    const int tb = (int)min((long long)a.t, part * blockIdx.y), te = (int)min((long long)a.t, tb + part);

    if (tid == 0) {
        for (int i = 0; i < (int)nst; ++i) {
            mbar_init(smem_u32(&sh.full[i]), GR_LOADERS);
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        mbar_init(smem_u32(&sh.acc), 1);
        fence_mbar_init();
    }
    if (warp == GR_WARPS) {
        tc::tmem_alloc(smem_u32(&sh.tmem), 128);
        tc::tmem_relinquish();
    }
    griddep_wait();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;

    uint32_t it = 0;        // stages so far
    uint32_t acc = 0;
    bool ok = true;
    for (int w0 = tb; w0 < te; w0 += GR_WINDOW) {
        // the window's rows of the adapter in order, an eighth per warp: all
        // of its ids on their way at once
        constexpr int LOOKS = GR_WINDOW / GR_LOADERS;
        const int we = min(te, w0 + GR_WINDOW), qb = w0 + warp * (32 * LOOKS), qe = min(we, qb + 32 * LOOKS);
        uint32_t in[LOOKS];
        if (warp < GR_WARPS) {
            int ids[LOOKS], n = 0;
#pragma unroll
            for (int i = 0; i < LOOKS; ++i) {
                const int t = qb + i * 32 + lane;
                ids[i] = t < qe ? a.ids[t] : -1;
            }
#pragma unroll
            for (int i = 0; i < LOOKS; ++i) {
                in[i] = __ballot_sync(0xffffffffu, ids[i] == id);
                n += __popc(in[i]);
            }
            if (lane == 0) sh.wsum[warp] = n;
        }
        __syncthreads();   // (and the window before is used up)
        int at = 0, count = 0;
        for (int w = 0; w < GR_WARPS; ++w) {
            if (w < warp) at += sh.wsum[w];
            count += sh.wsum[w];
        }
        if (warp < GR_WARPS) {
#pragma unroll
            for (int i = 0; i < LOOKS; ++i) {
                if (in[i] >> lane & 1) sh.list[at + __popc(in[i] & ((1u << lane) - 1))] = qb + i * 32 + lane;
                at += __popc(in[i]);
            }
        }
        __syncthreads();
        const int stages = (count + 63) / 64;
        if (warp < GR_WARPS) {
            const __nv_bfloat16 *x = pr.x + f0;
            const __nv_bfloat16 *parts = pr.parts + rb * 2 * nrank;
            const long long ldp = (long long)rblocks * 2 * nrank;
            // this thread's chunk of X (16 rows apart, so one place in the swizzle)
            // and of P (pch chunks a row)
            const int xr = tid >> 4, xc = tid & 15, xbytes = max(0, min(16, (pr.k - f0 - xc * 8) * 2));
            const uint32_t xdst = (xc >> 3) * (TC_M_BYTES / 2) + xr * 128 + (((xc & 7) ^ (xr & 7)) << 4);
            const int pch = nrank / 4, pr0 = tid / pch, pc = tid - pr0 * pch, pstep = GR_LOADERS / pch;
            const uint32_t pdst = TC_M_BYTES + (pc >> 3) * (TC_M_BYTES / 2);
            x += xc * 8;
            parts += pc * 8;
            for (int c = 0; c < stages + GR_AHEAD; ++c) {
                if (c < stages) {
                    const uint32_t i = it + c, s = i % nst;
                    ok = ok && mbar_wait(smem_u32(&sh.empty[s]), ((i / nst) & 1) ^ 1, kWaitGrad);
                    const uint32_t st = ring + s * stage_bytes;
                    const int left = count - c * 64;
                    const int *rows = sh.list + c * 64;
                    if (ok) {
                        // 64 rows of X and P; one that is not there is zeros
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int row = q * 16 + xr;
                            const uint32_t bytes = row < left ? (uint32_t)xbytes : 0u;
                            cp_async_16(st + xdst + q * 2048, bytes ? x + rows[row] * pr.ldx : pr.x, bytes);
                        }
                        if (pr0 < pstep) {
#pragma unroll 4
                            for (int row = pr0; row < 64; row += pstep)
                                cp_async_16(st + pdst + row * 128 + (((pc & 7) ^ (row & 7)) << 4),
                                            row < left ? parts + rows[row] * ldp : pr.parts, row < left ? 16u : 0u);
                        }
                    }
                }
                cp_async_commit();
                if (c >= GR_AHEAD) {
                    cp_async_wait<GR_AHEAD>();
                    tc::fence_proxy_async_smem();
                    mbar_arrive(smem_u32(&sh.full[(it + c - GR_AHEAD) % nst]));
                }
            }
            it += stages;
        } else if (lane == 0) {
            for (int c = 0; c < stages && ok; ++c, ++it) {
                const uint32_t s = it % nst, st = ring + s * stage_bytes;
                if (!(ok = mbar_wait(smem_u32(&sh.full[s]), (it / nst) & 1, kWaitGradMma))) break;
                tc::fence_after_sync();
                const uint64_t dx = tc::desc_mnmajor_sw128(st, TC_M_BYTES / 2);
                const uint64_t dp = tc::desc_mnmajor_sw128(st + TC_M_BYTES, TC_M_BYTES / 2);
                const uint32_t idesc = tc::idesc_bf16(TC_M, 2 * nrank, true, true);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    tc::mma_bf16(tmem, dx + (uint64_t)(q * 128), dp + (uint64_t)(q * 128), idesc, acc);
                    acc = 1;
                }
                tc::commit(smem_u32(&sh.empty[s]));
            }
        }
        __syncwarp();
    }
    if (warp == GR_WARPS && lane == 0) tc::commit(smem_u32(&sh.acc));
    if (warp < GR_WARPS) {
        mbar_wait(smem_u32(&sh.acc), 0, kWaitGradAcc);
        tc::fence_after_sync();
        const int quad = warp & 3, f = f0 + quad * 32 + lane;   // two warps to 32 features, each half of the ranks
        const bool any = it > 0;
        const long long line = (long long)id * a.r + r0;
        const int rm = (nr + 15) / 16 * 8, re = warp < 4 ? min(nr, rm) : nr;
        for (int r = warp < 4 ? 0 : rm; r < re; r += 8) {
            uint32_t hi[8], lo[8];
            __syncwarp();
            tc::ld_32x32b_x8(tmem + r + ((uint32_t)(quad * 32) << 16), hi);
            tc::ld_32x32b_x8(tmem + nrank + r + ((uint32_t)(quad * 32) << 16), lo);
            tc::wait_ld();
            if (f >= pr.k) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (r + i >= nr || !SG_IN(id < a.l && r0 + r + i < a.r)) continue;
                // (an infinity comes from the high parts, with their sign: the low ones may have the other)
                const float h = __uint_as_float(hi[i]), v = !any ? 0.f : fabsf(h) < INFINITY ? h + __uint_as_float(lo[i]) : h;
                if (a.splits > 1)
                    pr.ws[((long long)blockIdx.y * a.l * a.r + line + r + i) * pr.k + f] = v;
                else
                    pr.g[(line + r + i) * pr.k + f] = __float2bfloat16_rn(v);
            }
        }
        tc::fence_before_sync();
    }
    __syncthreads();
    if (warp == GR_WARPS) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 128);
    }
}

}  // namespace lora
}  // namespace sgemm_gb300
