// The shared projection with the adapters' part in its loop, on the tensor
// cores (bfloat16 matrices, FP32 accumulators):
//
//     Y[t][f] = sum_k X[t][k] W[k][f] + sum_r H[t][r] E[ids[t]][r][f]
//
// One MMA tile is 128 features (the operand M, from W) by BN rows of X (the
// operand N), so that few rows cost few columns: a single token runs the
// same kernel with BN = 16 as a batch of prompts with BN = 256.  W comes as
// stored by TMA, K-major or MN-major.
//
// The adapters extend the contraction.  Each tile of rows lists its distinct
// adapters; behind the stages of X and W follow stages in which the operand M
// is 32 of the listed adapters' rows of E and the operand N a row's H at its
// own adapter's place and zero at the others'.  The accumulator never leaves
// the tensor memory in between, Y is written once, and E is read once per tile
// of rows whatever the mixture.  H is two bfloat16 parts there (elem::parts,
// within 2^-16 of it) that meet the same E.  One part's rounding, 2^-8 of the
// adapters' part, is of the size of Y's own: with it Y was 1.1e-3 to 1.5e-3
// (2-norm) from FP32 products rounded once, with both it is 0.2e-4 to 2e-4, and
// no further than they are from the 64-bit result.
//
// A zero times an infinity is NaN: an adapter that is not finite would reach
// its tile's other rows, and its own rows' parts would meet it with two signs.
// So the listed adapters' values are looked over in shared memory before the
// MMA reads them.  Where one is not finite (or an H) zero takes its place and
// the adapter is marked; to the elements of a marked adapter's own rows the
// drain adds the terms that were left out (`own_terms`).  One adapter of 64 that
// is all NaN makes 64 rows of 4096 x 4096 34 us (27 without, the call alone), one
// of 16 makes 8192^3 923 us (665), one with infinities at every seventh feature
// 1566.
//
// Roles: warp 0 issues TMA loads, warp 1 the MMAs, warps 2-5 look the tile's
// adapters over and drain its accumulator (double-buffered in tensor memory, so
// that one tile's drain runs beside the next tile's loop), warps 6-9 list
// adapters and write H (looking over there too, those 64 rows took 1.5 us more).
// Few tiles are cut along k into the CTAs of a cluster, which add their
// accumulators through distributed shared memory in a fixed order.
//
// What bounds it, with one GB300's times.  Many rows: the tensor pipe and the
// power limit; 8192^3 with rank 32 takes 721 us with its shrink back to back
// (1540 TFLOP/s; 630 in short bursts), 8192 x 4096 x 4096 alone 148 (1860).  Few
// rows: latency; one row of 4096 x 4096 takes 10.5 us a call with its shrink
// where W's bytes need 5, 64 rows with an adapter each 16.3 of 7.6.
#pragma once
#include <cstdint>

#include <cuda.h>

#include "elem.cuh"
#include "raster.cuh"
#include "tcgen05_f16.cuh"

namespace sgemm_gb300 {
namespace lora {

constexpr int TC_M = 128;        // features per tile
constexpr int TC_K = 64;         // contraction per stage
constexpr int TC_THREADS = 320;
constexpr int TC_WRITERS = 128;  // threads of warps 6-9, and of warps 2-5
constexpr int TC_M_BYTES = TC_M * TC_K * 2;

// rows of X per stage and CTA: the tile's, or a pair's half of them
__host__ __device__ constexpr int tc_stages(int bn) { return bn == 256 ? 4 : bn == 128 ? 6 : bn == 64 ? 8 : bn == 32 ? 10 : 11; }
__host__ __device__ constexpr int tc_stage_bytes(int bn) { return TC_M_BYTES + bn * TC_K * 2; }

// shared memory behind the ring
struct TcShared {
    uint64_t full[11], empty[11];
    uint64_t grant[11];      // the producer hands an acquired stage to the writers of H
    uint64_t e_full[11];     // the adapters' values of a stage are here (their bytes), to be looked over
    uint64_t acc_full[2], acc_empty[2];
    uint64_t list_full[2], list_empty[2];
    uint64_t marks[2];       // every H of the tile is written
    uint32_t tmem;
    int count[2];            // distinct adapters of the tile
    int wsum[2][4];
    uint32_t marked[2][8];   // a bit per listed adapter: terms of it were left out of this CTA's products
    int list[2][256];        // their ids
    short slot[2][256];      // a row's place in the list, -1: no adapter
};
__host__ __device__ constexpr int tc_smem_bytes(int bn) { return 1024 + tc_stages(bn) * tc_stage_bytes(bn) + (int)sizeof(TcShared); }

struct TcArgs {
    int t, n, k, l, r;       // rows, features, contraction, adapters, rank (l or r 0: none)
    int tiles_n, tiles_t, group;
    const float *h;
    const int *ids;
    __nv_bfloat16 *y;
    long long ldy;
    // the operands as the maps address them
    const __nv_bfloat16 *x, *w, *e;
    long long ldx, ldw, lde;
};

constexpr int kWaitProducer = 0x211, kWaitMma = 0x212, kWaitAcc = 0x213, kWaitList = 0x214, kWaitWriter = 0x215, kWaitLook = 0x21c;

// The rows of the operand M (values of r) that one adapter takes in a stage:
// r rounded up to the MMA's step of 16, EXT at most.  The operand N has the
// high parts of their H in the stage's first EXT columns, the low ones behind.
constexpr int EXT = TC_K / 2;
__host__ __device__ __forceinline__ int ext_rows(int r) { return r >= EXT ? EXT : (r + 15) / 16 * 16; }

struct Ext {
    int rows, per_stage, chunks;   // rows of an adapter, adapters of a stage, stages of an adapter (r > EXT)
    __device__ __forceinline__ explicit Ext(int r)
        : rows(ext_rows(r)), per_stage(r > 0 ? EXT / ext_rows(r) : 1), chunks((r + EXT - 1) / EXT) {}
    __device__ __forceinline__ int stages(int count) const {
        return chunks > 1 ? count * chunks : (count + per_stage - 1) / per_stage;
    }
    // adapters of stage e and its first one
    __device__ __forceinline__ int first(int e) const { return chunks > 1 ? e / chunks : e * per_stage; }
    __device__ __forceinline__ int adapters(int e, int count) const {
        return chunks > 1 ? 1 : min(per_stage, count - e * per_stage);
    }
};

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// The same, and whether `ok` held for all of them.
__device__ __forceinline__ bool named_barrier_and(int id, int threads, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n"
        ".reg .pred p, q;\n"
        "setp.ne.u32 p, %3, 0;\n"
        "bar.red.and.pred q, %1, %2, p;\n"
        "selp.u32 %0, 1, 0, q;\n"
        "}\n"
        : "=r"(all)
        : "r"(id), "r"(threads), "r"((uint32_t)ok)
        : "memory");
    return all != 0;
}

// The distinct adapters of rows t0 .. t0 + BN - 1 in the order of their first
// rows, and each row's place among them (-1: no adapter); the number of them.
// Whole warps, TC_WRITERS threads (`tid` among them), barrier 1; the lists
// are complete for these threads behind another barrier.
template <int BN>
__device__ __forceinline__ int list_adapters(const int *ids, int l, long long t0, int t, int *list, short *slot, int *wsum,
                                             int tid) {
    const int lane = tid & 31, wl = tid >> 5;
    int count = 0;
    for (int c = 0; c < BN; c += TC_WRITERS) {
        const int i = c + tid;
        int id = -1;
        if (i < BN && t0 + i < t) {
            id = ids[t0 + i];
            if (id >= l) id = -1;
        }
        // rows of a warp with one id: its first lane stands for them, the warps in turn
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        const int leader = __ffs(same) - 1;
        for (int w = 0; w < TC_WRITERS / 32; ++w) {
            if (wl == w) {
                int at = -1;
                if (id >= 0)
                    for (int j = 0; j < count; ++j)
                        if (list[j] == id) at = j;
                __syncwarp();
                const bool leads = id >= 0 && at < 0 && leader == lane;
                const uint32_t lead = __ballot_sync(0xffffffffu, leads);
                if (leads) {
                    at = count + __popc(lead & ((1u << lane) - 1));
                    list[at] = id;
                }
                at = __shfl_sync(0xffffffffu, at, leader);
                if (i < BN) slot[i] = (short)(id >= 0 ? at : -1);
                count += __popc(lead);
                if (lane == 0) wsum[w] = count;
            }
            named_barrier(1, TC_WRITERS);
            count = wsum[w];
        }
    }
    return count;
}

// Whether a magnitude of a bfloat16 word's two values is infinite or NaN.
constexpr uint32_t MAGNITUDES = 0x7fff7fffu;
__device__ __forceinline__ bool not_finite(uint32_t magnitudes) {
    return (magnitudes & 0xffffu) >= 0x7f80u || magnitudes >= 0x7f800000u;
}
__device__ __forceinline__ uint32_t largest(const uint4 &v) {
    return __vmaxu2(__vmaxu2(v.x & MAGNITUDES, v.y & MAGNITUDES), __vmaxu2(v.z & MAGNITUDES, v.w & MAGNITUDES));
}
// Zeros in the place of those.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}
__device__ __forceinline__ uint4 finite_only(const uint4 &v) {
    return make_uint4(finite_only(v.x), finite_only(v.y), finite_only(v.z), finite_only(v.w));
}

// v, and the terms of a row's H and its own adapter's values at a feature (r of
// them, lde apart) that the MMA left out: each is an infinity or NaN, so adding
// one again changes nothing.
static __device__ __noinline__ float own_terms(float v, const __nv_bfloat16 *e, long long lde, const float *h, int r) {
    for (int r0 = 0; r0 < r && v == v; r0 += 8) {   // (eight ranks' loads on their way together)
        float x[8], y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = min(r0 + i, r - 1);
            x[i] = elem::to_f32(e[at * lde]);
            y[i] = h[at];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(fabsf(x[i]) < INFINITY) || !(fabsf(y[i]) < INFINITY)) v = fmaf(y[i], x[i], v);
    }
    return v;
}

// PAIR: the two CTAs of a cluster share a tile of 256 features by 256 rows
// (cta_group::2): each brings its 128 features of W and E and its 128 rows of
// X and H, both count them on the even CTA's barriers, whose MMA reads both
// shared memories, and each drains its own 128 features.  A stage then costs
// each SM 32 KB instead of 48 for the same MMA time.
template <int BN, bool W_MN, bool PAIR>
__global__ void __launch_bounds__(TC_THREADS, 1)
    project_tc_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                      const __grid_constant__ CUtensorMap map_e, const TcArgs a) {
    constexpr int XR = PAIR ? BN / 2 : BN;   // rows of X in this CTA's shared memory
    constexpr int STAGES = tc_stages(XR), STAGE = tc_stage_bytes(XR);
    constexpr int CTAS = PAIR ? 2 : 1;
    constexpr uint32_t COLS = 2 * BN;   // two accumulators
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
    TcShared &sh = *reinterpret_cast<TcShared *>(ring_ptr + STAGES * STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = (int)tc::cluster_ctarank(), cluster = (int)tc::cluster_nctarank();
    const int rank = PAIR ? 0 : crank, nsplit = PAIR ? 1 : cluster;   // of the CTAs along k
    const int half = PAIR ? crank : 0;                                // of the pair
    const bool leads = half == 0;
    const int nk_all = (a.k + TC_K - 1) / TC_K;
    const int kb = (int)((long long)nk_all * rank / nsplit), nk = (int)((long long)nk_all * (rank + 1) / nsplit) - kb;
    const int tiles = a.tiles_n * a.tiles_t, step = (int)gridDim.x / cluster, first = (int)blockIdx.x / cluster;
    const bool adapters = a.l > 0 && a.r > 0;
    const Ext ext(a.r);
    auto mark = [&](int b, int j) { atomicOr(&sh.marked[b][j >> 5], 1u << (j & 31)); };
    // the even CTA's copy of a barrier
    auto lead = [&](const uint64_t &bar) { return PAIR ? tc::map_shared_rank(smem_u32(&bar), 0) : smem_u32(&bar); };

    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_x);
        if (adapters) tma_prefetch_desc(&map_e);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1 + 5 * CTAS);   // TMA's bytes, each CTA's H and its four looks (the producer again where there are none)
            mbar_init(smem_u32(&sh.empty[i]), 1);
            mbar_init(smem_u32(&sh.grant[i]), 1);
            mbar_init(smem_u32(&sh.e_full[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.acc_full[i]), 1);
            mbar_init(smem_u32(&sh.acc_empty[i]), 4 * CTAS);
            mbar_init(smem_u32(&sh.list_full[i]), 1);
            mbar_init(smem_u32(&sh.marks[i]), 1);
            mbar_init(smem_u32(&sh.list_empty[i]), leads ? 6 : 5);   // producer, MMA (the even CTA's), four draining warps
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        if (PAIR) {
            tc::tmem_alloc_pair(smem_u32(&sh.tmem), COLS);
            tc::tmem_relinquish_pair();
        } else {
            tc::tmem_alloc(smem_u32(&sh.tmem), COLS < 32 ? 32 : COLS);
            tc::tmem_relinquish();
        }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (PAIR) tc::cluster_sync();   // the other CTA's barriers exist
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;

    if (warp == 0) {
        auto load_2d = [&](uint32_t dst, const void *m, int x, int y, uint32_t bar) {
            if (PAIR) tc::tma_load_2d_pair(dst, m, x, y, bar);
            else tma_load_2d(dst, m, x, y, bar);
        };
        if (lane == 0) {
            uint32_t it = 0;
            int n = 0;
            for (int tile = first; tile < tiles; tile += step, ++n) {
                int tf, tt;
                raster_tile(tile, a.tiles_n, a.tiles_t, a.group, tf, tt);
                const int f0 = (tf * CTAS + half) * TC_M, t0 = tt * BN + half * XR;
                bool ok = true;
                for (int k = 0; k < nk && ok; ++k, ++it) {
                    const uint32_t s = it % STAGES, st = ring + s * STAGE, bar = lead(sh.full[s]);
                    if (!(ok = mbar_wait(smem_u32(&sh.empty[s]), ((it / STAGES) & 1) ^ 1, kWaitProducer))) break;
                    if (leads) {
                        mbar_arrive_expect_tx(smem_u32(&sh.full[s]), CTAS * STAGE);
                        mbar_arrive_n(smem_u32(&sh.full[s]), 5 * CTAS);
                    }
                    const int kx = (kb + k) * TC_K;
                    if (W_MN) {
                        load_2d(st, &map_w, f0, kx, bar);
                        load_2d(st + TC_M_BYTES / 2, &map_w, f0 + 64, kx, bar);
                    } else {
                        load_2d(st, &map_w, kx, f0, bar);
                    }
                    load_2d(st + TC_M_BYTES, &map_x, kx, t0, bar);
                }
                if (!ok) break;
                if (adapters) {
                    const int b = n & 1;
                    if (!mbar_wait(smem_u32(&sh.list_full[b]), (n >> 1) & 1, kWaitList)) break;
                    const int count = sh.count[b], ne = ext.stages(count);
                    for (int e = rank; e < ne && ok; e += nsplit, ++it) {
                        const uint32_t s = it % STAGES, st = ring + s * STAGE, bar = smem_u32(&sh.e_full[s]);
                        if (!(ok = mbar_wait(smem_u32(&sh.empty[s]), ((it / STAGES) & 1) ^ 1, kWaitProducer))) break;
                        const int j0 = ext.first(e), nj = ext.adapters(e, count);
                        const int r0 = ext.chunks > 1 ? (e % ext.chunks) * EXT : 0;
                        mbar_arrive(smem_u32(&sh.grant[s]));
                        mbar_arrive_expect_tx(bar, (uint32_t)(nj * ext.rows * 256));
                        if (leads) mbar_arrive(smem_u32(&sh.full[s]));
                        for (int j = 0; j < nj; ++j) {
                            const int id = sh.list[b][j0 + j];
                            tma_load_3d(st + j * ext.rows * 128, &map_e, f0, r0, id, bar);
                            tma_load_3d(st + TC_M_BYTES / 2 + j * ext.rows * 128, &map_e, f0 + 64, r0, id, bar);
                        }
                    }
                    mbar_arrive(smem_u32(&sh.list_empty[b]));
                    if (!ok) break;
                }
            }
        }
    } else if (warp == 1) {
        constexpr int M = CTAS * TC_M;
        auto wait = [&](const uint64_t &bar, uint32_t parity) {
            return PAIR ? mbar_wait_cluster(smem_u32(&bar), parity, kWaitMma) : mbar_wait(smem_u32(&bar), parity, kWaitMma);
        };
        auto mma = [&](uint32_t d, uint64_t x, uint64_t y, uint32_t idesc, uint32_t acc) {
            if (PAIR) tc::mma_bf16_pair(d, x, y, idesc, acc);
            else tc::mma_bf16(d, x, y, idesc, acc);
        };
        auto commit = [&](const uint64_t &bar) {
            if (PAIR) tc::commit_pair(smem_u32(&bar), 3);
            else tc::commit(smem_u32(&bar));
        };
        if (lane == 0 && leads) {
            uint32_t it = 0;
            int n = 0;
            for (int tile = first; tile < tiles; tile += step, ++n) {
                const int b = n & 1;
                const uint32_t d = tmem + b * BN;
                uint32_t acc = 0;
                bool ok = wait(sh.acc_empty[b], ((n >> 1) & 1) ^ 1);
                if (!ok) break;
                tc::fence_after_sync();
                for (int k = 0; k < nk; ++k, ++it) {
                    const uint32_t s = it % STAGES, st = ring + s * STAGE;
                    if (!(ok = wait(sh.full[s], (it / STAGES) & 1))) break;
                    tc::fence_after_sync();
                    const uint64_t dw = W_MN ? tc::desc_mnmajor_sw128(st, TC_M_BYTES / 2) : tc::desc_kmajor_sw128(st);
                    const uint64_t dx = tc::desc_kmajor_sw128(st + TC_M_BYTES);
#pragma unroll
                    for (int q = 0; q < TC_K / 16; ++q) {
                        mma(d, dw + (uint64_t)(W_MN ? q * 128 : q * 2), dx + (uint64_t)(q * 2), tc::idesc_bf16(M, BN, W_MN, false), acc);
                        acc = 1;
                    }
                    commit(sh.empty[s]);
                }
                if (!ok) break;
                if (adapters) {
                    if (!mbar_wait(smem_u32(&sh.list_full[b]), (n >> 1) & 1, kWaitList)) break;
                    const int count = sh.count[b], ne = ext.stages(count);
                    for (int e = rank; e < ne; e += nsplit, ++it) {
                        const uint32_t s = it % STAGES, st = ring + s * STAGE;
                        if (!(ok = wait(sh.full[s], (it / STAGES) & 1))) break;
                        tc::fence_after_sync();
                        const uint64_t de = tc::desc_mnmajor_sw128(st, TC_M_BYTES / 2);
                        const uint64_t dh = tc::desc_kmajor_sw128(st + TC_M_BYTES);
                        const int steps = ext.adapters(e, count) * ext.rows / 16;
                        for (int q = 0; q < steps; ++q) {
                            mma(d, de + (uint64_t)(q * 128), dh + (uint64_t)(q * 2), tc::idesc_bf16(M, BN, true, false), acc);
                            mma(d, de + (uint64_t)(q * 128), dh + (uint64_t)(q * 2 + EXT / 8), tc::idesc_bf16(M, BN, true, false), 1);
                            acc = 1;
                        }
                        commit(sh.empty[s]);
                    }
                    mbar_arrive(smem_u32(&sh.list_empty[b]));
                    if (!ok) break;
                }
                commit(sh.acc_full[b]);
            }
        }
    } else if (warp < 6) {
        const int quad = warp & 3;   // the tensor-memory lanes this warp may read
        const int tid = threadIdx.x - 64;
        uint32_t it = 0, looked = 0;   // (as the writers' granted)
        int n = 0;
        for (int tile = first; tile < tiles; tile += step, ++n) {
            int tf, tt;
            raster_tile(tile, a.tiles_n, a.tiles_t, a.group, tf, tt);
            const int b = n & 1;
            bool ok = true;
            if (adapters) {
                ok = mbar_wait(smem_u32(&sh.list_full[b]), (n >> 1) & 1, kWaitList);
                const int count = ok ? sh.count[b] : 0, ne = ext.stages(count);
                it += nk;
                for (int e = rank; e < ne; e += nsplit, ++it) {
                    const uint32_t s = it % STAGES;
                    ok = ok && mbar_wait(smem_u32(&sh.e_full[s]), (looked >> s) & 1, kWaitLook);
                    looked ^= 1u << s;
                    // lines of 16 chunks of 16 bytes, eight in either box of features
                    const int chunks = ok ? ext.adapters(e, count) * ext.rows * 16 : 0;
                    auto chunk = [&](int q) {
                        return reinterpret_cast<uint4 *>(ring_ptr + s * STAGE + (q >> 3 & 1) * (TC_M_BYTES / 2) + (q >> 4) * 128 + ((q & 7) << 4));
                    };
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < EXT * 16 / TC_WRITERS; ++i)
                        if (tid + i * TC_WRITERS < chunks) top = __vmaxu2(top, largest(*chunk(tid + i * TC_WRITERS)));
                    if (not_finite(top)) {
                        for (int q = tid; q < chunks; q += TC_WRITERS) {
                            const uint4 v = *chunk(q);
                            if (!not_finite(largest(v))) continue;
                            mark(b, ext.first(e) + (q >> 4) / ext.rows);
                            *chunk(q) = finite_only(v);
                        }
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (PAIR) mbar_arrive_cluster(lead(sh.full[s]));
                        else mbar_arrive(smem_u32(&sh.full[s]));
                    }
                }
                if (!named_barrier_and(2, TC_WRITERS, ok)) break;   // the marks of all four warps
                ok = mbar_wait(smem_u32(&sh.marks[b]), (n >> 1) & 1, kWaitAcc);
            }
            ok = ok && mbar_wait(smem_u32(&sh.acc_full[b]), (n >> 1) & 1, kWaitAcc);
            if (__any_sync(0xffffffffu, !ok)) break;
            tc::fence_after_sync();
            const int f = (tf * CTAS + half) * TC_M + quad * 32 + lane;
            const long long t0 = (long long)tt * BN;
            uint32_t marked = 0;
            for (int i = 0; adapters && i < 8; ++i) marked |= sh.marked[b][i];
            // all of the warp's features exist and rows of Y hold whole pairs:
            // stores of two features at a time (8192 x 512 x 4096 takes 40 us,
            // with one at a time 78: the drain was longer than the loop)
            const bool whole = (f | 31) < a.n && a.ldy % 2 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 3) == 0;
            constexpr int STEP = BN < 32 ? 16 : 32;
#pragma unroll 1
            for (int c = 0; c < BN; c += STEP) {
                if (t0 + c >= a.t) break;
                __syncwarp();
                uint32_t v[STEP];
                const uint32_t at = tmem + b * BN + c + ((uint32_t)(quad * 32) << 16);
                if constexpr (STEP == 16) tc::ld_32x32b_x16(at, v);
                else tc::ld_32x32b_x32(at, v);
                tc::wait_ld();
                if (marked != 0) {
                    griddep_wait();   // H
#pragma unroll
                    for (int j = 0; j < STEP; ++j) {
                        const int own = sh.slot[b][c + j];
                        if (f < a.n && own >= 0 && (sh.marked[b][own >> 5] >> (own & 31) & 1) != 0)
                            v[j] = __float_as_uint(own_terms(__uint_as_float(v[j]), a.e + (long long)sh.list[b][own] * a.r * a.lde + f, a.lde,
                                                             a.h + (t0 + c + j) * a.r, a.r));
                    }
                }
                if (!PAIR && nsplit > 1) {
                    float *stage = reinterpret_cast<float *>(ring_ptr);
#pragma unroll
                    for (int j = 0; j < STEP; ++j) stage[(c + j) * TC_M + quad * 32 + lane] = __uint_as_float(v[j]);
                }
                if (PAIR || nsplit == 1) {
                    if (whole && t0 + c + STEP <= a.t) {
                        // neighbouring lanes swap every second row, so that each
                        // stores two features of its own rows at a time
                        __syncwarp();
                        const bool odd = lane & 1;
                        __nv_bfloat16 *y = a.y + (t0 + c + odd) * a.ldy + (f & ~1);
#pragma unroll
                        for (int j = 0; j < STEP; j += 2) {
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
                            const float x[2] = {__uint_as_float(odd ? got : v[j]), __uint_as_float(odd ? v[j + 1] : got)};
                            if (SG_IN(f < a.n)) *reinterpret_cast<uint32_t *>(y) = elem::Word<__nv_bfloat16>::pack(x);
                            y += 2 * a.ldy;
                        }
                    } else if (f < a.n) {
                        __nv_bfloat16 *y = a.y + (t0 + c) * a.ldy + f;
                        const int rows = (int)min((long long)STEP, a.t - t0 - c);
#pragma unroll
                        for (int j = 0; j < STEP; ++j) {
                            if (j < rows && SG_IN(f < a.n)) *y = __float2bfloat16_rn(__uint_as_float(v[j]));
                            y += a.ldy;
                        }
                    }
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) mbar_arrive_cluster(lead(sh.acc_empty[b]));
                else mbar_arrive(smem_u32(&sh.acc_empty[b]));
                if (adapters) mbar_arrive(smem_u32(&sh.list_empty[b]));
            }
        }
    } else {
        griddep_wait();   // H may come from the kernel in front of this one
        const int tid = threadIdx.x - 192;
        // A parity names a phase only to a thread that has seen the one before
        // it.  The writers pass over the stages of X and W, so they do not wait
        // on `empty`: each stage's grants are their own to count (one bit).
        uint32_t it = 0, granted = 0;
        constexpr int PLACES = XR * (EXT / 8), BATCH = PLACES >= 4 * TC_WRITERS ? 4 : PLACES > TC_WRITERS ? 2 : 1;
        const bool hvec = a.r % 4 == 0 && (reinterpret_cast<uintptr_t>(a.h) & 15) == 0;
        int n = 0;
        for (int tile = first; adapters && tile < tiles; tile += step, ++n) {
            int tf, tt;
            raster_tile(tile, a.tiles_n, a.tiles_t, a.group, tf, tt);
            const int b = n & 1;
            const long long t0 = (long long)tt * BN;
            bool ok = mbar_wait(smem_u32(&sh.list_empty[b]), ((n >> 1) & 1) ^ 1, kWaitList);
            const int count = list_adapters<BN>(a.ids, a.l, t0, a.t, sh.list[b], sh.slot[b], sh.wsum[b], tid);
            if (tid == 0) sh.count[b] = count;
            if (tid < 8) sh.marked[b][tid] = 0;
            named_barrier(1, TC_WRITERS);
            if (tid == 0) mbar_arrive(smem_u32(&sh.list_full[b]));
            it += nk;
            const int ne = ext.stages(count);
            for (int e = rank; e < ne; e += nsplit, ++it) {
                const uint32_t s = it % STAGES;
                uint8_t *dst = ring_ptr + s * STAGE + TC_M_BYTES;
                const int j0 = ext.first(e), r0 = ext.chunks > 1 ? (e % ext.chunks) * EXT : 0;
                // eight ranks of a row at a time; a batch's loads are on their
                // way together, the first one's before the stage is free
#pragma unroll 1
                for (int q0 = tid; q0 - tid < PLACES; q0 += BATCH * TC_WRITERS) {
                    float x[BATCH][8];
                    int at[BATCH];   // its adapter of the stage, -1: zeros
#pragma unroll
                    for (int u = 0; u < BATCH; ++u) {
                        const int q = q0 + u * TC_WRITERS, row = q / (EXT / 8), ch = q % (EXT / 8), trow = half * XR + row;   // its place in the tile
                        const int j = ch * 8 / ext.rows, r = r0 + ch * 8 - j * ext.rows;
                        at[u] = q < PLACES && j < ext.per_stage && sh.slot[b][trow] == j0 + j ? j : -1;
                        const float *h = a.h + (t0 + trow) * a.r + r;
                        const int left = at[u] >= 0 ? a.r - r : 0;
                        if (hvec) {
                            *reinterpret_cast<float4 *>(x[u]) = elem::fetch4<float, true>(h, left);
                            *reinterpret_cast<float4 *>(x[u] + 4) = elem::fetch4<float, true>(h + 4, left - 4);
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[u][i] = i < left ? h[i] : 0.f;
                        }
                    }
                    if (q0 == tid) ok = ok && mbar_wait(smem_u32(&sh.grant[s]), (granted >> s) & 1, kWaitWriter);
#pragma unroll
                    for (int u = 0; u < BATCH; ++u) {
                        const int q = q0 + u * TC_WRITERS, row = q / (EXT / 8), ch = q % (EXT / 8);
                        if (!ok || q >= PLACES) continue;
                        uint4 hi, lo;
                        elem::parts8(x[u], hi, lo);
                        if (not_finite(largest(hi))) {
                            mark(b, j0 + at[u]);
                            hi = finite_only(hi);
                        }
                        *reinterpret_cast<uint4 *>(dst + row * 128 + ((ch ^ (row & 7)) << 4)) = hi;
                        *reinterpret_cast<uint4 *>(dst + row * 128 + (((ch + EXT / 8) ^ (row & 7)) << 4)) = lo;
                    }
                }
                granted ^= 1u << s;
                __syncwarp();
                tc::fence_proxy_async_smem();
                named_barrier(1, TC_WRITERS);
                if (tid == 0) {
                    if (PAIR) mbar_arrive_cluster(lead(sh.full[s]));
                    else mbar_arrive(smem_u32(&sh.full[s]));
                }
            }
            if (!named_barrier_and(1, TC_WRITERS, ok)) break;
            if (tid == 0) mbar_arrive(smem_u32(&sh.marks[b]));
        }
    }

    __syncwarp();
    if (!PAIR && nsplit > 1) {
        // the ranks' accumulators, added in rank order: each rank writes every nsplit-th row of the tile
        tc::cluster_sync();
        int tf, tt;
        raster_tile(first, a.tiles_n, a.tiles_t, a.group, tf, tt);
        const int f0 = tf * TC_M;
        const long long t0 = (long long)tt * BN;
        const int rows = (int)min((long long)BN, a.t - t0);
        const bool yvec = (reinterpret_cast<uintptr_t>(a.y) & 7) == 0 && a.ldy % 4 == 0;
        for (int q = threadIdx.x;; q += TC_THREADS) {
            const int row = rank + (q >> 5) * nsplit, f = (q & 31) * 4;
            if (row >= rows) break;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t at = ring + (uint32_t)(row * TC_M + f) * 4;
            for (int p = 0; p < nsplit; ++p) {
                const float4 u = tc::ld_cluster_v4(tc::map_shared_rank(at, (uint32_t)p));
                v.x += u.x;
                v.y += u.y;
                v.z += u.z;
                v.w += u.w;
            }
            if (f0 + f >= a.n) continue;
            if (SG_IN(t0 + row < a.t)) elem::store4(a.y + (t0 + row) * a.ldy + f0 + f, v, a.n - f0 - f, yvec);
        }
        tc::cluster_sync();   // no CTA leaves while another reads its shared memory
    }
    tc::fence_before_sync();
    if (PAIR) tc::cluster_sync();   // neither CTA leaves while the other's MMA, copies or arrivals may reach it
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        if (PAIR) tc::tmem_dealloc_pair(tmem, COLS);
        else tc::tmem_dealloc(tmem, COLS < 32 ? 32 : COLS);
    }
}

}  // namespace lora
}  // namespace sgemm_gb300
