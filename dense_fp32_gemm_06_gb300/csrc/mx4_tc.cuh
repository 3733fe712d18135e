// Y = X^ W^^T of two matrices in 4 bits on the tensor cores (kind::mxf4: exact
// products, the two blocks' powers of two applied by the tensor core, FP32
// accumulators).
//
// One MMA tile is 128 features (the operand M, from W) by BN rows of X (the
// operand N), so that few rows cost few columns.  Codes come by TMA as they
// lie, 256 of a row in a 128-byte line.  The scales of 512 values of a row are
// 16 bytes; TMA brings those of 128 rows as 16-byte lines, a warp turns them
// into the order that the copies to tensor memory read (512 bytes are the
// scales of 128 rows by 128 values: four bytes of row 32 c + l at line l, word
// c), in place, and the MMA's thread copies them beside the accumulators.
//
// FUSED: up to 16 rows of X come as real values.  Every CTA quantises its part
// of them itself, eight warps four rows by 256 values each in turn, into the
// lines and scales that TMA would have brought: one launch, nothing in memory in
// between, where that takes less than two (mx4_fused).  Calls of 4096 x 4096, us,
// against two launches: 1 row 5.5 / 7.3, 16 rows 6.3 / 7.3; of 8192 x 8192: 1 row 10.8 / 12.9,
// 12 rows 12.8 / 13.3, 16 rows 14.8 / 13.5 (two are taken); 32 rows (4096) 9.9 / 8.0.
//
// PAIR: two CTAs share 256 features by 256 or 128 rows, each brings its half of both
// (and all of the rows' scales) and drains its own features.
//
// FP32 results: the tensor core truncates its sum once per MMA, so accumulators
// are taken out every 1024 values and added in registers.
//
// What bounds it, with one GB300's times.  8192^3: the power limit (1357 W at
// 1.76 GHz) and the tensor pipe, 159 to 165 us (6.9 PFLOP/s; 14 tiles a pair of 32 stages of
// 512 cycles are 130 us at that clock; the rest is each tile's drain, which the
// single accumulator does not hide, and starts).  (224 rows a tile leave room for
// two accumulators, but took 163: an MMA of 224 rows is no faster than one of 256.)
// FP32 results: tiles of 128 rows, 8192^3 275 us; bfloat16 results in such tiles take
// 250.  In copies of the kernel the promotions are 18 of the 275, the stores 12, and
// without X's loads it is no faster: a stage of 128 rows takes ~550 cycles whatever is
// beside it, one of 256 rows ~640 with its share of the drain.  2048^3 9.9, 128 tiles for
// 76 pairs.  Few rows: latency; 64 x 4096 x 4096 5.9 us where W's bytes need 1.4.
#pragma once
#include <type_traits>

#include <cuda.h>

#include "mx_drain.cuh"
#include "mx_store.cuh"
#include "tcgen05_mx4.cuh"

namespace sgemm_gb300 {
namespace mx {

constexpr int M4_K = 256;         // values of a row in a stage
constexpr int M4_UNIT = 512;      // and in a unit of scales: two stages
constexpr int M4_THREADS = 384;   // TMA, MMA, 8 draining warps, the scales' order, TMA of the scales
constexpr int M4_FUSED = 256;     // and where X is quantised: threads, and rows at a time
constexpr int M4_ROWS = 4;
constexpr int M4_SEGMENT = 4;     // stages between two promotions of an FP32 result
constexpr int M4_DEEP = MOST_MMAS / (M4_K / 64);   // the same of a bfloat16 one
constexpr int M4_A_BYTES = TC_M * M4_K / 2;

// rows of X in a CTA's shared memory: codes, and scales in whole 128s.  (Rings of
// half that for few rows let two CTAs share an SM, and the next call start beside
// this one's end; but CTAs of one call then shared SMs too: 64 x 4096 x 4096 took
// 7.4 us a call, 5.9 so.)
__host__ __device__ constexpr int m4_stages(int xr) { return xr >= 256 ? 4 : xr == 128 ? 6 : xr == 64 ? 8 : xr == 32 ? 9 : 10; }
__host__ __device__ constexpr int m4_stage_bytes(int xr) { return M4_A_BYTES + xr * (M4_K / 2); }
__host__ __device__ constexpr int m4_units(int xr) { return xr == 16 ? 8 : m4_stages(xr) / 2 + 1; }
__host__ __device__ constexpr int m4_blocks(int bn) { return 1 + (bn + 127) / 128; }   // groups of 128 rows of scales
__host__ __device__ constexpr int m4_unit_bytes(int bn) { return m4_blocks(bn) * 2048; }

struct M4Shared {
    uint64_t full[10], empty[10];
    uint64_t raw[8], scaled[8], used[8];   // a unit's scales: as they lie, in the copies' order, read
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tmem;
};
__host__ __device__ constexpr int m4_smem_bytes(int bn, bool pair) {
    const int xr = pair ? bn / 2 : bn;
    return 1024 + m4_stages(xr) * m4_stage_bytes(xr) + m4_units(xr) * m4_unit_bytes(bn) + (int)sizeof(M4Shared);
}

struct M4Args {
    Out out;
    int blocks;               // of a row
    int tiles_n, tiles_t, group;
    const uint8_t *x, *xs, *w, *ws;   // as the maps address them
    long long ldx, ldxs, ldw, ldws;
    const void *real;                 // (FUSED) X, out.rows x k, its pitch, and whether rows start at multiples of 16 bytes
    long long ldr;
    int k;
    bool vec;
    float *sums;                      // (bfloat16 results of more than M4_DEEP stages) sums_of the launch
};

constexpr int kWait4Producer = 0x221, kWait4Mma = 0x222, kWait4Acc = 0x223, kWait4Scales = 0x224, kWait4Quantiser = 0x225;

template <int BN, bool F32, bool PAIR, bool FUSED>
__global__ void __launch_bounds__(M4_THREADS + (FUSED ? M4_FUSED : 0), 1)
    mx4_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
               const __grid_constant__ CUtensorMap map_ws, const __grid_constant__ CUtensorMap map_xs, const M4Args a) {
    constexpr int XR = PAIR ? BN / 2 : BN;
    constexpr int STAGES = m4_stages(XR), STAGE = m4_stage_bytes(XR), UNITS = m4_units(XR), UNIT = m4_unit_bytes(BN);
    constexpr int CTAS = PAIR ? 2 : 1, GROUPS = m4_blocks(BN);
    constexpr int ACCS = BN == 256 ? 1 : 2;
    constexpr uint32_t SCALES = ACCS * BN;                       // first column of the scales, two stages' in turn
    constexpr uint32_t USED = SCALES + 2 * 2 * GROUPS * 4;
    constexpr uint32_t COLS = USED <= 64 ? 64 : USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
    constexpr int QUANTISERS = FUSED ? M4_FUSED : 0, THREADS = M4_THREADS + QUANTISERS;
    static_assert(USED <= 512, "tensor memory");
    static_assert(!FUSED || (BN == 16 && !PAIR), "one tile of rows");
    static_assert(!F32 || BN <= 128, "an FP32 tile is summed in registers");
    static_assert(PAIR || BN * TC_M * 4 <= STAGES * STAGE, "a split tile's floats lie in the ring");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
    const uint32_t units = ring + STAGES * STAGE;
    uint8_t *units_ptr = ring_ptr + STAGES * STAGE;
    M4Shared &sh = *reinterpret_cast<M4Shared *>(units_ptr + UNITS * UNIT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = (int)tc::cluster_ctarank(), cluster = (int)tc::cluster_nctarank();
    const int rank = PAIR ? 0 : crank, nsplit = PAIR ? 1 : cluster;
    const int half = PAIR ? crank : 0;
    const bool leads = half == 0;
    // a row's stages; a CTA that shares a tile's contraction takes whole units of them
    const int nk_all = (a.blocks + 7) / 8, nu_all = (nk_all + 1) / 2;
    const int kb = 2 * (int)((long long)nu_all * rank / nsplit);
    const int nk = min(2 * (int)((long long)nu_all * (rank + 1) / nsplit), nk_all) - kb;
    const int tiles = a.tiles_n * a.tiles_t, step = (int)gridDim.x / cluster, first = (int)blockIdx.x / cluster;
    constexpr int per_seg = F32 ? M4_SEGMENT : M4_DEEP;
    const int segs = (nk + per_seg - 1) / per_seg;
    auto lead = [&](const uint64_t &bar) { return PAIR ? tc::map_shared_rank(smem_u32(&bar), 0) : smem_u32(&bar); };

    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_ws);
        if (!FUSED) {
            tma_prefetch_desc(&map_x);
            tma_prefetch_desc(&map_xs);
        }
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1 + (FUSED ? (a.out.rows + M4_ROWS - 1) / M4_ROWS : 0));   // TMA's bytes, and X's rows
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < UNITS; ++i) {
            mbar_init(smem_u32(&sh.raw[i]), 1);
            mbar_init(smem_u32(&sh.scaled[i]), CTAS);
            mbar_init(smem_u32(&sh.used[i]), 1);
        }
        for (int i = 0; i < ACCS; ++i) {
            mbar_init(smem_u32(&sh.acc_full[i]), 1);
            mbar_init(smem_u32(&sh.acc_empty[i]), 8 * CTAS);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        if (PAIR) {
            tc::tmem_alloc_pair(smem_u32(&sh.tmem), COLS);
            tc::tmem_relinquish_pair();
        } else {
            tc::tmem_alloc(smem_u32(&sh.tmem), COLS);
            tc::tmem_relinquish();
        }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (PAIR) tc::cluster_sync();   // the other CTA's barriers exist
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sh.tmem;
    griddep_launch_dependents();
    griddep_wait();   // X's codes, or W's, may come from the kernel in front of this one

    if (warp == 0) {
        auto load_2d = [&](uint32_t dst, const void *m, int x, int y, uint32_t bar) {
            if (PAIR) tc::tma_load_2d_pair(dst, m, x, y, bar);
            else tma_load_2d(dst, m, x, y, bar);
        };
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                int tf, tt;
                raster_tile(tile, a.tiles_n, a.tiles_t, a.group, tf, tt);
                const int f0 = (tf * CTAS + half) * TC_M, t0 = tt * BN;
                for (int k = 0; k < nk; ++k, ++it) {
                    const uint32_t s = it % STAGES, st = ring + s * STAGE, bar = lead(sh.full[s]);
                    if (!(ok = mbar_wait(smem_u32(&sh.empty[s]), ((it / STAGES) & 1) ^ 1, kWait4Producer))) break;
                    if (leads) mbar_arrive_expect_tx(smem_u32(&sh.full[s]), FUSED ? M4_A_BYTES : CTAS * STAGE);
                    const int kx = (kb + k) * (M4_K / 2);
                    load_2d(st, &map_w, kx, f0, bar);
                    if (!FUSED) load_2d(st + M4_A_BYTES, &map_x, kx, t0 + half * XR, bar);
                }
            }
        }
    } else if (warp == 1) {
        constexpr int M = CTAS * TC_M;
        auto wait = [&](const uint64_t &bar, uint32_t parity) {
            return PAIR ? mbar_wait_cluster(smem_u32(&bar), parity, kWait4Mma) : mbar_wait(smem_u32(&bar), parity, kWait4Mma);
        };
        auto commit = [&](const uint64_t &bar) {
            if (PAIR) tc::commit_pair(smem_u32(&bar), 3);
            else tc::commit(smem_u32(&bar));
        };
        if (leads) {
            uint32_t it = 0, un = 0, seq = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                for (int k = 0; k < nk; ++k, ++it) {
                    const uint32_t b = seq % ACCS, d = tmem + b * BN, u = un % UNITS, s = it % STAGES, st = ring + s * STAGE;
                    const bool opens = k % per_seg == 0, closes = k % per_seg == per_seg - 1 || k == nk - 1, ends = k % 2 == 1 || k == nk - 1;
                    if (opens) ok = wait(sh.acc_empty[b], ((seq / ACCS) & 1) ^ 1);
                    if (k % 2 == 0) ok = ok && wait(sh.scaled[u], (un / UNITS) & 1);
                    ok = ok && wait(sh.full[s], (it / STAGES) & 1);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t cols = tmem + SCALES + (it & 1) * (2 * GROUPS * 4);
                    const uint64_t dw = tc::desc_kmajor_sw128(st), dx = tc::desc_kmajor_sw128(st + M4_A_BYTES);
                    const uint64_t ds = tc::desc_scales(units + u * UNIT + (k & 1) * 1024);   // the words of this half of the unit
                    const uint32_t more = !opens;
                    if (elect_one()) {
#pragma unroll
                        for (int w = 0; w < 2; ++w)   // 128 values each
#pragma unroll
                            for (int g = 0; g < GROUPS; ++g) tc::copy_scales<PAIR>(cols + (w * GROUPS + g) * 4, ds + (uint64_t)((g * 2048 + w * 512) >> 4));
#pragma unroll
                        for (int q = 0; q < M4_K / 64; ++q) {
                            const uint32_t sc = cols + (q / 2) * GROUPS * 4;
                            tc::mma_mx4<PAIR>(d, dw + (uint64_t)(q * 2), dx + (uint64_t)(q * 2), tc::idesc_mx4(M, BN, (q & 1) * 2), sc, sc + 4, q > 0 ? 1 : more);
                        }
                        commit(sh.empty[s]);
                        if (ends) commit(sh.used[u]);
                        if (closes) commit(sh.acc_full[b]);
                    }
                    __syncwarp();
                    un += ends;
                    seq += closes;
                }
            }
        }
    } else if (warp < 10) {
        // two warps to a quarter of the tensor-memory lanes, half of the columns each
        constexpr int NC = BN / 2;
        const int quad = warp & 3, c0 = (warp - 2) / 4 * NC;
        uint32_t seq = 0;
        auto acquire = [&](uint32_t &at) {
            const uint32_t b = seq % ACCS;
            const bool ok = mbar_wait(smem_u32(&sh.acc_full[b]), (seq / ACCS) & 1, kWait4Acc);
            tc::fence_after_sync();
            at = tmem + b * BN + c0 + ((uint32_t)(quad * 32) << 16);
            return __all_sync(0xffffffffu, ok) != 0;
        };
        auto release = [&]() {
            const uint32_t b = seq++ % ACCS;
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) mbar_arrive_peer(lead(sh.acc_empty[b]));
                else mbar_arrive(smem_u32(&sh.acc_empty[b]));
            }
        };
        float *stage = reinterpret_cast<float *>(ring_ptr) + c0 * TC_M + quad * 32 + lane;
        auto each = [&](auto &&drain_tile) {
            for (int tile = first; tile < tiles; tile += step) {
                int tf, tt;
                raster_tile(tile, a.tiles_n, a.tiles_t, a.group, tf, tt);
                if (!drain_tile((long long)tt * BN + c0, (tf * CTAS + half) * TC_M + quad * 32 + lane)) break;
            }
        };
        if (F32 || segs == 1)
            each([&](long long t, int f) { return drain<NC, F32, 1, false>(a.out, segs, !PAIR && nsplit > 1, stage, t, f, acquire, release); });
        else
            each([&](long long t, int f) {
                float *sums = a.sums + sums_of(blockIdx.x, BN) + c0 * TC_M + quad * 32 + lane;
                return drain_deep<NC, false>(a.out, segs, !PAIR && nsplit > 1, stage, sums, t, f, acquire, release);
            });
    } else if (warp == 10) {
        uint32_t un = 0;
        bool ok = true;
        const int nu = (nk + 1) / 2;
        for (int tile = first; tile < tiles && ok; tile += step)
            for (int i = 0; i < nu; ++i, ++un) {
                const uint32_t u = un % UNITS;
                ok = mbar_wait(smem_u32(&sh.raw[u]), (un / UNITS) & 1, kWait4Scales);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                // line l of word w: bytes 4 w .. 4 w + 3 of rows l, 32 + l, 64 + l and 96 + l
#pragma unroll
                for (int g = 0; g < (FUSED ? 1 : GROUPS); ++g) {
                    uint4 *at = reinterpret_cast<uint4 *>(units_ptr + u * UNIT + g * 2048) + lane;
                    const uint4 r0 = at[0], r1 = at[32], r2 = at[64], r3 = at[96];
                    __syncwarp();
                    at[0] = make_uint4(r0.x, r1.x, r2.x, r3.x);
                    at[32] = make_uint4(r0.y, r1.y, r2.y, r3.y);
                    at[64] = make_uint4(r0.z, r1.z, r2.z, r3.z);
                    at[96] = make_uint4(r0.w, r1.w, r2.w, r3.w);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) mbar_arrive_peer(lead(sh.scaled[u]));
                    else mbar_arrive(smem_u32(&sh.scaled[u]));
                }
            }
    } else if (warp == 11) {
        // in a thread of its own: the scales' way to the MMA is longer than the codes'
        if (lane == 0) {
            constexpr int SR = BN < 128 ? BN : 128;   // rows of a box of X's scales
            uint32_t un = 0;
            bool ok = true;
            const int nu = (nk + 1) / 2;
            for (int tile = first; tile < tiles && ok; tile += step) {
                int tf, tt;
                raster_tile(tile, a.tiles_n, a.tiles_t, a.group, tf, tt);
                const int f0 = (tf * CTAS + half) * TC_M, t0 = tt * BN;
                for (int i = 0; i < nu; ++i, ++un) {
                    const uint32_t u = un % UNITS, at = units + u * UNIT, bar = smem_u32(&sh.raw[u]);
                    if (!(ok = mbar_wait(smem_u32(&sh.used[u]), ((un / UNITS) & 1) ^ 1, kWait4Producer))) break;
                    mbar_arrive_expect_tx(bar, 2048 + (FUSED ? 0 : (GROUPS - 1) * SR * 16));
                    const int sx = (kb / 2 + i) * 16;
                    tma_load_2d(at, &map_ws, sx, f0, bar);
#pragma unroll
                    for (int g = 1; g < GROUPS && !FUSED; ++g) tma_load_2d(at + g * 2048, &map_xs, sx, t0 + (g - 1) * 128, bar);
                }
            }
        }
    } else if constexpr (FUSED) {
        using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
        // Batches of R rows by a stage, counted over all tiles, go round the warps.
        // A warp waits for the slots of its own batches' stages alone, at most WARPS
        // stages (units, where a tile has one stage) apart: with rings as long, the
        // use of a slot before the last one has always been seen to end, and a
        // parity names one phase.
        constexpr int WARPS = QUANTISERS / 32, R = M4_ROWS;
        static_assert(STAGES >= WARPS && UNITS >= WARPS, "rings as long as the round of the warps");
        const int rows = a.out.rows, batches = (rows + R - 1) / R, nu = (nk + 1) / 2, blk = lane >> 2;
        const Source<T> x = {static_cast<const T *>(a.real), a.ldr, rows, a.k, a.vec};
        auto at = [&](int k, int row) { return x.row(min(row, rows - 1)) + (kb + k) * M4_K + lane * 8; };
        // the loads of a whole stage of aligned rows come ahead, others where they are needed
        auto whole = [&](int k) { return a.vec && (kb + k) * M4_K <= a.k - M4_K; };
        Raw<T> next[R];
        auto fetch = [&](uint32_t n) {
            const int k = (int)(n / batches % nk), row = (int)(n % batches) * R;
            if (whole(k)) {
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (SG_IN(x.has(at(k, row + i), 8))) next[i].load(at(k, row + i));
            }
        };
        uint32_t n = warp - M4_THREADS / 32;
        fetch(n);
        for (;; n += WARPS) {
            const uint32_t it = n / batches, seq = it / nk;   // the stage among all tiles', the tile among the CTA's
            if (first + (long long)seq * step >= tiles) break;
            const int k = (int)(it - seq * nk), row = (int)(n % batches) * R;
            const uint32_t un = seq * nu + k / 2, s = it % STAGES, u = un % UNITS;
            Raw<T> now[R];
#pragma unroll
            for (int i = 0; i < R; ++i) now[i] = next[i];
            fetch(n + WARPS);
            uint32_t codes[R], bytes[R];
            const bool ahead = whole(k);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float f[8];
                if (ahead) now[i].unpack(f);
                else load8(x, min(row + i, rows - 1), (kb + k) * M4_K + lane * 8, f);
                uint32_t m = largest_bits(f);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                bytes[i] = scale_byte<4>(m);
                codes[i] = codes_of<4>(f, bytes[i]).x;
            }
            bool ok = mbar_wait(smem_u32(&sh.used[u]), ((un / UNITS) & 1) ^ 1, kWait4Quantiser);
            ok = ok && mbar_wait(smem_u32(&sh.empty[s]), ((it / STAGES) & 1) ^ 1, kWait4Quantiser);
            if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll
            for (int i = 0; i < R; ++i) {   // (rows that do not exist: columns that no one reads)
                const int r = row + i, word = ((k & 1) * 2 + (blk >> 2)) * 512 + r * 16 + (blk & 3);
                if (!SG_IN(r < XR && 2048 + word < UNIT)) continue;
                *reinterpret_cast<uint32_t *>(ring_ptr + s * STAGE + M4_A_BYTES + r * 128 + ((blk ^ (r & 7)) << 4) + (lane & 3) * 4) = codes[i];
                if ((lane & 3) == 0) units_ptr[u * UNIT + 2048 + word] = (uint8_t)bytes[i];
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.full[s]));
        }
    }

    __syncwarp();
    if (!PAIR && nsplit > 1) {
        int tf, tt;
        raster_tile(first, a.tiles_n, a.tiles_t, a.group, tf, tt);
        if constexpr (F32) join_split<float, THREADS>(a.out, ring, BN, (long long)tt * BN, tf * TC_M, rank, nsplit);
        else join_split<__nv_bfloat16, THREADS>(a.out, ring, BN, (long long)tt * BN, tf * TC_M, rank, nsplit);
    }
    tc::fence_before_sync();
    if (PAIR) tc::cluster_sync();   // neither CTA leaves while the other's MMA, copies or arrivals may reach it
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        if (PAIR) tc::tmem_dealloc_pair(tmem, COLS);
        else tc::tmem_dealloc(tmem, COLS);
    }
}

}  // namespace mx
}  // namespace sgemm_gb300
