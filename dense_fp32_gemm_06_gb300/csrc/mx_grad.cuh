// The gradients of a projection beside a microscaled matrix, on the tensor
// cores:
//
//     out[p][c] (+)= sum_r dY[p][r] M^[r][c]
//
// dX = dY W^ (p a token, r a feature) and dW = dY^T X^ (p a feature, r a
// token: dY as stored is transposed).  M^'s codes run along c, which is not
// contracted, so no scaled MMA can read them: a scale would have to belong to
// 32 values of r.  But every value code 2^e is a bfloat16 number, so M^ is
// decoded on its way and the products are exact.
//
// One MMA tile is 128 columns c (the operand M) by BN rows p (the operand N,
// dY's, by TMA as it lies), 64 values of r a stage.  64 lines of 128 codes and
// their scales come by TMA into a ring of their own; two groups of four warps
// take every second stage each.  A warp has one block's 32 columns: it reads the
// codes transposed (ldmatrix), four values of r of a column a word, decodes them
// and stores them to tensor memory, where the MMA reads its operand M, columns at
// the lanes.  (Decoded into shared memory, the 16 KB written and read again a
// stage, three times by FP32's planes, were what bound the kernel: 8192 x 4096 x
// 4096 in 8 bits took 193 us, 185 so, FP32 2048^3 47, 42.5 so then.)  PAIR: two CTAs
// share 256 columns by BN rows, each decodes its own half (64 rows of FP32 that way:
// 256 x 4096 x 4096 28.1 us, 32.6 by a CTA each, 33.6 as pairs' 128).
//
// What bounds it, with one GB300's times.  Large sizes: the power limit (1354 W at
// 1.73 GHz; 8192 x 4096 x 4096 in 4 bits 159 us, 1725 TFLOP/s, in 8 bits 167, both
// of dY as stored; transposed 171 and 170) and CTAs without a last tile (256 tiles
// on 76 pairs).  Tiles of 128 rows or less: the decoding (~500 cycles a stage, many of
// them masks and byte permutes) and the loads (~390); 512 x 4096 x 4096 21.9 us.
// (Codes read a stage ahead of their decoding: 1024 x 4096 x 4096 27.6 us against
// 24.8.)  FP32 2048^3: the three planes' MMAs, 28 of 31 us, behind 7 us that make the
// planes.  Few rows: latency (16 x 4096 x 4096 7.8 us).
//
// FP32 gradients come as three bfloat16 planes (hi + mid + lo, all 24 bits),
// which all meet a stage's decoded columns.  The tensor core truncates its sum
// once per MMA, so FP32 accumulators are taken out every 128 values (24 MMAs)
// and added in registers.
#pragma once
#include <type_traits>

#include <cuda.h>

#include "mx_drain.cuh"
#include "mx_store.cuh"

namespace sgemm_gb300 {
namespace mx {

constexpr int G_K = 64;            // contraction per stage
constexpr int G_THREADS = 608;     // TMA of dY, MMA, 8 draining warps, 8 decoding ones, TMA of codes
constexpr int G_GROUPS = 2, G_GROUP_WARPS = 4;
constexpr int G_SEGMENT = 2;       // stages between two promotions of an FP32 result
constexpr int G_DEEP = MOST_MMAS / (G_K / 16);   // the same of a bfloat16 one
constexpr int G_A_COLS = G_K / 2;  // of tensor memory, a stage's decoded columns

__host__ __device__ constexpr int g_code_bytes(int bits) { return TC_M * G_K * bits / 8; }
__host__ __device__ constexpr int g_raw_bytes(int bits) { return g_code_bytes(bits) + G_K * 16; }   // codes, scales
// rows of dY in a CTA's shared memory, in whole boxes where TMA brings boxes of 64
__host__ __device__ constexpr int g_x_bytes(int xr) { return (xr < 64 ? xr : (xr + 63) / 64 * 64) * G_K * 2; }
__host__ __device__ constexpr int g_stage_bytes(int xr, bool f32) { return (f32 ? 3 : 1) * g_x_bytes(xr); }
// slots of the two rings, of dY beside the decoded columns and of the codes: even,
// so that each group of decoders sees every use of its own slots (a barrier's
// parity names a phase to those alone)
__host__ __device__ constexpr int g_stages(bool f32) { return f32 ? 6 : 8; }
constexpr int G_RAWS = 8;

struct GShared {
    uint64_t full[8], empty[8];
    uint64_t raw_full[G_RAWS], raw_empty[G_RAWS];
    uint64_t acc_full[2], acc_empty[2];
    uint16_t scale[G_GROUPS * G_GROUP_WARPS][G_K];   // a decoding warp's scales as bfloat16 values
    uint32_t tmem;
};
__host__ __device__ constexpr int g_smem_bytes(int bn, bool pair, int bits, bool f32) {
    const int xr = pair ? bn / 2 : bn;
    return 1024 + g_stages(f32) * g_stage_bytes(xr, f32) + G_RAWS * g_raw_bytes(bits) + (int)sizeof(GShared);
}

struct GradArgs {
    Out out;
    int depth;                // of the contraction
    int tiles_c, tiles_p, group;
    float *sums;              // (bfloat16 results of more than G_DEEP stages) sums_of the launch
};

constexpr int kWaitGProducer = 0x231, kWaitGMma = 0x232, kWaitGAcc = 0x233, kWaitGDecoder = 0x234;

// A scale as a bfloat16 value: byte 0 is a subnormal, 255 NaN.
__device__ __forceinline__ uint32_t scale_bf16(uint32_t byte) { return byte == 0 ? 0x0040u : byte == NOT_FINITE ? 0x7fc0u : byte << 7; }
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;\n" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// Four bytes of consecutive r, each two 4-bit codes, as bfloat16 pairs of r times
// the scales' pairs: of the low codes and of the high ones.  The three bits of a
// magnitude in bfloat16's last exponent bits and first mantissa bit are the
// magnitude 2^-126, subnormal 0.5 among them.  A scale times 2^126 is a bfloat16
// number up to byte 128 (SMALL: `scale` is that product), else the two multiply
// one after the other; each product is exact.
template <bool SMALL>
__device__ __forceinline__ void decode4(uint32_t w, const uint2 &scale, uint32_t *low, uint32_t *high) {
    constexpr uint32_t up = 0x7e807e80u;   // 2^126
    // a nibble times two powers of two is two copies of it, one with the sign in place
    // and one with the magnitude: the multiplications are not the pipe of the
    // shifts and masks, which bounds the decoding (two shifts each: 1024 x 4096 x 4096 25.0 us, 23.9 so)
    const uint32_t lo = w & 0x0f0f0f0fu, hi = w & 0xf0f0f0f0u, s[2] = {scale.x, scale.y};
    const uint32_t p[2] = {__byte_perm(lo, 0, 0x4140), __byte_perm(lo, 0, 0x4342)}, q[2] = {__byte_perm(hi, 0, 0x4140), __byte_perm(hi, 0, 0x4342)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a = p[i] * ((1u << 12) + (1u << 6)) & 0x81c081c0u;
        const uint32_t b = q[i] * ((1u << 8) + (1u << 2)) & 0x81c081c0u;
        low[i] = SMALL ? mul2(a, s[i]) : mul2(mul2(a, up), s[i]);
        high[i] = SMALL ? mul2(b, s[i]) : mul2(mul2(b, up), s[i]);
    }
}

// Four 8-bit codes of consecutive r, the same.  A byte u in bfloat16's low bits is
// u 2^-133, subnormal up to 127 and normal above; with u = code + 128 the difference
// to 128 2^-133 is the code's, here times 2^64.  A scale times 2^69 is a bfloat16
// number up to byte 185 (SMALL), else the two multiply one after the other.  (With the
// sign bits masked and spread by themselves, twice the masks and permutes: 8192 x 4096 x
// 4096 184 us, 170 so.)
template <bool SMALL>
__device__ __forceinline__ void decode8(uint32_t w, const uint2 &scale, uint32_t *out) {
    constexpr uint32_t up = 0x5f805f80u, middle = 0xa080a080u, rest = 0x62006200u;   // 2^64, -128 2^-69, 2^69
    const uint32_t u = w ^ 0x80808080u, p[2] = {__byte_perm(u, 0, 0x4140), __byte_perm(u, 0, 0x4342)}, s[2] = {scale.x, scale.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t c = fma2(p[i], up, middle);
        out[i] = SMALL ? mul2(c, s[i]) : mul2(mul2(c, rest), s[i]);
    }
}

// The largest scale byte of SMALL, and the power of two in its scales.
__host__ __device__ constexpr uint32_t g_small(int bits) { return bits == 4 ? 128 : 185; }
__host__ __device__ constexpr uint32_t g_small_power(int bits) { return bits == 4 ? 126 : 69; }

// The column of a block that lane i of its quarter of the tensor memory holds:
// 4-bit codes' low ones (even columns) are at the first 16 lanes.
template <int BITS>
__device__ __forceinline__ int column_of(int i) {
    return BITS == 4 ? (i & 15) * 2 + (i >> 4) : i;
}

// TRANSPOSED: dY is stored r x p.  F32: promoted sums, FP32 output.
template <int BN, int BITS, bool TRANSPOSED, bool F32, bool PAIR>
__global__ void __launch_bounds__(G_THREADS, 1)
    grad_kernel(const __grid_constant__ CUtensorMap map_codes, const __grid_constant__ CUtensorMap map_scales,
                const __grid_constant__ CUtensorMap map_dy, const GradArgs a) {
    constexpr int XR = PAIR ? BN / 2 : BN;   // rows p in this CTA's shared memory
    constexpr int STAGES = g_stages(F32), STAGE = g_stage_bytes(XR, F32), CTAS = PAIR ? 2 : 1, PLANES = F32 ? 3 : 1;
    constexpr int RAWS = G_RAWS, RAW = g_raw_bytes(BITS), SCALES_AT = g_code_bytes(BITS);
    static_assert(STAGES % G_GROUPS == 0 && RAWS % G_GROUPS == 0, "a group sees every use of its slots");
    // tensor memory: one or two accumulators, and the decoded columns of the stages
    constexpr int ACCS = BN == 256 ? 1 : 2;
    constexpr uint32_t COLS = 512, A_AT = ACCS * BN;
    static_assert(A_AT + STAGES * G_A_COLS <= COLS, "tensor memory");
    constexpr int BOXES = (XR + 63) / 64, X_BYTES = (TRANSPOSED ? BOXES * 64 : XR) * G_K * 2;        // of a plane of dY, as TMA brings it
    static_assert(!TRANSPOSED || XR >= 64, "boxes of 64 rows p");
    static_assert(!F32 || BN <= 128, "an FP32 tile is summed in registers");
    static_assert(PAIR || BN * TC_M * 4 <= STAGES * STAGE, "a split tile's floats lie in the ring");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *ring_ptr = smem_raw + (ring - smem_u32(smem_raw));
    const uint32_t raws = ring + STAGES * STAGE;
    uint8_t *raws_ptr = ring_ptr + STAGES * STAGE;
    GShared &sh = *reinterpret_cast<GShared *>(raws_ptr + RAWS * RAW);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = (int)tc::cluster_ctarank(), cluster = (int)tc::cluster_nctarank();
    const int rank = PAIR ? 0 : crank, nsplit = PAIR ? 1 : cluster;
    const int half = PAIR ? crank : 0;
    const bool leads = half == 0;
    // stages; a CTA that shares a tile's contraction takes a run of them
    const long long all = ((long long)a.depth + G_K - 1) / G_K;
    const int kb = (int)(all * rank / nsplit), nk = (int)(all * (rank + 1) / nsplit) - kb;
    const int tiles = a.tiles_c * a.tiles_p, step = (int)gridDim.x / cluster, first = (int)blockIdx.x / cluster;
    constexpr int per_seg = F32 ? G_SEGMENT : G_DEEP;
    const int segs = (nk + per_seg - 1) / per_seg;
    auto lead = [&](const uint64_t &bar) { return PAIR ? tc::map_shared_rank(smem_u32(&bar), 0) : smem_u32(&bar); };

    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&map_codes);
        tma_prefetch_desc(&map_scales);
        tma_prefetch_desc(&map_dy);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1 + CTAS * G_GROUP_WARPS);   // TMA's bytes, and a group's decoding warps of each CTA
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < RAWS; ++i) {
            mbar_init(smem_u32(&sh.raw_full[i]), 1);
            mbar_init(smem_u32(&sh.raw_empty[i]), G_GROUP_WARPS);
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
    griddep_wait();   // dY's planes may come from the kernel in front of this one

    if (warp == 0) {
        auto load_dy = [&](uint32_t dst, int x, int y, int z, uint32_t bar) {
            if (PAIR) tc::tma_load_3d_pair(dst, &map_dy, x, y, z, bar);
            else tma_load_3d(dst, &map_dy, x, y, z, bar);
        };
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                int tcol, tp;
                raster_tile(tile, a.tiles_c, a.tiles_p, a.group, tcol, tp);
                const int p0 = tp * BN + half * XR;
                for (int k = 0; k < nk; ++k, ++it) {
                    const uint32_t s = it % STAGES, bar = lead(sh.full[s]);
                    if (!(ok = mbar_wait(smem_u32(&sh.empty[s]), ((it / STAGES) & 1) ^ 1, kWaitGProducer))) break;
                    if (leads) mbar_arrive_expect_tx(smem_u32(&sh.full[s]), CTAS * PLANES * X_BYTES);
                    const int r0 = (kb + k) * G_K;
#pragma unroll
                    for (int z = 0; z < PLANES; ++z) {
                        const uint32_t at = ring + s * STAGE + z * g_x_bytes(XR);
                        if (TRANSPOSED) {
#pragma unroll
                            for (int i = 0; i < BOXES; ++i) load_dy(at + i * 8192, p0 + i * 64, r0, z, bar);
                        } else {
                            load_dy(at, r0, p0, z, bar);
                        }
                    }
                }
            }
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = tc::idesc_bf16(CTAS * TC_M, BN, false, TRANSPOSED);
        auto wait = [&](const uint64_t &bar, uint32_t parity) {
            return PAIR ? mbar_wait_cluster(smem_u32(&bar), parity, kWaitGMma) : mbar_wait(smem_u32(&bar), parity, kWaitGMma);
        };
        auto commit = [&](const uint64_t &bar) {
            if (PAIR) tc::commit_pair(smem_u32(&bar), 3);
            else tc::commit(smem_u32(&bar));
        };
        if (leads) {
            uint32_t it = 0, seq = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                for (int k = 0; k < nk; ++k, ++it) {
                    const uint32_t b = seq % ACCS, d = tmem + b * BN, s = it % STAGES, st = ring + s * STAGE, m = tmem + A_AT + s * G_A_COLS;
                    const bool opens = k % per_seg == 0, closes = k % per_seg == per_seg - 1 || k == nk - 1;
                    if (opens) ok = wait(sh.acc_empty[b], ((seq / ACCS) & 1) ^ 1);
                    ok = ok && wait(sh.full[s], (it / STAGES) & 1);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint64_t dx = TRANSPOSED ? tc::desc_mnmajor_sw128(st, 8192) : tc::desc_kmajor_sw128(st);
                    constexpr uint64_t plane = g_x_bytes(XR) >> 4;
                    const uint32_t more = !opens;
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < PLANES * (G_K / 16); ++i) {
                            const int q = i / PLANES;
                            const uint64_t x = dx + (uint64_t)(TRANSPOSED ? q * 128 : q * 2) + i % PLANES * plane;
                            if (PAIR) tc::mma_bf16_ts_pair(d, m + q * 8, x, idesc, i > 0 ? 1 : more);
                            else tc::mma_bf16_ts(d, m + q * 8, x, idesc, i > 0 ? 1 : more);
                        }
                        commit(sh.empty[s]);
                        if (closes) commit(sh.acc_full[b]);
                    }
                    __syncwarp();
                    seq += closes;
                }
            }
        }
    } else if (warp < 10) {
        // two warps to a quarter of the tensor-memory lanes, half of the rows p each
        constexpr int NC = BN / 2;
        const int quad = warp & 3, j0 = (warp - 2) / 4 * NC, col = quad * 32 + column_of<BITS>(lane);
        uint32_t seq = 0;
        auto acquire = [&](uint32_t &at) {
            const uint32_t b = seq % ACCS;
            const bool ok = mbar_wait(smem_u32(&sh.acc_full[b]), (seq / ACCS) & 1, kWaitGAcc);
            tc::fence_after_sync();
            at = tmem + b * BN + j0 + ((uint32_t)(quad * 32) << 16);
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
        float *stage = reinterpret_cast<float *>(ring_ptr) + j0 * TC_M + col;
        auto each = [&](auto &&drain_tile) {
            for (int tile = first; tile < tiles; tile += step) {
                int tcol, tp;
                raster_tile(tile, a.tiles_c, a.tiles_p, a.group, tcol, tp);
                if (!drain_tile((long long)tp * BN + j0, (tcol * CTAS + half) * TC_M + col)) break;
            }
        };
        if (F32 || segs == 1)
            each([&](long long p, int c) { return drain<NC, F32, BITS == 4 ? 16 : 1, true>(a.out, segs, !PAIR && nsplit > 1, stage, p, c, acquire, release); });
        else
            each([&](long long p, int c) {
                float *sums = a.sums + sums_of(blockIdx.x, BN) + j0 * TC_M + quad * 32 + lane;
                return drain_deep<NC, true>(a.out, segs, !PAIR && nsplit > 1, stage, sums, p, c, acquire, release);
            });
    } else if (warp == 18) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                int tcol, tp;
                raster_tile(tile, a.tiles_c, a.tiles_p, a.group, tcol, tp);
                const int c0 = (tcol * CTAS + half) * TC_M;
                for (int k = 0; k < nk; ++k, ++it) {
                    const int r0 = (kb + k) * G_K;
                    const uint32_t r = it % RAWS, at = raws + r * RAW, bar = smem_u32(&sh.raw_full[r]);
                    if (!(ok = mbar_wait(smem_u32(&sh.raw_empty[r]), ((it / RAWS) & 1) ^ 1, kWaitGProducer))) break;
                    mbar_arrive_expect_tx(bar, RAW);
                    tma_load_2d(at, &map_codes, c0 / 8 * BITS, r0, bar);
                    tma_load_2d(at + SCALES_AT, &map_scales, c0 / BLOCK & ~15, r0, bar);
                }
            }
        }
    } else {
        const int group = (warp - 10) / G_GROUP_WARPS, quad = warp & 3;   // the lanes, and the tile's block of columns
        uint16_t *const table = sh.scale[warp - 10];
        uint32_t all_it = 0;   // the first stage of a tile
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += step, all_it += nk) {
            int tcol, tp;
            raster_tile(tile, a.tiles_c, a.tiles_p, a.group, tcol, tp);
            const int sc = ((tcol * CTAS + half) * TC_M / BLOCK & 15) + quad;
            for (uint32_t it = all_it + ((all_it ^ (uint32_t)group) & 1); it < all_it + nk; it += G_GROUPS) {
                const uint32_t s = it % STAGES, r = it % RAWS;
                const uint8_t *raw = raws_ptr + r * RAW;
                ok = mbar_wait(smem_u32(&sh.raw_full[r]), (it / RAWS) & 1, kWaitGDecoder);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                const bool in = SG_IN(SCALES_AT + (lane + 32) * 16 + sc < RAW);
                const uint32_t b0 = in ? raw[SCALES_AT + lane * 16 + sc] : 0, b1 = in ? raw[SCALES_AT + (lane + 32) * 16 + sc] : 0;
                const bool small = __all_sync(0xffffffffu, max(b0, b1) <= g_small(BITS));
                table[lane] = (uint16_t)(small ? (b0 + g_small_power(BITS)) << 7 : scale_bf16(b0));
                table[lane + 32] = (uint16_t)(small ? (b1 + g_small_power(BITS)) << 7 : scale_bf16(b1));
                // the block's codes: a 16-byte chunk of each line (8 bits: two), 16 lines a matrix
                constexpr int CHUNKS = BITS / 4;
                uint32_t w[CHUNKS][8], v[2][16];
#pragma unroll
                for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const uint32_t line = g * 32 + lane;
                        const uint32_t chunk = BITS == 4 ? line * 64 + ((quad ^ (line >> 1 & 3)) << 4) : line * 128 + (((quad * 2 + i) ^ (line & 7)) << 4);
                        const uint32_t at = raws + r * RAW + (SG_IN(chunk + 16 <= SCALES_AT) ? chunk : 0);   // (a warp loads as a whole)
                        tc::load_transposed_bytes(at, w[i][4 * g], w[i][4 * g + 1], w[i][4 * g + 2], w[i][4 * g + 3]);
                    }
                __syncwarp();   // the table
                auto decode = [&](auto is_small) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {   // 16 values of r, four of them this lane's
                        const uint2 scale = *reinterpret_cast<const uint2 *>(table + g * 16 + (lane & 3) * 4);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {   // (columns at lanes t / 4 and t / 4 + 8)
                            if constexpr (BITS == 4) {
                                decode4<decltype(is_small)::value>(w[0][2 * g + h], scale, &v[0][4 * g + 2 * h], &v[1][4 * g + 2 * h]);
                            } else {
                                decode8<decltype(is_small)::value>(w[0][2 * g + h], scale, &v[0][4 * g + 2 * h]);
                                decode8<decltype(is_small)::value>(w[CHUNKS - 1][2 * g + h], scale, &v[1][4 * g + 2 * h]);
                            }
                        }
                    }
                };
                if (small) decode(std::true_type{});
                else decode(std::false_type{});
                ok = mbar_wait(smem_u32(&sh.empty[s]), ((it / STAGES) & 1) ^ 1, kWaitGDecoder);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t at = tmem + A_AT + s * G_A_COLS + ((uint32_t)(quad * 32) << 16);
                tc::st_16x256b_x4(at, v[0]);
                tc::st_16x256b_x4(at + (16u << 16), v[1]);
                tc::wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    // (released right behind the loads of the codes, the next ones could come before the
                    // last loads had been made: the stores above needed their values)
                    mbar_arrive(smem_u32(&sh.raw_empty[r]));
                    if (PAIR) mbar_arrive_peer(lead(sh.full[s]));
                    else mbar_arrive(smem_u32(&sh.full[s]));
                }
            }
        }
    }

    __syncwarp();
    if (!PAIR && nsplit > 1) {
        int tcol, tp;
        raster_tile(first, a.tiles_c, a.tiles_p, a.group, tcol, tp);
        if constexpr (F32) join_split<float, G_THREADS>(a.out, ring, BN, (long long)tp * BN, tcol * TC_M, rank, nsplit);
        else join_split<__nv_bfloat16, G_THREADS>(a.out, ring, BN, (long long)tp * BN, tcol * TC_M, rank, nsplit);
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

// An FP32 matrix as three bfloat16 planes, hi + mid + lo = all 24 bits; what
// is not finite is hi alone.  Or a bfloat16 matrix whose rows TMA cannot read
// (a base or pitch that is not a multiple of 16 bytes) as one plane of such rows.
struct PlaneArgs {
    const void *x;
    long long ldx;
    __nv_bfloat16 *planes;
    long long ld, plane;   // elements between rows (a multiple of 8) and planes
    int rows, cols;
    bool vec;
};

constexpr int PLANE_THREADS = 256;

template <class T>
__global__ void __launch_bounds__(PLANE_THREADS) planes_kernel(const PlaneArgs a) {
    __shared__ __align__(16) float lines[PLANE_THREADS / 32][256];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Source<T> m = {static_cast<const T *>(a.x), a.ldx, a.rows, a.cols, a.vec};
    for (Runs at(a.cols / 256 + (a.cols % 256 != 0), PLANE_THREADS / 32); at.row < a.rows; at.next()) {
        const long long row = at.row;
        const int c0 = at.run * 256, c = c0 + lane * 8;
        __align__(16) float f[8];
        if (a.vec) {
            load8(m, row, c, f);
        } else {
            T v[8];
            load_run(m, row, c0, v);
            turn_run(v, lines[warp], f);
        }
        if (c >= a.cols) continue;
        __nv_bfloat16 *to = a.planes + row * a.ld + c;
        if (!SG_IN(row < a.rows && c + 8 <= a.ld)) continue;
        if constexpr (sizeof(T) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = elem::Word<__nv_bfloat16>::pack(f + 2 * i);
            *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            uint4 hi, mid, lo;
            float g[8];
            elem::parts8(f, hi, mid);   // mid: what hi left, rounded; lo: what both left
            float h[8], m[8];
            elem::unpack16<__nv_bfloat16>(hi, h);
            elem::unpack16<__nv_bfloat16>(mid, m);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = fabsf(f[i]) < INFINITY ? (f[i] - h[i]) - m[i] : 0.f;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = elem::Word<__nv_bfloat16>::pack(g + 2 * i);
            lo = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4 *>(to) = hi;
            *reinterpret_cast<uint4 *>(to + a.plane) = mid;
            *reinterpret_cast<uint4 *>(to + 2 * a.plane) = lo;
        }
    }
}

}  // namespace mx
}  // namespace sgemm_gb300
