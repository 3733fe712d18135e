// Tile choice, tensor maps and launches of the products of 4-bit matrices.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "mx_units.h"

namespace sgemm_gb300 {
namespace units {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 g_encode_tiled = nullptr;

}  // namespace

cudaError_t mx_map(CUtensorMap *map, CUtensorMapDataType type, int size, const void *base, long long inner, long long rows,
                   long long pitch, int b0, int b1, bool swizzle) {
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)pitch};
    const cuuint32_t box[2] = {(cuuint32_t)b0, (cuuint32_t)b1}, one[2] = {1, 1};
    const CUtensorMapSwizzle sw = !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : b0 * size == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    const CUresult r = g_encode_tiled(map, type, 2, const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t mx_map3(CUtensorMap *map, const void *base, long long inner, long long rows, int planes, long long pitch, long long plane, int b0, int b1) {
    const cuuint64_t dims[3] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)plane * 2};
    const cuuint32_t box[3] = {(cuuint32_t)b0, (cuuint32_t)b1, 1}, one[3] = {1, 1, 1};
    const CUresult r = g_encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, one,
                                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

template <int BN, bool F32, bool PAIR = false, bool FUSED = false>
cudaError_t attr() {
    return cudaFuncSetAttribute(mx::mx4_kernel<BN, F32, PAIR, FUSED>, cudaFuncAttributeMaxDynamicSharedMemorySize, mx::m4_smem_bytes(BN, PAIR));
}

template <int BN, bool F32, bool PAIR = false, bool FUSED = false>
cudaError_t launch(const cudaLaunchConfig_t &cfg, const CUtensorMap *m, const mx::M4Args &a) {
    return cudaLaunchKernelEx(&cfg, mx::mx4_kernel<BN, F32, PAIR, FUSED>, m[0], m[1], m[2], m[3], a);
}

}  // namespace

// The rows' tile and the split of the contraction that an estimate of the time
// prefers: per stage the larger of the MMA's cycles (2 BN) and the stage's
// bytes at ~64 bytes a cycle, per tile a start and a drain, per cluster its
// exchange.  Of 40 sizes with all choices timed (17 to 8192 rows, k and n of 300 to
// 30000) the one taken was within 5 % of the best, but for 257 x 1500 x 1000 (6 %) and
// 300 x 1024 x 1024 (9 %, 0.4 us).
MxPlan mx4_plan(int t, int n, int nk, bool f32, const MxDevice &d) {
    const long long tiles_n = ((long long)n + mx::TC_M - 1) / mx::TC_M;
    const int nu = (nk + 1) / 2;
    MxPlan best = {16, 1, false};
    double best_cost = 1e300;
    for (int bn = 16; bn <= (f32 ? 128 : 256); bn *= 2) {
        // CTA pairs (0), and 1 to 8 CTAs that split the contraction
        for (int s = 0; s <= 8; ++s) {
            const bool pair = s == 0;
            if (pair ? bn < 128 : bn == 256 && s == 1) continue;
            const long long tiles = (pair ? (tiles_n + 1) / 2 : tiles_n) * (((long long)t + bn - 1) / bn), fit = pair ? d.sms / 2 : d.sms;
            const int split = pair ? 1 : s;
            if (split > 1 && (tiles > d.clusters[s] || nu < s)) continue;
            const double bytes = (double)mx::m4_stage_bytes(pair ? bn / 2 : bn) / 64.0, stage = 2.0 * bn > bytes ? 2.0 * bn : bytes;
            const long long waves = split > 1 ? 1 : (tiles + fit - 1) / fit;
            const double cost = (double)waves * (2 * ((nu + split - 1) / split) * stage + 800.0 + (bn == 256 ? 2.0 * bn : 0.0)) + 700.0 + 4.0 * bn + (pair ? 700.0 : 0.0) + (split > 1 ? 1000.0 + 8.0 * bn : 0.0);
            if (cost < best_cost) {
                best_cost = cost;
                best = {bn, split, pair};
            }
        }
        if (bn >= t) break;
    }
    return best;
}

// Its tiles, and the clusters that take them: one each, or as many as fit and
// each takes tiles in turn.
MxGrid mx_grid(const MxPlan &p, int rows, int features, const MxDevice &d) {
    const int m_tile = p.pair ? 2 * mx::TC_M : mx::TC_M;
    MxGrid g;
    g.tiles_f = (int)(((long long)features + m_tile - 1) / m_tile);
    g.tiles_r = (int)(((long long)rows + p.bn - 1) / p.bn);
    g.tiles = (long long)g.tiles_f * g.tiles_r;
    const long long fit = d.sms / (p.pair ? 2 : 1);
    g.clusters = p.split > 1 || g.tiles < fit ? g.tiles : fit;
    return g;
}

// A CTA that quantises X's rows itself does so in each of its stages: a batch of
// four rows takes ~0.15 us (FP32: 0.2) of it, of which 0.33 us are hidden behind the
// stage's bytes of W; a launch of the quantiser costs ~2 us.  Of 112 calls timed both
// ways (1 to 16 rows, k and n of 1024 to 16384, both types, one after the other and in
// a graph) the way taken was within 4 % of the better: 16 x 8192 x 8192 13.5 us in two
// launches, 14.8 fused (FP32 13.2 and 17.9), 12 rows 13.3 and 12.8, one row 12.9 and 10.8.
bool mx4_fused(int t, int n, int blocks, bool f32, const MxDevice &d) {
    const int batches = (t + mx::M4_ROWS - 1) / mx::M4_ROWS, nk = blocks / 8 + (blocks % 8 != 0);
    if (t > MX4_FUSED_ROWS) return false;
    const double more = batches * (f32 ? 0.2 : 0.15) - 0.33;
    if (more <= 0) return true;
    const MxPlan p = mx4_plan(t, n, nk, f32, d);
    const MxGrid g = mx_grid(p, t, n, d);
    return (double)((g.tiles + g.clusters - 1) / g.clusters) * ((nk + p.split - 1) / p.split) * more <= 2.0;
}

size_t mx_sums_bytes(const MxPlan &p, int rows, int features, long long stages, int deep, const MxDevice &d) {
    return stages <= deep ? 0 : mx::sums_of(mx_grid(p, rows, features, d).clusters * (p.pair ? 2 : p.split), p.bn) * sizeof(float);
}

size_t mx4_sums_bytes(int t, int n, int blocks, bool f32, const MxDevice &d) {
    const int nk = blocks / 8 + (blocks % 8 != 0), nu = (nk + 1) / 2;
    if (f32 || nk <= mx::M4_DEEP) return 0;
    const MxPlan p = mx4_plan(t, n, nk, f32, d);
    return mx_sums_bytes(p, t, n, 2 * ((nu + p.split - 1) / p.split), mx::M4_DEEP, d);
}

cudaError_t mx4_setup(int sms, MxDevice *d) {
    cudaError_t e;
    if (g_encode_tiled == nullptr) {
        cudaDriverEntryPointQueryResult q;
        void *fn = nullptr;
        e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || fn == nullptr) return e != cudaSuccess ? e : cudaErrorSymbolNotFound;
        g_encode_tiled = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    cudaError_t (*const attrs[])() = {attr<16, false>, attr<16, true>, attr<32, false>, attr<32, true>, attr<64, false>, attr<64, true>,
                                      attr<128, false>, attr<128, true>, attr<128, false, true>, attr<128, true, true>, attr<256, false>, attr<256, false, true>, attr<16, false, false, true>, attr<16, true, false, true>};
    for (auto f : attrs)
        if ((e = f()) != cudaSuccess) return e;
    d->sms = sms;
    for (int s = 2; s <= 8; ++s) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(s * 64), 1, 1);
        cfg.blockDim = dim3((unsigned)mx::M4_THREADS, 1, 1);
        cfg.dynamicSmemBytes = (size_t)mx::m4_smem_bytes(128, false);   // one CTA an SM
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)s;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&d->clusters[s], mx::mx4_kernel<128, false, false, false>, &cfg)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t mx4_product(const mx::M4Args &args, bool f32, const MxDevice &d, cudaStream_t s) {
    mx::M4Args a = args;
    const int t = a.out.rows, n = a.out.cols, nk = (a.blocks + 7) / 8;
    const MxPlan p = mx4_plan(t, n, nk, f32, d);
    const MxGrid g = mx_grid(p, t, n, d);
    const int ctas = p.pair ? 2 : p.split, x_rows = p.pair ? p.bn / 2 : p.bn;
    a.tiles_n = g.tiles_f;
    a.tiles_t = g.tiles_r;
    a.group = p.pair ? 8 : 16;
    CUtensorMap m[4] = {};
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    cudaError_t e = mx_map(&m[0], u8, 1, a.w, (long long)a.blocks * 16, n, a.ldw, mx::M4_K / 2, mx::TC_M, true);
    const bool fused = a.real != nullptr;
    if (e == cudaSuccess && !fused) e = mx_map(&m[1], u8, 1, a.x, (long long)a.blocks * 16, t, a.ldx, mx::M4_K / 2, x_rows, true);
    if (e == cudaSuccess) e = mx_map(&m[2], u8, 1, a.ws, a.blocks, n, a.ldws, 16, mx::TC_M, false);
    if (e == cudaSuccess && !fused) e = mx_map(&m[3], u8, 1, a.xs, a.blocks, t, a.ldxs, 16, p.bn < 128 ? p.bn : 128, false);
    if (e != cudaSuccess) return e;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(g.clusters * ctas), 1, 1);
    cfg.blockDim = dim3((unsigned)(mx::M4_THREADS + (fused ? mx::M4_FUSED : 0)), 1, 1);
    cfg.dynamicSmemBytes = (size_t)mx::m4_smem_bytes(p.bn, p.pair);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    unsigned na = 0;
    if (ctas > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = (unsigned)ctas;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    cfg.attrs = attr;
    cfg.numAttrs = na;
    if (fused) return f32 ? launch<16, true, false, true>(cfg, m, a) : launch<16, false, false, true>(cfg, m, a);
    switch (p.bn) {
        case 16: return f32 ? launch<16, true>(cfg, m, a) : launch<16, false>(cfg, m, a);
        case 32: return f32 ? launch<32, true>(cfg, m, a) : launch<32, false>(cfg, m, a);
        case 64: return f32 ? launch<64, true>(cfg, m, a) : launch<64, false>(cfg, m, a);
        case 128:
            if (p.pair) return f32 ? launch<128, true, true>(cfg, m, a) : launch<128, false, true>(cfg, m, a);
            return f32 ? launch<128, true>(cfg, m, a) : launch<128, false>(cfg, m, a);
        default: return p.pair ? launch<256, false, true>(cfg, m, a) : launch<256, false>(cfg, m, a);
    }
}

cudaError_t mx4_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300
