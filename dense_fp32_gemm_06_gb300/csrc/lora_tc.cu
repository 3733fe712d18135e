// Tile choice, tensor maps and launches of the tensor-core projection.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "adapters_units.h"

namespace sgemm_gb300 {
namespace units {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 g_encode_tiled = nullptr;

}  // namespace

cudaError_t lora_map(CUtensorMap *map, const void *base, int rank, long long d0, long long d1, long long d2,
                     long long pitch, long long plane, int b0, int b1) {
    const cuuint64_t dims[3] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2};
    const cuuint64_t strides[2] = {(cuuint64_t)pitch * 2, (cuuint64_t)plane * 2};
    const cuuint32_t box[3] = {(cuuint32_t)b0, (cuuint32_t)b1, 1};
    const cuuint32_t one[3] = {1, 1, 1};
    const CUresult r = g_encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base),
                                      dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

template <int BN, bool W_MN, bool PAIR = false>
cudaError_t attr() {
    return cudaFuncSetAttribute(lora::project_tc_kernel<BN, W_MN, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                lora::tc_smem_bytes(PAIR ? BN / 2 : BN));
}

template <int BN, bool PAIR = false>
cudaError_t launch(const cudaLaunchConfig_t &cfg, bool w_mn, const CUtensorMap *m, const lora::TcArgs &a) {
    return w_mn ? cudaLaunchKernelEx(&cfg, lora::project_tc_kernel<BN, true, PAIR>, m[0], m[1], m[2], a)
                : cudaLaunchKernelEx(&cfg, lora::project_tc_kernel<BN, false, PAIR>, m[0], m[1], m[2], a);
}

}  // namespace

cudaError_t lora_tc_setup(int sms, TcDevice *d) {
    cudaError_t e;
    if (g_encode_tiled == nullptr) {
        cudaDriverEntryPointQueryResult q;
        void *fn = nullptr;
        e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || fn == nullptr)
            return e != cudaSuccess ? e : cudaErrorSymbolNotFound;
        g_encode_tiled = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    cudaError_t (*const attrs[])() = {attr<16, false>, attr<16, true>, attr<32, false>, attr<32, true>, attr<64, false>,
                                      attr<64, true>, attr<128, false>, attr<128, true>, attr<256, false>, attr<256, true>, attr<256, false, true>, attr<256, true, true>};
    for (auto f : attrs)
        if ((e = f()) != cudaSuccess) return e;
    d->sms = sms;
    for (int s = 2; s <= 8; ++s) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(s * 64), 1, 1);
        cfg.blockDim = dim3((unsigned)lora::TC_THREADS, 1, 1);
        cfg.dynamicSmemBytes = (size_t)lora::tc_smem_bytes(16);
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)s;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&d->clusters[s], lora::project_tc_kernel<16, false, false>, &cfg)) != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

// The rows' tile and the split of the contraction that an estimate of the
// time prefers: per stage the larger of the MMA's cycles (2 BN) and the
// stage's bytes at ~64 bytes a cycle, per tile a start and a drain, per
// cluster its exchange.  Within 5 % of the best choice where all were timed but
// for 384 x 1024 x 1024 (9.2 us, best 8.0).
TcPlan lora_tc_plan(int t, int n, int k, const TcDevice &d) {
    const long long tiles_n = ((long long)n + lora::TC_M - 1) / lora::TC_M;
    const int nk = (k + lora::TC_K - 1) / lora::TC_K;
    TcPlan best = {256, 1, false};
    double best_cost = 1e300;
    for (int bn = 16; bn <= 256; bn *= 2) {
        const long long tiles = tiles_n * (((long long)t + bn - 1) / bn);
        const double stage = 2.0 * bn > lora::tc_stage_bytes(bn) / 64.0 ? 2.0 * bn : lora::tc_stage_bytes(bn) / 64.0;
        for (int s = 1; s <= 8; ++s) {
            if (s > 1 && (tiles > d.clusters[s] || nk < 2 * s)) continue;
            const long long waves = s > 1 ? 1 : (tiles + d.sms - 1) / d.sms;
            const double cost = (double)waves * ((nk + s - 1) / s) * stage + 1500.0 + 4.0 * bn + (s > 1 ? 1500.0 + 12.0 * bn : 0.0);
            if (cost < best_cost) {
                best_cost = cost;
                best = {bn, s, false};
            }
        }
        if (bn >= t) break;
    }
    best.pair = best.split == 1 && best.bn == 256;
    return best;
}

TcGrid lora_tc_grid(const TcPlan &p, int t, int n, const TcDevice &d) {
    const int m_tile = p.pair ? 2 * lora::TC_M : lora::TC_M;
    TcGrid g;
    g.tiles_n = (int)(((long long)n + m_tile - 1) / m_tile);
    g.tiles_t = (int)(((long long)t + p.bn - 1) / p.bn);
    g.tiles = (long long)g.tiles_n * g.tiles_t;
    const long long fit = d.sms / (p.pair ? 2 : 1);
    g.clusters = p.split > 1 || g.tiles < fit ? g.tiles : fit;
    return g;
}

cudaError_t lora_project(const lora::TcArgs &args, bool w_mn, const TcDevice &d, bool after_shrink, cudaStream_t s) {
    lora::TcArgs a = args;
    const TcPlan p = lora_tc_plan(a.t, a.n, a.k, d);
    const int ctas = p.pair ? 2 : p.split;   // of a cluster
    const TcGrid g = lora_tc_grid(p, a.t, a.n, d);
    const int x_rows = p.pair ? p.bn / 2 : p.bn;
    a.tiles_n = g.tiles_n;
    a.tiles_t = g.tiles_t;
    a.group = p.pair ? 8 : 16;
    CUtensorMap m[3] = {};
    cudaError_t e = w_mn ? lora_map(&m[0], a.w, 2, a.n, a.k, 1, a.ldw, 0, 64, lora::TC_K)
                         : lora_map(&m[0], a.w, 2, a.k, a.n, 1, a.ldw, 0, lora::TC_K, lora::TC_M);
    if (e == cudaSuccess) e = lora_map(&m[1], a.x, 2, a.k, a.t, 1, a.ldx, 0, lora::TC_K, x_rows);
    if (e == cudaSuccess && a.l > 0 && a.r > 0)
        e = lora_map(&m[2], a.e, 3, a.n, a.r, a.l, a.lde, (long long)a.r * a.lde, 64, lora::ext_rows(a.r));
    if (e != cudaSuccess) return e;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(g.clusters * ctas), 1, 1);
    cfg.blockDim = dim3((unsigned)lora::TC_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)lora::tc_smem_bytes(x_rows);
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
    if (after_shrink) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    switch (p.bn) {
        case 16: return launch<16>(cfg, w_mn, m, a);
        case 32: return launch<32>(cfg, w_mn, m, a);
        case 64: return launch<64>(cfg, w_mn, m, a);
        case 128: return launch<128>(cfg, w_mn, m, a);
        default: return p.pair ? launch<256, true>(cfg, w_mn, m, a) : launch<256>(cfg, w_mn, m, a);
    }
}

cudaError_t lora_tc_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300
