// Launches of the adapters' skinny products on the tensor cores.
#include <cuda.h>

#include "adapters_units.h"

namespace sgemm_gb300 {
namespace units {

cudaError_t lora_skinny_setup() {
    cudaError_t e = cudaFuncSetAttribute(lora::shrink_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, lora::SH_SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(lora::grad_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 lora::gr_smem(32) > lora::gr_smem(64) ? lora::gr_smem(32) : lora::gr_smem(64));
    return e;
}

cudaError_t lora_shrink_tc(const lora::ShrinkArgs &g, void *parts, const TcDevice &d, cudaStream_t s) {
    // CTAs along k: as many as the device takes (two to an SM), each keeping
    // at least four stages
    const long long tiles = ((long long)g.t + lora::SH_BN - 1) / lora::SH_BN;
    const int nk = (g.k + lora::TC_K - 1) / lora::TC_K;
    int split = 1;
    // and CTAs that share out the passes of a tile, as many as there can be
    const int per = g.r >= 128 ? 1 : 128 / ((g.r + 7) / 8 * 8);
    const long long passes = ((long long)(g.l < lora::SH_BN ? g.l : lora::SH_BN) + per - 1) / per * ((g.r + 127) / 128);
    while (split < 8 && tiles * split * 2 <= 2LL * d.sms && nk >= 8 * split) split *= 2;
    long long share = 2LL * d.sms / (tiles * split);
    if (share > passes) share = passes;
    if (share < 1) share = 1;
    CUtensorMap m[2] = {};
    const int rows = g.r >= 128 ? 128 : (g.r + 7) / 8 * 8;
    cudaError_t e = lora_map(&m[0], g.s, 3, g.k, g.r, g.l, g.lds, (long long)g.r * g.lds, lora::TC_K, rows);
    if (e == cudaSuccess) e = lora_map(&m[1], g.x, 2, g.k, g.t, 1, g.ldx, 0, lora::TC_K, lora::SH_BN);
    if (e != cudaSuccess) return e;
    lora::ShrinkTcArgs a = {g.t, g.k, g.l, g.r, g.ids, g.scale, g.h, static_cast<__nv_bfloat16 *>(parts)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * split), (unsigned)share, 1);
    cfg.blockDim = dim3((unsigned)lora::SH_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)lora::SH_SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, lora::shrink_tc_kernel, m[0], m[1], a);
}

size_t lora_parts_bytes(int t, int r) { return (size_t)t * lora::gr_blocks(r) * lora::gr_ranks(r) * 4; }

cudaError_t lora_parts(const float *p, void *parts, int t, int r, cudaStream_t s) {
    const long long n = (long long)t * lora::gr_blocks(r) * lora::gr_ranks(r);
    const lora::PartsArgs a = {p, static_cast<__nv_bfloat16 *>(parts), t, r};
    return launch_early(lora::parts_kernel, dim3((unsigned)((n + 255) / 256)), 256, 0, a, s);
}

// Parts of the rows: none while adapters, ranks and features make two CTAs to
// an SM, and never below 256 rows.
int lora_grad_tc_splits(int t, int ka, int kb, int l, int r, int sms) {
    const long long tiles = ((long long)ka + lora::TC_M - 1) / lora::TC_M + ((long long)kb + lora::TC_M - 1) / lora::TC_M;
    const long long ctas = tiles * l * lora::gr_blocks(r);
    long long s = 2LL * sms / (ctas > 0 ? ctas : 1);
    if (s > t / 256) s = t / 256;
    return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}

cudaError_t lora_grad_tc(const lora::GradTcArgs &a, cudaStream_t s) {
    const int tiles = (a.of[0].k + lora::TC_M - 1) / lora::TC_M + (a.of[1].k + lora::TC_M - 1) / lora::TC_M;
    const dim3 grid((unsigned)((long long)a.l * lora::gr_blocks(a.r) * tiles), (unsigned)a.splits);   // (the other axes end at 65535)
    const cudaError_t e = launch_early(lora::grad_tc_kernel, grid, lora::GR_THREADS, (size_t)lora::gr_smem(a.r), a, s);
    if (e == cudaSuccess && a.splits > 1) {
        lora::GradSumArgs<__nv_bfloat16> b = {{a.of[0].ws, a.of[1].ws}, {a.of[0].g, a.of[1].g},
                                              {(long long)a.l * a.r * a.of[0].k, (long long)a.l * a.r * a.of[1].k}, a.splits};
        return launch_early(lora::grad_sum_kernel<__nv_bfloat16>, dim3((unsigned)((b.count[0] + b.count[1] + 255) / 256)), 256, 0, b, s);
    }
    return e;
}

cudaError_t lora_skinny_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300
