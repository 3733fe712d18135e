// The instances and launches of the adapters' CUDA-core products.
#include "adapters_units.h"

namespace sgemm_gb300 {
namespace units {

namespace {

template <class T>
cudaError_t shrink_type(const lora::ShrinkArgs &a, int sms, cudaStream_t s) {
    const int groups = (a.r + 3) / 4;
    // a row and four ranks per CTA up to a few waves: the same time as tiles of
    // eight rows where those share an adapter (684 x 2624, rank 16, whole call:
    // 64 against 66 us), less where they do not (77 against 111)
    if ((long long)a.t * groups <= 32LL * sms) {
        const dim3 grid((unsigned)a.t, (unsigned)groups);
        const long long es = (long long)sizeof(T);
        if (a.ldx * es % 16 == 0 && a.lds * es % 16 == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 &&
            (reinterpret_cast<uintptr_t>(a.s) & 15) == 0)
            return launch_early(lora::shrink_row_kernel<T, true>, grid, lora::SHRINK_THREADS, 0, a, s);
        return launch_early(lora::shrink_row_kernel<T, false>, grid, lora::SHRINK_THREADS, 0, a, s);
    }
    const dim3 grid((unsigned)(((long long)a.t + lora::SHRINK_ROWS - 1) / lora::SHRINK_ROWS));
    auto tile = [&](auto *vec, auto *any) { return launch_early(a.vec ? vec : any, grid, lora::SHRINK_THREADS, 0, a, s); };
    if (groups >= 8)
        return tile(lora::shrink_tile_kernel<T, 1, true>, lora::shrink_tile_kernel<T, 1, false>);
    if (groups >= 4)
        return tile(lora::shrink_tile_kernel<T, 2, true>, lora::shrink_tile_kernel<T, 2, false>);
    if (groups >= 2)
        return tile(lora::shrink_tile_kernel<T, 4, true>, lora::shrink_tile_kernel<T, 4, false>);
    return tile(lora::shrink_tile_kernel<T, 8, true>, lora::shrink_tile_kernel<T, 8, false>);
}

}  // namespace

cudaError_t lora_shrink(const lora::ShrinkArgs &a, int dtype, int sms, cudaStream_t s) {
    return dtype == ADAPTERS_F32 ? shrink_type<float>(a, sms, s) : shrink_type<__nv_bfloat16>(a, sms, s);
}

cudaError_t lora_expand(const lora::ExpandArgs &a, cudaStream_t s) {
    const dim3 grid((unsigned)(((long long)a.t + lora::EXPAND_ROWS - 1) / lora::EXPAND_ROWS),
                    (unsigned)(((long long)a.n + 4 * lora::EXPAND_THREADS - 1) / (4 * lora::EXPAND_THREADS)));
    return launch_early(a.vec ? lora::expand_kernel<true> : lora::expand_kernel<false>, grid, lora::EXPAND_THREADS, 0, a, s);
}

namespace {

constexpr int few_smem(int rows) { return lora::FEW_STAGES * (lora::FEW_W + rows * lora::FEW_K) * 4; }

template <int ROWS, bool W_MN>
cudaError_t few_attr() {
    return cudaFuncSetAttribute(lora::few_rows_kernel<ROWS, W_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem(ROWS));
}

template <int ROWS, bool W_MN>
cudaError_t launch_few(const lora::FewArgs &a, int sms, bool after_shrink, cudaStream_t s) {
    static_assert(few_smem(ROWS) >= 4 * ROWS * lora::FEW_COLS * 4, "the groups' sums");
    // CTAs along k until two or three occupy each SM, each keeping eight stages
    const long long tiles = ((long long)a.n + lora::FEW_COLS - 1) / lora::FEW_COLS, blocks = ((long long)a.t + ROWS - 1) / ROWS;
    const int nk = (a.k + lora::FEW_K - 1) / lora::FEW_K;
    int split = 1;
    while (split < 8 && tiles * blocks * split * 2 <= 3LL * sms && nk >= 16 * split) split *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * split), (unsigned)blocks, 1);
    cfg.blockDim = dim3((unsigned)lora::FEW_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)few_smem(ROWS);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_shrink ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, lora::few_rows_kernel<ROWS, W_MN>, a);
}

template <bool W_MN>
cudaError_t few_rows(const lora::FewArgs &a, int sms, bool after_shrink, cudaStream_t s) {
    if (a.t == 1) return launch_few<1, W_MN>(a, sms, after_shrink, s);
    if (a.t <= 4) return launch_few<4, W_MN>(a, sms, after_shrink, s);
    if (a.t <= 8) return launch_few<8, W_MN>(a, sms, after_shrink, s);
    return launch_few<16, W_MN>(a, sms, after_shrink, s);
}

}  // namespace

cudaError_t lora_simt_setup() {
    cudaError_t (*const attrs[])() = {few_attr<1, false>, few_attr<1, true>, few_attr<4, false>, few_attr<4, true>,
                                      few_attr<8, false>, few_attr<8, true>, few_attr<16, false>, few_attr<16, true>};
    for (auto f : attrs) {
        const cudaError_t e = f();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t lora_few_rows(const lora::FewArgs &a, bool w_mn, int sms, bool after_shrink, cudaStream_t s) {
    return w_mn ? few_rows<true>(a, sms, after_shrink, s) : few_rows<false>(a, sms, after_shrink, s);
}

// Parts the rows are cut into so that the gradients' CTAs (two to an SM)
// occupy the device; none when adapters, columns and ranks do already, and
// no part below a quarter of a window.
int lora_grad_splits(int t, int ka, int kb, int l, int r, int sms) {
    const long long cols = ((long long)ka + lora::GRAD_COLS - 1) / lora::GRAD_COLS + ((long long)kb + lora::GRAD_COLS - 1) / lora::GRAD_COLS;
    const long long ctas = cols * l * ((r + lora::GRAD_RANKS - 1) / lora::GRAD_RANKS);
    long long s = (2LL * sms + ctas - 1) / (ctas > 0 ? ctas : 1);
    if (s > t / 256) s = t / 256;
    return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}

cudaError_t lora_grad(const lora::GradArgs &a, cudaStream_t s) {
    const int rblocks = (a.r + lora::GRAD_RANKS - 1) / lora::GRAD_RANKS;
    const int cols = (a.of[0].k + lora::GRAD_COLS - 1) / lora::GRAD_COLS + (a.of[1].k + lora::GRAD_COLS - 1) / lora::GRAD_COLS;
    const cudaError_t e = launch_early(a.vec ? lora::grad_kernel<true> : lora::grad_kernel<false>,
                                       dim3((unsigned)((long long)a.l * rblocks * cols), (unsigned)a.splits), lora::GRAD_THREADS, 0, a, s);
    if (e == cudaSuccess && a.splits > 1) {
        lora::GradSumArgs<float> b = {{a.of[0].ws, a.of[1].ws}, {a.of[0].g, a.of[1].g},
                                      {(long long)a.l * a.r * a.of[0].k, (long long)a.l * a.r * a.of[1].k}, a.splits};
        return launch_early(lora::grad_sum_kernel<float>, dim3((unsigned)((b.count[0] + b.count[1] + 255) / 256)), 256, 0, b, s);
    }
    return e;
}

cudaError_t lora_pad_rows(const lora::PadArgs &a, int sms, cudaStream_t s) {
    long long blocks = 1;
    for (int i = 0; i < a.jobs; ++i)
        if ((a.job[i].rows + 7) / 8 > blocks) blocks = (a.job[i].rows + 7) / 8;
    if (blocks > 8LL * sms) blocks = 8LL * sms;
    return launch_early(lora::pad_rows_kernel, dim3((unsigned)blocks), 256, 0, a, s);
}

cudaError_t lora_simt_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300
