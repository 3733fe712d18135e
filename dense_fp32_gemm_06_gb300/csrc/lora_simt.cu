// The instances and launches of the adapters' CUDA-core products.
#include "adapters_units.h"

namespace sgemm_gb300 {
namespace units {

namespace {

template <class T>
void shrink_type(const lora::ShrinkArgs &a, int sms, cudaStream_t s) {
    const int groups = (a.r + 3) / 4;
    // a row and four ranks per CTA while that is a few waves at most
    if ((long long)a.t * groups <= 8LL * sms) {
        const dim3 grid((unsigned)a.t, (unsigned)groups);
        const long long es = (long long)sizeof(T);
        if (a.ldx * es % 16 == 0 && a.lds * es % 16 == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 &&
            (reinterpret_cast<uintptr_t>(a.s) & 15) == 0)
            lora::shrink_row_kernel<T, true><<<grid, lora::SHRINK_THREADS, 0, s>>>(a);
        else
            lora::shrink_row_kernel<T, false><<<grid, lora::SHRINK_THREADS, 0, s>>>(a);
        return;
    }
    const dim3 grid((unsigned)(((long long)a.t + lora::SHRINK_ROWS - 1) / lora::SHRINK_ROWS));
    auto tile = [&](auto *vec, auto *any) { (a.vec ? vec : any)<<<grid, lora::SHRINK_THREADS, 0, s>>>(a); };
    if (groups >= 8)
        tile(lora::shrink_tile_kernel<T, 1, true>, lora::shrink_tile_kernel<T, 1, false>);
    else if (groups >= 4)
        tile(lora::shrink_tile_kernel<T, 2, true>, lora::shrink_tile_kernel<T, 2, false>);
    else if (groups >= 2)
        tile(lora::shrink_tile_kernel<T, 4, true>, lora::shrink_tile_kernel<T, 4, false>);
    else
        tile(lora::shrink_tile_kernel<T, 8, true>, lora::shrink_tile_kernel<T, 8, false>);
}

}  // namespace

cudaError_t lora_shrink(const lora::ShrinkArgs &a, int dtype, int sms, cudaStream_t s) {
    dtype == ADAPTERS_F32 ? shrink_type<float>(a, sms, s) : shrink_type<__nv_bfloat16>(a, sms, s);
    return cudaGetLastError();
}

cudaError_t lora_expand(const lora::ExpandArgs &a, cudaStream_t s) {
    const dim3 grid((unsigned)(((long long)a.t + lora::EXPAND_ROWS - 1) / lora::EXPAND_ROWS),
                    (unsigned)(((long long)a.n + 4 * lora::EXPAND_THREADS - 1) / (4 * lora::EXPAND_THREADS)));
    (a.vec ? lora::expand_kernel<true> : lora::expand_kernel<false>)<<<grid, lora::EXPAND_THREADS, 0, s>>>(a);
    return cudaGetLastError();
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
    (a.vec ? lora::grad_kernel<true> : lora::grad_kernel<false>)<<<dim3((unsigned)(a.l * rblocks), (unsigned)cols, (unsigned)a.splits), lora::GRAD_THREADS, 0, s>>>(a);
    if (a.splits > 1) {
        lora::GradSumArgs<float> b = {{a.of[0].ws, a.of[1].ws}, {a.of[0].g, a.of[1].g},
                                      {(long long)a.l * a.r * a.of[0].k, (long long)a.l * a.r * a.of[1].k}, a.splits};
        lora::grad_sum_kernel<float><<<(unsigned)((b.count[0] + b.count[1] + 255) / 256), 256, 0, s>>>(b);
    }
    return cudaGetLastError();
}

cudaError_t lora_pad_rows(const lora::PadArgs &a, int sms, cudaStream_t s) {
    long long blocks = 1;
    for (int i = 0; i < a.jobs; ++i)
        if ((a.job[i].rows + 7) / 8 > blocks) blocks = (a.job[i].rows + 7) / 8;
    if (blocks > 8LL * sms) blocks = 8LL * sms;
    lora::pad_rows_kernel<<<(unsigned)blocks, 256, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t lora_simt_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300
