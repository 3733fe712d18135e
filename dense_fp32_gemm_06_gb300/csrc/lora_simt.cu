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
    if (groups >= 8)
        lora::shrink_tile_kernel<T, 1><<<grid, lora::SHRINK_THREADS, 0, s>>>(a);
    else if (groups >= 4)
        lora::shrink_tile_kernel<T, 2><<<grid, lora::SHRINK_THREADS, 0, s>>>(a);
    else if (groups >= 2)
        lora::shrink_tile_kernel<T, 4><<<grid, lora::SHRINK_THREADS, 0, s>>>(a);
    else
        lora::shrink_tile_kernel<T, 8><<<grid, lora::SHRINK_THREADS, 0, s>>>(a);
}

void grad(const lora::GradArgs &a, cudaStream_t s) {
    const int rblocks = (a.r + lora::GRAD_RANKS - 1) / lora::GRAD_RANKS;
    const dim3 grid((unsigned)(a.l * rblocks), (unsigned)((a.k + lora::GRAD_COLS - 1) / lora::GRAD_COLS),
                    (unsigned)a.splits);
    lora::grad_kernel<<<grid, lora::GRAD_THREADS, 0, s>>>(a);
    if (a.splits > 1) {
        const long long count = (long long)a.l * a.r * a.k;
        lora::grad_sum_kernel<float><<<(unsigned)((count + 255) / 256), 256, 0, s>>>(a.ws, a.g, count, a.splits);
    }
}

}  // namespace

cudaError_t lora_shrink(const lora::ShrinkArgs &a, int dtype, int sms, cudaStream_t s) {
    dtype == ADAPTERS_F32 ? shrink_type<float>(a, sms, s) : shrink_type<__nv_bfloat16>(a, sms, s);
    return cudaGetLastError();
}

cudaError_t lora_expand(const lora::ExpandArgs &a, cudaStream_t s) {
    const dim3 grid((unsigned)(((long long)a.t + lora::EXPAND_ROWS - 1) / lora::EXPAND_ROWS),
                    (unsigned)(((long long)a.n + 4 * lora::EXPAND_THREADS - 1) / (4 * lora::EXPAND_THREADS)));
    lora::expand_kernel<<<grid, lora::EXPAND_THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

// Parts the rows are cut into so that the gradient's CTAs occupy the device:
// none when the adapters' column and rank blocks do already.
int lora_grad_splits(int t, int k, int l, int r, int sms) {
    const long long ctas = (long long)((k + lora::GRAD_COLS - 1) / lora::GRAD_COLS) * l *
                           ((r + lora::GRAD_RANKS - 1) / lora::GRAD_RANKS);
    long long s = (2LL * sms + ctas - 1) / (ctas > 0 ? ctas : 1);
    if (s > t / 256) s = t / 256;   // a part keeps a list of 256 rows
    return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}

cudaError_t lora_grad(const lora::GradArgs &a, cudaStream_t s) {
    grad(a, s);
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
