// The instances and launches of the row losses.
#include "row_loss.cuh"
#include "adapters_units.h"

namespace sgemm_gb300 {
namespace units {

namespace {

template <class T, rowloss::Kind KIND, int NV, bool CACHED>
cudaError_t launch_one(const rowloss::Args &a, int cluster, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.t * (unsigned)cluster, 1, 1);
    cfg.blockDim = dim3((unsigned)rowloss::THREADS, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, rowloss::row_loss_kernel<T, KIND, NV, CACHED>, a);
}

template <class T, rowloss::Kind KIND>
cudaError_t launch_type(const rowloss::Args &a, int sms, cudaStream_t s) {
    // vectors of a row at most, and the CTAs that share it: as few as hold
    // it in registers (8 vectors a thread), more while rows are too few to
    // occupy the device and a part keeps a vector for every thread
    const long long nv = ((long long)a.v * (long long)sizeof(T) + 15) / 16;
    int c = 1;
    while (c < rowloss::MAX_CLUSTER &&
           (nv > 8LL * rowloss::THREADS * c || ((long long)a.t * c < sms && nv >= 2LL * rowloss::THREADS * c)))
        c *= 2;
    const long long per = (nv + c - 1) / c;
    if (per <= rowloss::THREADS) return launch_one<T, KIND, 1, true>(a, c, s);
    if (per <= 2 * rowloss::THREADS) return launch_one<T, KIND, 2, true>(a, c, s);
    if (per <= 4 * rowloss::THREADS) return launch_one<T, KIND, 4, true>(a, c, s);
    if (per <= 8 * rowloss::THREADS) return launch_one<T, KIND, 8, true>(a, c, s);
    return launch_one<T, KIND, 1, false>(a, c, s);
}

template <rowloss::Kind KIND>
cudaError_t launch_kind(const rowloss::Args &a, int dtype, int sms, cudaStream_t s) {
    if (dtype == ADAPTERS_F32) return launch_type<float, KIND>(a, sms, s);
    if (dtype == ADAPTERS_BF16) return launch_type<__nv_bfloat16, KIND>(a, sms, s);
    return launch_type<__half, KIND>(a, sms, s);
}

}  // namespace

cudaError_t distill_launch(const rowloss::Args &a, int dtype, int sms, cudaStream_t s) {
    return launch_kind<rowloss::DISTILL>(a, dtype, sms, s);
}
cudaError_t policy_launch(const rowloss::Args &a, int dtype, int sms, cudaStream_t s) {
    return launch_kind<rowloss::POLICY>(a, dtype, sms, s);
}
cudaError_t row_loss_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300
