// The instances and launches of the row losses.
#include <atomic>

#include "row_loss.cuh"
#include "adapters_units.h"

namespace sgemm_gb300 {
namespace units {

namespace {

constexpr int kMaxDevices = 64;

// One launch of a row's cluster of `cluster` CTAs: a cluster per row while
// they are resident at once, else as many as are, each taking rows in turn
// through a buffer of the data threads' NV vectors.
template <class T, rowloss::Kind KIND, int THREADS, int NV, bool CACHED>
cudaError_t launch_one(const rowloss::Args &a, int cluster, int dev, cudaStream_t s) {
    static std::atomic<int> resident[kMaxDevices][4][2];   // clusters of 1, 2, 4, 8 CTAs; 0: not asked yet
    auto *kernel = rowloss::row_loss_kernel<T, KIND, THREADS, NV, CACHED>;
    const int lists = KIND == rowloss::DISTILL ? rowloss::places_bytes(a.top) : 0;
    constexpr int DATA = KIND == rowloss::DISTILL ? THREADS - 32 : THREADS;   // (the last warp keeps the places)
    const int buffer = CACHED ? DATA * NV * 16 : 0, lg = cluster == 8 ? 3 : cluster / 2;
    const int smem = (lists + 127) / 128 * 128 + buffer;
    const int room = KIND == rowloss::DISTILL ? 20 * 1024 : 0;
    const int most = buffer + (KIND == rowloss::DISTILL ? rowloss::places_bytes(rowloss::MAX_TOP) : 0);
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3((unsigned)THREADS, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // lists of up to 20 KB (390 places) leave every CTA its place; longer ones are asked for apart
    const int crowd = KIND == rowloss::DISTILL && lists > room ? 1 : 0;
    int fit = resident[dev][lg][crowd].load(std::memory_order_relaxed);
    if (fit == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        cfg.gridDim = dim3((unsigned)cluster * 64, 1, 1);
        cfg.dynamicSmemBytes = (size_t)(crowd ? most : buffer + room);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
        if (e != cudaSuccess) return e;
        if (fit < 1) fit = 1;
        resident[dev][lg][crowd].store(fit, std::memory_order_relaxed);
    }
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
    const bool one = a.t <= fit;
    cfg.gridDim = dim3((unsigned)(one ? a.t : fit) * (unsigned)cluster, 1, 1);
    cfg.dynamicSmemBytes = (size_t)(one ? lists : smem);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <class T, rowloss::Kind KIND>
cudaError_t launch_type(const rowloss::Args &a, int sms, int dev, cudaStream_t s) {
    // vectors of a row, and the CTAs that share it: as few as hold it in
    // registers, more while rows are too few to occupy the device and a part
    // keeps 128 vectors
    const long long nv = ((long long)a.v * (long long)sizeof(T) + 15) / 16;
    int c = 1;
    while (c < rowloss::MAX_CLUSTER && (nv > 4096LL * c || ((long long)a.t * c < 2 * sms && nv >= 1024LL * c))) c *= 2;
    const long long per = (nv + c - 1) / c;
    // distill's last warp has no vectors: the others take a share more
    constexpr int D = KIND == rowloss::DISTILL;
    if (per <= 256) return launch_one<T, KIND, 32 + 32 * D, 8, true>(a, c, dev, s);
    if (per <= 512) return launch_one<T, KIND, 64 + 32 * D, 8, true>(a, c, dev, s);
    if (per <= 1024) return launch_one<T, KIND, 256, 4 + D, true>(a, c, dev, s);
    if (per <= 2048) return launch_one<T, KIND, 256, 8 + 2 * D, true>(a, c, dev, s);
    if (per <= 4096) return launch_one<T, KIND, 512, 8 + D, true>(a, c, dev, s);
    return launch_one<T, KIND, 512, 1, false>(a, c, dev, s);
}

template <rowloss::Kind KIND>
cudaError_t launch_kind(const rowloss::Args &a, int dtype, int sms, int dev, cudaStream_t s) {
    if (dtype == ADAPTERS_F32) return launch_type<float, KIND>(a, sms, dev, s);
    if (dtype == ADAPTERS_BF16) return launch_type<__nv_bfloat16, KIND>(a, sms, dev, s);
    return launch_type<__half, KIND>(a, sms, dev, s);
}

}  // namespace

cudaError_t distill_launch(const rowloss::Args &a, int dtype, int sms, int dev, cudaStream_t s) {
    return launch_kind<rowloss::DISTILL>(a, dtype, sms, dev, s);
}
cudaError_t policy_launch(const rowloss::Args &a, int dtype, int sms, int dev, cudaStream_t s) {
    return launch_kind<rowloss::POLICY>(a, dtype, sms, dev, s);
}
cudaError_t row_loss_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300
