// Scratch of one call: a stream-ordered allocation from a pool that its
// library keeps per device.
#pragma once
#include <cuda_runtime.h>

#include <cstdlib>
#include <cstring>

namespace sgemm_gb300 {

// A pool that keeps up to `keep` bytes mapped between calls (the default pool
// unmaps at every synchronisation).
inline cudaError_t make_pool(int dev, unsigned long long keep, cudaMemPool_t *pool) {
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    cudaError_t e = cudaMemPoolCreate(pool, &props);
    if (e != cudaSuccess) {
        *pool = nullptr;
        return e;
    }
    return cudaMemPoolSetAttribute(*pool, cudaMemPoolAttrReleaseThreshold, &keep);
}

// Its parts are 256-byte aligned.  SGEMM_GB300_FAIL_ALLOC: as in
// sgemm_gb300.h; of the value "sgemm" it fails sgemm's own allocations alone.
class Scratch {
  public:
    explicit Scratch(cudaStream_t s) : stream_(s) {}
    Scratch(const Scratch &) = delete;
    Scratch &operator=(const Scratch &) = delete;
    size_t add(size_t bytes) {
        const size_t at = total_;
        total_ += (bytes + 255) / 256 * 256;
        return at;
    }
    cudaError_t take(cudaMemPool_t pool) {
        if (total_ == 0) return cudaSuccess;
        const char *fail = std::getenv("SGEMM_GB300_FAIL_ALLOC");
        const cudaError_t e = fail != nullptr && std::strcmp(fail, "sgemm") != 0
                                  ? cudaErrorMemoryAllocation
                                  : cudaMallocFromPoolAsync(reinterpret_cast<void **>(&base_), total_, pool, stream_);
        if (e != cudaSuccess) base_ = nullptr;
        return e;
    }
    template <class T>
    T *at(size_t off) const {
        return reinterpret_cast<T *>(base_ + off);
    }
    ~Scratch() {
        if (base_ != nullptr) cudaFreeAsync(base_, stream_);
    }

  private:
    cudaStream_t stream_;
    char *base_ = nullptr;
    size_t total_ = 0;
};

}  // namespace sgemm_gb300
