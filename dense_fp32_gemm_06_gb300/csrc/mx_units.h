// Host entry points of the microscaled operators' translation units;
// microscale_api.cu reaches the kernels through these.
#pragma once
#include <cuda_runtime.h>

#include "../../include/microscale_gb300.h"
#include "mx_simple.cuh"
#include "mx_store.cuh"

namespace sgemm_gb300 {
namespace units {

cudaError_t mx_quantize(const mx::QuantArgs &a, int dtype, int bits, bool transposed, int sms, cudaStream_t s);
cudaError_t mx_dequantize(const mx::DequantArgs &a, int dtype, int bits, int sms, cudaStream_t s);
cudaError_t mx_store_status(int *status, int *line, bool clear);

cudaError_t mx_simple(const mx::SimpleArgs &a, cudaStream_t s);

}  // namespace units
}  // namespace sgemm_gb300
