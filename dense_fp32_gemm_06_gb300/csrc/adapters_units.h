// Host entry points of the adapter and loss operators' translation units;
// adapters_api.cu reaches the kernels through these.
#pragma once
#include <cuda_runtime.h>

#include "../../include/adapters_gb300.h"
#include "lora_simt.cuh"
#include "row_loss.cuh"

namespace sgemm_gb300 {
namespace units {

cudaError_t distill_launch(const rowloss::Args &a, int dtype, int sms, cudaStream_t s);
cudaError_t policy_launch(const rowloss::Args &a, int dtype, int sms, cudaStream_t s);
cudaError_t row_loss_status(int *status, int *line, bool clear);

cudaError_t lora_shrink(const lora::ShrinkArgs &a, int dtype, int sms, cudaStream_t s);
cudaError_t lora_expand(const lora::ExpandArgs &a, int dtype, cudaStream_t s);
int lora_grad_splits(int t, int k, int l, int r, int sms);
cudaError_t lora_grad(const lora::GradArgs &a, int dtype, cudaStream_t s);
cudaError_t lora_project(const lora::ProjectArgs &a, cudaStream_t s);
cudaError_t lora_simt_status(int *status, int *line, bool clear);

}  // namespace units
}  // namespace sgemm_gb300
