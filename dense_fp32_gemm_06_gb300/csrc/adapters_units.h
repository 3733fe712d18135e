// Host entry points of the adapter and loss operators' translation units;
// adapters_api.cu reaches the kernels through these.
#pragma once
#include <cuda_runtime.h>

#include "../../include/adapters_gb300.h"
#include "lora_simt.cuh"
#include "lora_skinny.cuh"
#include "lora_tc.cuh"
#include "launch.h"
#include "row_loss.cuh"

namespace sgemm_gb300 {
namespace units {

cudaError_t distill_launch(const rowloss::Args &a, int dtype, int sms, int dev, cudaStream_t s);
cudaError_t policy_launch(const rowloss::Args &a, int dtype, int sms, int dev, cudaStream_t s);
cudaError_t row_loss_status(int *status, int *line, bool clear);

cudaError_t lora_shrink(const lora::ShrinkArgs &a, int dtype, int sms, cudaStream_t s);
// Y = X op(W) + H E_a of few FP32 rows (`after_shrink`: as lora_project's).
cudaError_t lora_simt_setup();
cudaError_t lora_few_rows(const lora::FewArgs &a, bool w_mn, int sms, bool after_shrink, cudaStream_t s);
cudaError_t lora_expand(const lora::ExpandArgs &a, cudaStream_t s);
int lora_grad_splits(int t, int ka, int kb, int l, int r, int sms);
cudaError_t lora_grad(const lora::GradArgs &a, cudaStream_t s);
cudaError_t lora_pad_rows(const lora::PadArgs &a, int sms, cudaStream_t s);

// The tensor-core projection: one-time set-up of the device (kernel
// attributes, clusters that fit), and the launch.  `after_shrink`: the
// kernel in front of it on the stream writes H and lets it start early.
struct TcDevice {
    int sms = 0;
    int clusters[9] = {};   // clusters of S CTAs (S = 2 .. 8) that fit at once
};
cudaError_t lora_tc_setup(int sms, TcDevice *d);
// Map of bfloat16 values, `rank` (2 or 3) axes, innermost first; pitch in
// elements between rows, plane between matrices; boxes of b0 x b1 with the
// 128-byte swizzle.
cudaError_t lora_map(CUtensorMap *map, const void *base, int rank, long long d0, long long d1, long long d2,
                     long long pitch, long long plane, int b0, int b1);
struct TcPlan {
    int bn, split;
    bool pair;
};
TcPlan lora_tc_plan(int t, int n, int k, const TcDevice &d);
// Its tiles along n and t, and the clusters that take them: one each, or as
// many as fit and each takes tiles in turn.
struct TcGrid {
    int tiles_n, tiles_t;
    long long tiles, clusters;
};
TcGrid lora_tc_grid(const TcPlan &p, int t, int n, const TcDevice &d);
cudaError_t lora_project(const lora::TcArgs &a, bool w_mn, const TcDevice &d, bool after_shrink, cudaStream_t s);
cudaError_t lora_tc_status(int *status, int *line, bool clear);

// The adapters' skinny products of bfloat16 matrices on the tensor cores:
// shrink of more than SHRINK_TC_ROWS rows (also into the parts that the
// gradient reads, unless NULL), and the gradients (their P in two bfloat16
// parts, lora_parts).  Rows of x and of the stack 16 bytes apart.
constexpr int SHRINK_TC_ROWS = 128;
cudaError_t lora_skinny_setup();
cudaError_t lora_shrink_tc(const lora::ShrinkArgs &a, void *parts, const TcDevice &d, cudaStream_t s);
size_t lora_parts_bytes(int t, int r);
cudaError_t lora_parts(const float *p, void *parts, int t, int r, cudaStream_t s);
int lora_grad_tc_splits(int t, int ka, int kb, int l, int r, int sms);
cudaError_t lora_grad_tc(const lora::GradTcArgs &a, cudaStream_t s);
cudaError_t lora_skinny_status(int *status, int *line, bool clear);
cudaError_t lora_simt_status(int *status, int *line, bool clear);

}  // namespace units
}  // namespace sgemm_gb300
