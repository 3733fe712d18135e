// Host entry points of the microscaled operators' translation units;
// microscale_api.cu reaches the kernels through these.
#pragma once
#include <cuda_runtime.h>

#include <cuda.h>

#include "../../include/microscale_gb300.h"
#include "launch.h"
#include "mx4_tc.cuh"
#include "mx_grad.cuh"
#include "mx_store.cuh"

namespace sgemm_gb300 {
namespace units {

cudaError_t mx_quantize(const mx::QuantArgs &a, int dtype, int bits, bool transposed, int sms, cudaStream_t s);
cudaError_t mx_dequantize(const mx::DequantArgs &a, int dtype, int bits, int sms, cudaStream_t s);
cudaError_t mx_store_status(int *status, int *line, bool clear);

struct MxDevice {
    int sms = 0;
    int clusters[9] = {};   // clusters of S CTAs (S = 2 .. 8) that fit at once
};
// Rows of an output tile, CTAs that share its contraction, whether CTA pairs
// share tiles; the tiles along features and rows, and the clusters that take them.
struct MxPlan {
    int bn, split;
    bool pair;
};
struct MxGrid {
    int tiles_f, tiles_r;
    long long tiles, clusters;
};
MxGrid mx_grid(const MxPlan &p, int rows, int features, const MxDevice &d);
// Bytes of a launch's `sums` where its CTAs take up to `stages` stages of the contraction each and an accumulator `deep`.
size_t mx_sums_bytes(const MxPlan &p, int rows, int features, long long stages, int deep, const MxDevice &d);
// Map of a matrix of `inner` x `rows` elements of `size` bytes, `pitch` bytes
// between rows; boxes of b0 x b1 (b0: 64 or 128 bytes where swizzled by as much).
cudaError_t mx_map(CUtensorMap *map, CUtensorMapDataType type, int size, const void *base, long long inner, long long rows,
                   long long pitch, int b0, int b1, bool swizzle);
// Y = X^ W^^T: one-time set-up of the device, and the launch.  Of up to
// MX4_FUSED_ROWS rows X may come as real values; mx4_fused: whether it should.
constexpr int MX4_FUSED_ROWS = 16;
bool mx4_fused(int t, int n, int blocks, bool f32, const MxDevice &d);
cudaError_t mx4_setup(int sms, MxDevice *d);
MxPlan mx4_plan(int t, int n, int nk, bool f32, const MxDevice &d);   // nk stages of M4_K
// Bytes that `sums` of such a product needs, mostly 0; the same of a gradient below.
size_t mx4_sums_bytes(int t, int n, int blocks, bool f32, const MxDevice &d);
cudaError_t mx4_product(const mx::M4Args &a, bool f32, const MxDevice &d, cudaStream_t s);
cudaError_t mx4_status(int *status, int *line, bool clear);
// Map of `planes` matrices of inner x rows bfloat16 values, pitch and plane in
// values; boxes of b0 (64) x b1 with the 128-byte swizzle.
cudaError_t mx_map3(CUtensorMap *map, const void *base, long long inner, long long rows, int planes, long long pitch,
                    long long plane, int b0, int b1);

// out (+)= dY M^ (out.rows x out.cols, `depth` contracted): one-time set-up of
// the device, dY's planes where it needs them, and the launch.
struct GradCall {
    mx::Out out;
    int depth, bits;
    bool transposed;          // dY is stored depth x rows
    const void *dy;           // bfloat16, 16-byte aligned rows; three planes: FP32 results
    long long lddy, plane;    // in values
    int planes;
    const void *codes, *scales;
    long long ldc, lds;
    float *sums;
};
size_t mx_grad_sums_bytes(const GradCall &g, bool f32, const MxDevice &d);
MxPlan mx_grad_plan(int p, int c, long long stages, int bits, bool transposed, bool f32, const MxDevice &d);
cudaError_t mx_grad_setup();
cudaError_t mx_planes(const mx::PlaneArgs &a, bool f32, int sms, cudaStream_t s);
cudaError_t mx_grad(const GradCall &g, const MxDevice &d, cudaStream_t s);
cudaError_t mx_grad_status(int *status, int *line, bool clear);
// (the parts of those in the units of 4 and 8 bits)
cudaError_t mx_grad4_setup();
cudaError_t mx_grad8_setup();
cudaError_t mx_grad4_launch(const cudaLaunchConfig_t &cfg, const MxPlan &p, bool transposed, bool f32, const CUtensorMap *m, const mx::GradArgs &a);
cudaError_t mx_grad8_launch(const cudaLaunchConfig_t &cfg, const MxPlan &p, bool transposed, bool f32, const CUtensorMap *m, const mx::GradArgs &a);
cudaError_t mx_grad4_status(int *status, int *line, bool clear);
cudaError_t mx_grad8_status(int *status, int *line, bool clear);

}  // namespace units
}  // namespace sgemm_gb300
