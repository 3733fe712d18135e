// The gradients beside a matrix in 4 bits.
#include "mx_grad_units.cuh"

namespace sgemm_gb300 {
namespace units {

cudaError_t mx_grad4_setup() { return grad_setup<4>(); }
cudaError_t mx_grad4_launch(const cudaLaunchConfig_t &cfg, const MxPlan &p, bool transposed, bool f32, const CUtensorMap *m, const mx::GradArgs &a) {
    return grad_launch<4>(cfg, p, transposed, f32, m, a);
}
cudaError_t mx_grad4_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300
