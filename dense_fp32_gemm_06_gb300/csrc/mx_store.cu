// Launches of the microscaled format's writers and readers.
#include <cstdint>

#include "mx_units.h"

namespace sgemm_gb300 {
namespace units {

namespace {

// `units` of a warp each, or of a CTA
template <class Args>
cudaError_t launch(void (*kernel)(Args), const Args &a, long long ctas, int sms, cudaStream_t s) {
    const long long most = (long long)sms * 8;
    return launch_early(kernel, dim3((unsigned)(ctas < most ? ctas : most)), mx::STORE_THREADS, 0, a, s);
}

int unroll(int dtype) { return dtype == MX_F32 ? mx::quant_unroll<float>() : mx::quant_unroll<__nv_bfloat16>(); }

long long row_ctas(int rows, int cols, int unroll) {
    const int run = 8 * unroll, runs = (mx::blocks(cols) + run - 1) / run, warps = mx::STORE_THREADS / 32;
    return ((long long)rows * runs + warps - 1) / warps;
}

}  // namespace

cudaError_t mx_quantize(const mx::QuantArgs &a, int dtype, int bits, bool transposed, int sms, cudaStream_t s) {
    using Kernel = void (*)(mx::QuantArgs);
    Kernel k;
    if (transposed) {
        const bool pairs = dtype == MX_BF16 && a.ldx % 2 == 0 && (reinterpret_cast<uintptr_t>(a.x) & 3) == 0;
        if (pairs) k = bits == 4 ? mx::quantize_t_kernel<__nv_bfloat16, 4, 2> : mx::quantize_t_kernel<__nv_bfloat16, 8, 2>;
        else if (dtype == MX_F32) k = bits == 4 ? mx::quantize_t_kernel<float, 4, 1> : mx::quantize_t_kernel<float, 8, 1>;
        else k = bits == 4 ? mx::quantize_t_kernel<__nv_bfloat16, 4, 1> : mx::quantize_t_kernel<__nv_bfloat16, 8, 1>;
        const int tile = pairs ? 64 : 32;
        return launch(k, a, ((long long)a.rows + tile - 1) / tile * ((mx::blocks(a.cols) + 7) / 8), sms, s);
    }
    if (a.vec)
        k = dtype == MX_F32 ? (bits == 4 ? mx::quantize_kernel<float, 4> : mx::quantize_kernel<float, 8>)
                            : (bits == 4 ? mx::quantize_kernel<__nv_bfloat16, 4> : mx::quantize_kernel<__nv_bfloat16, 8>);
    else
        k = dtype == MX_F32 ? (bits == 4 ? mx::quantize_any_kernel<float, 4> : mx::quantize_any_kernel<float, 8>)
                            : (bits == 4 ? mx::quantize_any_kernel<__nv_bfloat16, 4> : mx::quantize_any_kernel<__nv_bfloat16, 8>);
    return launch(k, a, row_ctas(a.rows, a.cols, a.vec ? unroll(dtype) : mx::QUANT_ANY_UNROLL), sms, s);
}

cudaError_t mx_dequantize(const mx::DequantArgs &a, int dtype, int bits, int sms, cudaStream_t s) {
    using Kernel = void (*)(mx::DequantArgs);
    const Kernel k = dtype == MX_F32 ? (bits == 4 ? mx::dequantize_kernel<float, 4> : mx::dequantize_kernel<float, 8>)
                                     : (bits == 4 ? mx::dequantize_kernel<__nv_bfloat16, 4> : mx::dequantize_kernel<__nv_bfloat16, 8>);
    return launch(k, a, row_ctas(a.rows, a.cols, unroll(dtype)), sms, s);
}

cudaError_t mx_store_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300
