// Launches of the microscaled format's writers and readers.
#include "mx_units.h"

namespace sgemm_gb300 {
namespace units {

namespace {

int store_grid(long long units, int sms) {
    const long long ctas = (units + mx::STORE_THREADS / 32 - 1) / (mx::STORE_THREADS / 32), most = (long long)sms * 8;
    return (int)(ctas < most ? ctas : most);
}

template <class T, int BITS>
void quantize(const mx::QuantArgs &a, bool transposed, int sms, cudaStream_t s) {
    const int segs = (mx::blocks(a.cols) + 7) / 8;
    if (transposed) {
        const long long tiles = ((long long)a.rows + 31) / 32 * segs, most = (long long)sms * 8;
        mx::quantize_t_kernel<T, BITS><<<(unsigned)(tiles < most ? tiles : most), mx::STORE_THREADS, 0, s>>>(a);
    } else {
        mx::quantize_kernel<T, BITS><<<store_grid((long long)a.rows * segs, sms), mx::STORE_THREADS, 0, s>>>(a);
    }
}

template <class T, int BITS>
void dequantize(const mx::DequantArgs &a, int sms, cudaStream_t s) {
    const int segs = (mx::blocks(a.cols) + 7) / 8;
    mx::dequantize_kernel<T, BITS><<<store_grid((long long)a.rows * segs, sms), mx::STORE_THREADS, 0, s>>>(a);
}

}  // namespace

cudaError_t mx_quantize(const mx::QuantArgs &a, int dtype, int bits, bool transposed, int sms, cudaStream_t s) {
    auto *f = dtype == MX_F32 ? (bits == 4 ? quantize<float, 4> : quantize<float, 8>)
                              : (bits == 4 ? quantize<__nv_bfloat16, 4> : quantize<__nv_bfloat16, 8>);
    f(a, transposed, sms, s);
    return cudaGetLastError();
}

cudaError_t mx_dequantize(const mx::DequantArgs &a, int dtype, int bits, int sms, cudaStream_t s) {
    auto *f = dtype == MX_F32 ? (bits == 4 ? dequantize<float, 4> : dequantize<float, 8>)
                              : (bits == 4 ? dequantize<__nv_bfloat16, 4> : dequantize<__nv_bfloat16, 8>);
    f(a, sms, s);
    return cudaGetLastError();
}

cudaError_t mx_store_status(int *status, int *line, bool clear) { return unit_status(status, line, clear); }

}  // namespace units
}  // namespace sgemm_gb300
