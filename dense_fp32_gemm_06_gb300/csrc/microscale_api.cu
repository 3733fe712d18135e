// C ABI of the microscaled operators: argument checks, scratch and launches.
// Declared in include/microscale_gb300.h.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "mx_units.h"
#include "scratch.h"

using namespace sgemm_gb300;

namespace {

thread_local int g_last_cuda_error = 0;

constexpr int kMaxDevices = 64;
constexpr unsigned long long kPoolKeepBytes = 256ull << 20;

struct DeviceState {
    bool ready = false;
    int sms = 0;
    units::MxDevice tc;
    cudaMemPool_t pool = nullptr;
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

int fail_cuda(cudaError_t e) {
    g_last_cuda_error = static_cast<int>(e);
    return SGEMM_STATUS_CUDA_ERROR;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? SGEMM_STATUS_OK : fail_cuda(e); }

int device_state(DeviceState **out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_cuda(e);
    if (dev < 0 || dev >= kMaxDevices) return fail_cuda(cudaErrorInvalidDevice);
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState &d = g_dev[dev];
    if (!d.ready) {
        if ((e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return fail_cuda(e);
        if ((e = units::mx4_setup(d.sms, &d.tc)) != cudaSuccess) return fail_cuda(e);
        if ((e = units::mx_grad_setup()) != cudaSuccess) return fail_cuda(e);
        if (d.pool == nullptr && (e = make_pool(dev, kPoolKeepBytes, &d.pool)) != cudaSuccess) return fail_cuda(e);
        d.ready = true;
    }
    *out = &d;
    return SGEMM_STATUS_OK;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool bad_ptr(const void *p, bool used, int align) { return (used && p == nullptr) || !aligned(p, (uintptr_t)align); }
int size_of(int dtype) { return dtype == MX_F32 ? 4 : 2; }
int imax(int a, int b) { return a > b ? a : b; }
bool known(int dtype) { return dtype == MX_F32 || dtype == MX_BF16; }

// a pitch of codes or scales
bool bad_pitch(int ld, long long row) { return ld < 16 || ld % 16 != 0 || ld < row; }
long long code_row(int cols, int bits) { return (long long)mx::blocks(cols) * mx::block_bytes(bits); }

int zeros(void *y, int ldy, int rows, int cols, int dtype, cudaStream_t stream) {
    const size_t es = (size_t)size_of(dtype);
    return status_of(cudaMemset2DAsync(y, ldy * es, 0, cols * es, (size_t)rows, stream));
}

mx::QuantArgs quant_args(int rows, int cols, int dtype, const void *X, int ldx, void *codes, long long ldc, void *scales, long long lds) {
    const int per16 = 16 / size_of(dtype);
    return {X, ldx, static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales), ldc, lds, rows, cols, aligned(X, 16) && ldx % per16 == 0};
}

int product4(const DeviceState &d, int t, int k, int n, int dtype, const void *X, int ldx, const void *xs, int ldxs, const void *W,
             int ldw, const void *ws, int ldws, void *Y, int ldy, float *sums, cudaStream_t stream) {
    auto bytes = [](const void *p) { return static_cast<const uint8_t *>(p); };
    const mx::M4Args a = {{Y, ldy, t, n, false}, mx::blocks(k), 0, 0, 0, bytes(X), bytes(xs), bytes(W), bytes(ws), ldx, ldxs, ldw, ldws, nullptr, 0, k, false, sums};
    return status_of(units::mx4_product(a, dtype == MX_F32, d.tc, stream));
}

// out (+)= dY M^: dY rows x depth, or (transposed) stored depth x rows
int gradient(int depth, int dtype, bool transposed, const void *dY, int lddy, int bits, const void *codes, int ldc,
             const void *scales, int lds, const mx::Out &out, cudaStream_t stream) {
    DeviceState *d;
    if (const int st = device_state(&d)) return st;
    Scratch ws(stream);
    units::GradCall g = {out, depth, bits, transposed, dY, lddy, lddy, 1, codes, scales, ldc, lds, nullptr};
    const int rows = transposed ? depth : out.rows, cols = transposed ? out.rows : depth;   // as stored
    const bool f32 = dtype == MX_F32, copy = f32 || !aligned(dY, 16) || lddy % 8 != 0;
    if (copy) {
        g.planes = f32 ? 3 : 1;
        g.lddy = ((long long)cols + 63) / 64 * 64;   // whole 128-byte lines
        g.plane = g.lddy * rows;
    }
    const size_t at = copy ? ws.add((size_t)g.plane * g.planes * 2) : 0, at_sums = ws.add(units::mx_grad_sums_bytes(g, f32, d->tc));
    if (const cudaError_t e = ws.take(d->pool)) return fail_cuda(e);
    g.sums = ws.at<float>(at_sums);
    if (copy) {
        const int per16 = 16 / size_of(dtype);
        const mx::PlaneArgs p = {dY, lddy, ws.at<__nv_bfloat16>(at), g.lddy, g.plane, rows, cols, aligned(dY, 16) && lddy % per16 == 0};
        g.dy = p.planes;
        if (const cudaError_t e = units::mx_planes(p, f32, d->sms, stream)) return fail_cuda(e);
    }
    return status_of(units::mx_grad(g, d->tc, stream));
}

}  // namespace

extern "C" {

int mx_quantize(int rows, int cols, int dtype, int op_x, const void *X, int ldx, int bits, void *codes, int ldc,
                void *scales, int lds, cudaStream_t stream) {
    if (rows < 0) return 1;
    if (cols < 0) return 2;
    if (!known(dtype)) return 3;
    if (op_x != SGEMM_OP_N && op_x != SGEMM_OP_T) return 4;
    const bool any = rows > 0 && cols > 0;
    if (bad_ptr(X, any, size_of(dtype))) return 5;
    if (ldx < imax(1, op_x == SGEMM_OP_N ? cols : rows)) return 6;
    if (bits != 4 && bits != 8) return 7;
    if (bad_ptr(codes, any, 16)) return 8;
    if (bad_pitch(ldc, code_row(cols, bits))) return 9;
    if (bad_ptr(scales, any, 16)) return 10;
    if (bad_pitch(lds, mx::blocks(cols))) return 11;
    if (!any) return SGEMM_STATUS_OK;
    DeviceState *d;
    if (const int st = device_state(&d)) return st;
    return status_of(units::mx_quantize(quant_args(rows, cols, dtype, X, ldx, codes, ldc, scales, lds), dtype, bits, op_x == SGEMM_OP_T, d->sms, stream));
}

int mx_dequantize(int rows, int cols, int dtype, int bits, const void *codes, int ldc, const void *scales, int lds,
                  void *Y, int ldy, cudaStream_t stream) {
    if (rows < 0) return 1;
    if (cols < 0) return 2;
    if (!known(dtype)) return 3;
    if (bits != 4 && bits != 8) return 4;
    const bool any = rows > 0 && cols > 0;
    if (bad_ptr(codes, any, 16)) return 5;
    if (bad_pitch(ldc, code_row(cols, bits))) return 6;
    if (bad_ptr(scales, any, 16)) return 7;
    if (bad_pitch(lds, mx::blocks(cols))) return 8;
    if (bad_ptr(Y, any, size_of(dtype))) return 9;
    if (ldy < imax(1, cols)) return 10;
    if (!any) return SGEMM_STATUS_OK;
    DeviceState *d;
    if (const int st = device_state(&d)) return st;
    const int per16 = 16 / size_of(dtype);
    const mx::DequantArgs a = {static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), ldc, lds, Y, ldy, rows, cols,
                               aligned(Y, 16) && ldy % per16 == 0};
    return status_of(units::mx_dequantize(a, dtype, bits, d->sms, stream));
}

int mx4_linear(int t, int k, int n, int dtype, const void *X, int ldx, const void *W, int ldw, const void *w_scales,
               int ldws, void *Y, int ldy, cudaStream_t stream) {
    if (t < 0) return 1;
    if (k < 0) return 2;
    if (n < 0) return 3;
    if (!known(dtype)) return 4;
    const bool out = t > 0 && n > 0;
    if (bad_ptr(X, out && k > 0, size_of(dtype))) return 5;
    if (ldx < imax(1, k)) return 6;
    if (bad_ptr(W, out && k > 0, 16)) return 7;
    if (bad_pitch(ldw, code_row(k, 4))) return 8;
    if (bad_ptr(w_scales, out && k > 0, 16)) return 9;
    if (bad_pitch(ldws, mx::blocks(k))) return 10;
    if (bad_ptr(Y, out, size_of(dtype))) return 11;
    if (ldy < imax(1, n)) return 12;
    if (!out) return SGEMM_STATUS_OK;
    if (k == 0) return zeros(Y, ldy, t, n, dtype, stream);
    DeviceState *d;
    if (const int st = device_state(&d)) return st;
    Scratch ws(stream);
    const size_t at_sums = ws.add(units::mx4_sums_bytes(t, n, mx::blocks(k), dtype == MX_F32, d->tc));
    if (units::mx4_fused(t, n, mx::blocks(k), dtype == MX_F32, d->tc)) {
        if (const cudaError_t e = ws.take(d->pool)) return fail_cuda(e);
        const mx::M4Args a = {{Y, ldy, t, n, false}, mx::blocks(k), 0, 0, 0, nullptr, nullptr, static_cast<const uint8_t *>(W), static_cast<const uint8_t *>(w_scales),
                              0, 0, ldw, ldws, X, ldx, k, aligned(X, 16) && ldx % (16 / size_of(dtype)) == 0, ws.at<float>(at_sums)};
        return status_of(units::mx4_product(a, dtype == MX_F32, d->tc, stream));
    }
    const int ldc = (int)code_row(k, 4), lds = (mx::blocks(k) + 15) / 16 * 16;
    const size_t at_c = ws.add((size_t)t * ldc), at_s = ws.add((size_t)t * lds);
    if (const cudaError_t e = ws.take(d->pool)) return fail_cuda(e);
    uint8_t *xc = ws.at<uint8_t>(at_c), *xs = ws.at<uint8_t>(at_s);
    if (const cudaError_t e = units::mx_quantize(quant_args(t, k, dtype, X, ldx, xc, ldc, xs, lds), dtype, 4, false, d->sms, stream)) return fail_cuda(e);
    return product4(*d, t, k, n, dtype, xc, ldc, xs, lds, W, ldw, w_scales, ldws, Y, ldy, ws.at<float>(at_sums), stream);
}

int mx4_matmul(int t, int k, int n, int dtype, const void *X, int ldx, const void *x_scales, int ldxs, const void *W,
               int ldw, const void *w_scales, int ldws, void *Y, int ldy, cudaStream_t stream) {
    if (t < 0) return 1;
    if (k < 0) return 2;
    if (n < 0) return 3;
    if (!known(dtype)) return 4;
    const bool out = t > 0 && n > 0;
    if (bad_ptr(X, out && k > 0, 16)) return 5;
    if (bad_pitch(ldx, code_row(k, 4))) return 6;
    if (bad_ptr(x_scales, out && k > 0, 16)) return 7;
    if (bad_pitch(ldxs, mx::blocks(k))) return 8;
    if (bad_ptr(W, out && k > 0, 16)) return 9;
    if (bad_pitch(ldw, code_row(k, 4))) return 10;
    if (bad_ptr(w_scales, out && k > 0, 16)) return 11;
    if (bad_pitch(ldws, mx::blocks(k))) return 12;
    if (bad_ptr(Y, out, size_of(dtype))) return 13;
    if (ldy < imax(1, n)) return 14;
    if (!out) return SGEMM_STATUS_OK;
    if (k == 0) return zeros(Y, ldy, t, n, dtype, stream);
    DeviceState *d;
    if (const int st = device_state(&d)) return st;
    Scratch ws(stream);
    const size_t at_sums = ws.add(units::mx4_sums_bytes(t, n, mx::blocks(k), dtype == MX_F32, d->tc));
    if (const cudaError_t e = ws.take(d->pool)) return fail_cuda(e);
    return product4(*d, t, k, n, dtype, X, ldx, x_scales, ldxs, W, ldw, w_scales, ldws, Y, ldy, ws.at<float>(at_sums), stream);
}

int mx_grad_input(int t, int k, int n, int dtype, const void *dY, int lddy, int bits, const void *W, int ldw,
                  const void *w_scales, int ldws, void *dX, int lddx, cudaStream_t stream) {
    if (t < 0) return 1;
    if (k < 0) return 2;
    if (n < 0) return 3;
    if (!known(dtype)) return 4;
    const bool out = t > 0 && k > 0;
    if (bad_ptr(dY, out && n > 0, size_of(dtype))) return 5;
    if (lddy < imax(1, n)) return 6;
    if (bits != 4 && bits != 8) return 7;
    if (bad_ptr(W, out && n > 0, 16)) return 8;
    if (bad_pitch(ldw, code_row(k, bits))) return 9;
    if (bad_ptr(w_scales, out && n > 0, 16)) return 10;
    if (bad_pitch(ldws, mx::blocks(k))) return 11;
    if (bad_ptr(dX, out, size_of(dtype))) return 12;
    if (lddx < imax(1, k)) return 13;
    if (!out) return SGEMM_STATUS_OK;
    if (n == 0) return zeros(dX, lddx, t, k, dtype, stream);
    return gradient(n, dtype, false, dY, lddy, bits, W, ldw, w_scales, ldws, {dX, lddx, t, k, false}, stream);
}

int mx_grad_weight(int t, int k, int n, int dtype, const void *dY, int lddy, int bits, const void *X, int ldx,
                   const void *x_scales, int ldxs, int accumulate, void *dW, int lddw, cudaStream_t stream) {
    if (t < 0) return 1;
    if (k < 0) return 2;
    if (n < 0) return 3;
    if (!known(dtype)) return 4;
    const bool out = n > 0 && k > 0;
    if (bad_ptr(dY, out && t > 0, size_of(dtype))) return 5;
    if (lddy < imax(1, n)) return 6;
    if (bits != 4 && bits != 8) return 7;
    if (bad_ptr(X, out && t > 0, 16)) return 8;
    if (bad_pitch(ldx, code_row(k, bits))) return 9;
    if (bad_ptr(x_scales, out && t > 0, 16)) return 10;
    if (bad_pitch(ldxs, mx::blocks(k))) return 11;
    if (bad_ptr(dW, out, size_of(dtype))) return 13;
    if (lddw < imax(1, k)) return 14;
    if (!out) return SGEMM_STATUS_OK;
    if (t == 0) return accumulate ? SGEMM_STATUS_OK : zeros(dW, lddw, n, k, dtype, stream);
    return gradient(t, dtype, true, dY, lddy, bits, X, ldx, x_scales, ldxs, {dW, lddw, n, k, accumulate != 0}, stream);
}

const char *mx_status_string(int status) {
    static const char *const arg[] = {
        "invalid argument 1",  "invalid argument 2",  "invalid argument 3",  "invalid argument 4",  "invalid argument 5",
        "invalid argument 6",  "invalid argument 7",  "invalid argument 8",  "invalid argument 9",  "invalid argument 10",
        "invalid argument 11", "invalid argument 12", "invalid argument 13", "invalid argument 14"};
    if (status >= 1 && status <= (int)(sizeof(arg) / sizeof(arg[0]))) return arg[status - 1];
    return sgemm_status_string(status);
}

int mx_last_cuda_error(void) { return g_last_cuda_error; }

int mx_plan_for(int call, int t, int k, int n, int dtype, int bits, mx_plan *plan) {
    if (call < MX_PLAN_LINEAR || call > MX_PLAN_GRAD_WEIGHT) return 1;
    if (t < 1) return 2;
    if (k < 1) return 3;
    if (n < 1) return 4;
    if (!known(dtype)) return 5;
    if (call != MX_PLAN_LINEAR && bits != 4 && bits != 8) return 6;
    if (plan == nullptr) return 7;
    DeviceState *d;
    if (const int st = device_state(&d)) return st;
    const bool f32 = dtype == MX_F32, weight = call == MX_PLAN_GRAD_WEIGHT;
    const int rows = weight ? n : t, features = call == MX_PLAN_LINEAR ? n : k, depth = weight ? t : n;
    const units::MxPlan p = call == MX_PLAN_LINEAR
                                ? units::mx4_plan(rows, features, (mx::blocks(k) + 7) / 8, f32, d->tc)
                                : units::mx_grad_plan(rows, features, ((long long)depth + mx::G_K - 1) / mx::G_K, bits, weight, f32, d->tc);
    const units::MxGrid g = units::mx_grid(p, rows, features, d->tc);
    *plan = {p.bn, p.split, p.pair, (int)((g.tiles + g.clusters - 1) / g.clusters)};
    return SGEMM_STATUS_OK;
}

int mx_device_status(int *flag, int clear) {
    if (flag == nullptr) return 1;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return fail_cuda(e);
    *flag = 0;
    cudaError_t (*const parts[])(int *, int *, bool) = {units::mx_store_status, units::mx4_status, units::mx_grad_status, units::mx_grad4_status, units::mx_grad8_status};
    for (auto part : parts) {
        int one = 0;
        if ((e = part(&one, nullptr, clear != 0)) != cudaSuccess) return fail_cuda(e);
        if (*flag == 0) *flag = one;
    }
    return SGEMM_STATUS_OK;
}

}  // extern "C"
