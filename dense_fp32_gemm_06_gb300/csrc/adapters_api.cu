// C ABI of the adapter and loss operators: argument checks, scratch and
// launches.  Declared in include/adapters_gb300.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "adapters_units.h"
#include "scratch.h"

using namespace sgemm_gb300;

namespace {

thread_local int g_last_cuda_error = 0;

constexpr int kMaxDevices = 64;
// scratch kept mapped between calls
constexpr unsigned long long kPoolKeepBytes = 256ull << 20;

// FP32 rows for the kernel that reads W once per 16 of them, instead of sgemm
// and the expand in front of it.  Whole calls with an adapter, us, few rows
// against sgemm: 1 x 4096 x 4096 16.7 / 56, 32 rows 65 / 74, 48 rows 100 / 74;
// by work 256 x 1024 x 1024 (2^28) 37.5 / 35.8, 256 x 512 x 512 16 / 33,
// 512 x 1024 x 1024 68 / 51, 512 x 512 x 512 32 / 42.
constexpr int kFewRows = 32;
constexpr double kFewWork = 268435456.0;   // 2^28

struct DeviceState {
    bool ready = false;
    int sms = 0;
    units::TcDevice tc;
    cudaMemPool_t pool = nullptr;
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

int fail_cuda(cudaError_t e) {
    g_last_cuda_error = static_cast<int>(e);
    return SGEMM_STATUS_CUDA_ERROR;
}

int device_state(DeviceState **out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_cuda(e);
    if (dev < 0 || dev >= kMaxDevices) return fail_cuda(cudaErrorInvalidDevice);
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState &d = g_dev[dev];
    if (!d.ready) {
        if ((e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return fail_cuda(e);
        if ((e = units::lora_tc_setup(d.sms, &d.tc)) != cudaSuccess) return fail_cuda(e);
        if ((e = units::lora_skinny_setup()) != cudaSuccess) return fail_cuda(e);
        if ((e = units::lora_simt_setup()) != cudaSuccess) return fail_cuda(e);
        if (d.pool == nullptr && (e = make_pool(dev, kPoolKeepBytes, &d.pool)) != cudaSuccess) return fail_cuda(e);
        d.ready = true;
    }
    *out = &d;
    return SGEMM_STATUS_OK;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int size_of(int dtype) { return dtype == ADAPTERS_F32 ? 4 : 2; }

// p is needed (when `used`) and aligned to its elements
bool bad_ptr(const void *p, bool used, int align) { return (used && p == nullptr) || !aligned(p, (uintptr_t)align); }

int imax(int a, int b) { return a > b ? a : b; }

bool vec4(const void *p, long long ld, int es) { return aligned(p, 4 * es) && ld % 4 == 0; }

// An operand as the kernels read it: as stored, or (16-bit, where TMA cannot
// read its rows: a base or a pitch that is not a multiple of 16 bytes) a copy
// in the scratch.
struct Operand {
    const void *p = nullptr;
    long long ld = 0, rows = 0;
    int cols = 0;
    bool copy = false;
    size_t at = 0;
    Operand() = default;
    Operand(const void *p_, long long ld_, long long rows_, int cols_, bool readable, Scratch &ws)
        : p(p_), ld(ld_), rows(rows_), cols(cols_), copy(readable && rows_ > 0 && cols_ > 0 && (!aligned(p_, 16) || ld_ % 8 != 0)) {
        if (copy) at = ws.add((size_t)rows * pitch() * 2);
    }
    // rows of whole 128-byte lines: TMA's 128-byte box rows otherwise touch two
    // (5226 x 1344 x 2816: 48 us, with pitches of 1336 and 2768 62)
    long long pitch() const { return ((long long)cols + 63) / 64 * 64; }
};

// The copies of a call, in one launch.
int make_copies(Operand *const *ops, int n, const Scratch &ws, int sms, cudaStream_t stream) {
    lora::PadArgs a = {};
    for (int i = 0; i < n; ++i) {
        Operand &o = *ops[i];
        if (!o.copy) continue;
        lora::PadJob &b = a.job[a.jobs++];
        const int by = aligned(o.p, 8) && o.ld % 4 == 0 ? 4 : aligned(o.p, 4) && o.ld % 2 == 0 ? 2 : 1;
        b = {static_cast<const uint16_t *>(o.p), ws.at<uint16_t>(o.at), o.ld, o.pitch(), o.rows, o.cols, by};
        o.p = b.dst;
        o.ld = b.ldd;
    }
    if (a.jobs == 0) return SGEMM_STATUS_OK;
    const cudaError_t e = units::lora_pad_rows(a, sms, stream);
    return e != cudaSuccess ? fail_cuda(e) : SGEMM_STATUS_OK;
}

// bfloat16 rows enough for the tensor-core shrink; below, a row and four
// ranks per CTA on the CUDA cores (which read any rows) answer sooner
bool shrink_on_tc(int t, int k, int dtype) { return dtype == ADAPTERS_BF16 && t > units::SHRINK_TC_ROWS && k > 0; }

// H or U: h = scale (x s_a^T), t x r
int shrink(const DeviceState &d, int t, int k, int l, int r, int dtype, const Operand &x, const Operand &s,
           const int *ids, const float *scale, float *h, void *parts, cudaStream_t stream) {
    const int es = size_of(dtype);
    const lora::ShrinkArgs a = {x.p, x.ld, s.p, s.ld, ids, scale, h, t, k, l, r, k % 4 == 0 && vec4(x.p, x.ld, es) && vec4(s.p, s.ld, es)};
    cudaError_t e;
    if (shrink_on_tc(t, k, dtype)) {
        e = units::lora_shrink_tc(a, parts, d.tc, stream);
    } else {
        e = units::lora_shrink(a, dtype, d.sms, stream);
        if (e == cudaSuccess && parts) e = units::lora_parts(h, parts, t, r, stream);
    }
    return e != cudaSuccess ? fail_cuda(e) : SGEMM_STATUS_OK;
}

// Whether the projection is the library's sgemm, with the adapters' part added
// to it: sgemm may ask for scratch, so it is enqueued before anything else of
// the call, and a failed allocation leaves every output as it was.
bool by_sgemm(int t, int k, int n, int dtype) {
    return dtype == ADAPTERS_F32 && k > 0 && t > kFewRows && ((double)t * n * k > kFewWork || t > 16 * 65535);
}

// y (t x n) = x op(w) of those, op(w) k x n
int product(int t, int k, int n, const Operand &x, int op_w, const Operand &w, void *y, int ldy, cudaStream_t stream) {
    const int st = sgemm_op(SGEMM_OP_N, op_w, t, n, k, 1.f, static_cast<const float *>(x.p), (int)x.ld,
                            static_cast<const float *>(w.p), (int)w.ld, 0.f, static_cast<float *>(y), ldy, stream, SGEMM_PATH_AUTO);
    return st == SGEMM_STATUS_CUDA_ERROR ? fail_cuda(static_cast<cudaError_t>(sgemm_last_cuda_error())) : st;
}

// y (t x n) = x op(w) + h e_a, op(w) k x n; y + h e_a of those by_sgemm
int project(const DeviceState &d, int t, int k, int n, int l, int r, int dtype, const Operand &x, int op_w,
            const Operand &w, const Operand &e, const int *ids, const float *h, void *y, int ldy, cudaStream_t stream) {
    const bool adapters = l > 0 && r > 0;
    cudaError_t err;
    if (k == 0) {   // nothing to contract, and H is zero
        const size_t es = (size_t)size_of(dtype);
        err = cudaMemset2DAsync(y, ldy * es, 0, n * es, (size_t)t, stream);
        return err != cudaSuccess ? fail_cuda(err) : SGEMM_STATUS_OK;
    }
    if (dtype == ADAPTERS_BF16) {
        lora::TcArgs a = {};
        a.t = t;
        a.n = n;
        a.k = k;
        a.l = adapters ? l : 0;
        a.r = adapters ? r : 0;
        a.h = h;
        a.ids = ids;
        a.y = static_cast<__nv_bfloat16 *>(y);
        a.ldy = ldy;
        a.x = static_cast<const __nv_bfloat16 *>(x.p);
        a.w = static_cast<const __nv_bfloat16 *>(w.p);
        a.e = static_cast<const __nv_bfloat16 *>(e.p);
        a.ldx = x.ld;
        a.ldw = w.ld;
        a.lde = e.ld;
        err = units::lora_project(a, op_w == SGEMM_OP_N, d.tc, adapters, stream);
        return err != cudaSuccess ? fail_cuda(err) : SGEMM_STATUS_OK;
    }
    if (!by_sgemm(t, k, n, dtype)) {
        const lora::FewArgs a = {static_cast<const float *>(x.p), static_cast<const float *>(w.p), static_cast<const float *>(e.p),
                                 x.ld, w.ld, h, ids, static_cast<float *>(y), ldy, t, k, n, adapters ? l : 0, adapters ? r : 0,
                                 aligned(w.p, 16) && w.ld % 4 == 0};
        err = units::lora_few_rows(a, op_w == SGEMM_OP_N, d.sms, adapters, stream);
        return err != cudaSuccess ? fail_cuda(err) : SGEMM_STATUS_OK;
    }
    if (!adapters) return SGEMM_STATUS_OK;
    const lora::ExpandArgs a = {h, static_cast<const float *>(e.p), ids, static_cast<float *>(y), ldy, t, n, l, r, vec4(e.p, n, 4) && vec4(y, ldy, 4)};
    return (err = units::lora_expand(a, stream)) != cudaSuccess ? fail_cuda(err) : SGEMM_STATUS_OK;
}

// The adapters' gradients, dA = sum u_t^T x_t and dB = sum h_t^T dy_t over the
// rows of each adapter, with their scratch: the parts of u and h (bfloat16)
// and the partial sums of the rows' parts.
struct Gradients {
    int t, l, r, dtype, splits = 1;
    int cols[2];   // of dA and dB; 0: not wanted
    size_t at_parts[2] = {0, 0}, at_ws[2] = {0, 0};
    Gradients(int t_, int ka, int kb, int l_, int r_, int dtype_, int sms, Scratch &ws)
        : t(t_), l(l_), r(r_), dtype(dtype_), cols{ka, kb} {
        if (t == 0 || (ka == 0 && kb == 0)) return;
        const bool tc = dtype == ADAPTERS_BF16;
        splits = tc ? units::lora_grad_tc_splits(t, ka, kb, l, r, sms) : units::lora_grad_splits(t, ka, kb, l, r, sms);
        for (int i = 0; i < 2; ++i) {
            if (cols[i] == 0) continue;
            if (tc) at_parts[i] = ws.add(units::lora_parts_bytes(t, r));
            if (splits > 1) at_ws[i] = ws.add((size_t)splits * l * r * cols[i] * sizeof(float));
        }
    }
    // where the shrink leaves u's parts
    void *parts_of_u(const Scratch &ws) const {
        return dtype == ADAPTERS_BF16 && cols[0] > 0 && t > 0 ? ws.at<void>(at_parts[0]) : nullptr;
    }
    int run(const Scratch &ws, const float *u, const float *h, const Operand &x, const Operand &dy, const int *ids, void *dA,
            void *dB, cudaStream_t stream) const {
        const float *p[2] = {u, h};
        const Operand *op[2] = {&x, &dy};
        void *g[2] = {dA, dB};
        cudaError_t e = cudaSuccess;
        if (t == 0) {
            for (int i = 0; i < 2 && e == cudaSuccess; ++i)
                if (cols[i] > 0) e = cudaMemsetAsync(g[i], 0, (size_t)l * r * cols[i] * size_of(dtype), stream);
        } else if (dtype == ADAPTERS_BF16) {
            lora::GradTcArgs a = {{}, ids, t, l, r, splits};
            for (int i = 0; i < 2; ++i)
                a.of[i] = {ws.at<__nv_bfloat16>(at_parts[i]), static_cast<const __nv_bfloat16 *>(op[i]->p), op[i]->ld,
                           static_cast<__nv_bfloat16 *>(g[i]), ws.at<float>(at_ws[i]), cols[i]};
            if (cols[1] > 0) e = units::lora_parts(h, ws.at<void>(at_parts[1]), t, r, stream);
            if (e == cudaSuccess) e = units::lora_grad_tc(a, stream);
        } else {
            lora::GradArgs a = {{}, true, ids, t, l, r, splits};
            for (int i = 0; i < 2; ++i) {
                a.of[i] = {p[i], static_cast<const float *>(op[i]->p), op[i]->ld, static_cast<float *>(g[i]), ws.at<float>(at_ws[i]), cols[i]};
                a.vec = a.vec && (cols[i] == 0 || (vec4(op[i]->p, op[i]->ld, 4) && vec4(g[i], cols[i], 4)));
            }
            e = units::lora_grad(a, stream);
        }
        return e != cudaSuccess ? fail_cuda(e) : SGEMM_STATUS_OK;
    }
};

}  // namespace

extern "C" {

int lora_forward(int t, int k, int n, int l, int r, int dtype, const void *X, int ldx, int op_w, const void *W,
                 int ldw, const void *A, const void *B, const int *ids, const float *scale, void *Y, int ldy, float *H,
                 cudaStream_t stream) {
    if (t < 0) return 1;
    if (k < 0) return 2;
    if (n < 0) return 3;
    if (l < 0) return 4;
    if (r < 0 || r > ADAPTERS_MAX_RANK) return 5;
    if (dtype != ADAPTERS_F32 && dtype != ADAPTERS_BF16) return 6;
    const int es = size_of(dtype);
    const bool out = t > 0 && n > 0, adapters = t > 0 && l > 0 && r > 0;
    if (bad_ptr(X, t > 0 && k > 0 && (n > 0 || (adapters && H)), es)) return 7;
    if (ldx < imax(1, k)) return 8;
    if (op_w != SGEMM_OP_N && op_w != SGEMM_OP_T) return 9;
    if (bad_ptr(W, out && k > 0, es)) return 10;
    if (ldw < imax(1, op_w == SGEMM_OP_N ? n : k)) return 11;
    if (bad_ptr(A, adapters && k > 0, es)) return 12;
    if (bad_ptr(B, adapters && n > 0, es)) return 13;
    if (bad_ptr(ids, adapters, 4)) return 14;
    if (bad_ptr(scale, false, 4)) return 15;
    if (bad_ptr(Y, out, es)) return 16;
    if (ldy < imax(1, n)) return 17;
    if (bad_ptr(H, false, 4)) return 18;
    if (!out && !(adapters && H)) return SGEMM_STATUS_OK;

    DeviceState *d;
    int st = device_state(&d);
    if (st) return st;
    Scratch ws(stream);
    const size_t at_h = adapters && !H ? ws.add((size_t)t * r * sizeof(float)) : 0;
    const bool tc = dtype == ADAPTERS_BF16 && out && k > 0, tc_h = adapters && shrink_on_tc(t, k, dtype);
    Operand x(X, ldx, t, k, tc || tc_h, ws);
    Operand w(W, ldw, op_w == SGEMM_OP_N ? k : n, op_w == SGEMM_OP_N ? n : k, tc, ws);
    Operand down(A, k, (long long)l * r, k, tc_h, ws), up(B, n, (long long)l * r, n, tc && adapters, ws);
    if (const cudaError_t e = ws.take(d->pool)) return fail_cuda(e);
    Operand *const all[] = {&x, &w, &down, &up};
    if (out && by_sgemm(t, k, n, dtype) && (st = product(t, k, n, x, op_w, w, Y, ldy, stream))) return st;
    if ((st = make_copies(all, 4, ws, d->sms, stream))) return st;
    float *h = H ? H : ws.at<float>(at_h);
    if (adapters && (st = shrink(*d, t, k, l, r, dtype, x, down, ids, scale, h, nullptr, stream))) return st;
    if (!out) return SGEMM_STATUS_OK;
    return project(*d, t, k, n, l, r, dtype, x, op_w, w, up, ids, h, Y, ldy, stream);
}

int lora_backward(int t, int k, int n, int l, int r, int dtype, const void *dY, int lddy, const void *X, int ldx,
                  int op_w, const void *W, int ldw, const void *A, const void *B, const int *ids, const float *scale,
                  const float *H, void *dX, int lddx, void *dA, void *dB, cudaStream_t stream) {
    if (t < 0) return 1;
    if (k < 0) return 2;
    if (n < 0) return 3;
    if (l < 0) return 4;
    if (r < 0 || r > ADAPTERS_MAX_RANK) return 5;
    if (dtype != ADAPTERS_F32 && dtype != ADAPTERS_BF16) return 6;
    const int es = size_of(dtype);
    const bool adapters = t > 0 && l > 0 && r > 0;
    const bool want_x = dX && t > 0 && k > 0, want_a = dA && l > 0 && r > 0 && k > 0, want_b = dB && l > 0 && r > 0 && n > 0;
    if (bad_ptr(dY, t > 0 && n > 0 && (want_x || want_a || want_b), es)) return 7;
    if (lddy < imax(1, n)) return 8;
    if (bad_ptr(X, want_a && t > 0, es)) return 9;
    if (ldx < imax(1, k)) return 10;
    if (op_w != SGEMM_OP_N && op_w != SGEMM_OP_T) return 11;
    if (bad_ptr(W, want_x && n > 0, es)) return 12;
    if (ldw < imax(1, op_w == SGEMM_OP_N ? n : k)) return 13;
    if (bad_ptr(A, adapters && want_x, es)) return 14;
    if (bad_ptr(B, adapters && (want_x || want_a) && n > 0, es)) return 15;
    if (bad_ptr(ids, adapters && (want_x || want_a || want_b), 4)) return 16;
    if (bad_ptr(scale, false, 4)) return 17;
    if (bad_ptr(H, want_b && t > 0, 4)) return 18;
    if (!aligned(dX, es)) return 19;
    if (lddx < imax(1, k)) return 20;
    if (!aligned(dA, es)) return 21;
    if (!aligned(dB, es)) return 22;
    if (!want_x && !want_a && !want_b) return SGEMM_STATUS_OK;

    DeviceState *d;
    int st = device_state(&d);
    if (st) return st;
    Scratch ws(stream);
    const bool need_u = adapters && (want_x || want_a);
    const size_t at_u = need_u ? ws.add((size_t)t * r * sizeof(float)) : 0;
    const bool b16 = dtype == ADAPTERS_BF16, tc = b16 && want_x && n > 0, tc_u = need_u && shrink_on_tc(t, n, dtype);
    Operand dy(dY, lddy, t, n, tc || tc_u || (b16 && want_b), ws), x(X, ldx, t, k, b16 && want_a, ws);
    Operand w(W, ldw, op_w == SGEMM_OP_N ? k : n, op_w == SGEMM_OP_N ? n : k, tc, ws);
    Operand down(B, n, (long long)l * r, n, tc_u, ws), up(A, k, (long long)l * r, k, tc && adapters, ws);
    const Gradients grads(t, want_a ? k : 0, want_b ? n : 0, l, r, dtype, d->sms, ws);
    if (const cudaError_t e = ws.take(d->pool)) return fail_cuda(e);
    Operand *const all[] = {&dy, &x, &w, &down, &up};
    const int op_t = op_w == SGEMM_OP_N ? SGEMM_OP_T : SGEMM_OP_N;   // the frozen projection's transpose
    if (want_x && by_sgemm(t, n, k, dtype) && (st = product(t, n, k, dy, op_t, w, dX, lddx, stream))) return st;
    if ((st = make_copies(all, 5, ws, d->sms, stream))) return st;
    float *u = ws.at<float>(at_u);
    if (need_u && (st = shrink(*d, t, n, l, r, dtype, dy, down, ids, scale, u, grads.parts_of_u(ws), stream))) return st;
    if (want_x && (st = project(*d, t, n, k, l, r, dtype, dy, op_t, w, up, ids, u, dX, lddx, stream))) return st;
    if (!want_a && !want_b) return SGEMM_STATUS_OK;
    return grads.run(ws, u, H, x, dy, ids, dA, dB, stream);
}

int distill_topk(int t, int v, int top, int dtype, const void *logits, int ldz, const float *teacher,
                 const int *index, const float *weight, float temperature, float *loss, void *grad, int ldg,
                 cudaStream_t stream) {
    if (t < 0) return 1;
    if (v < 0) return 2;
    if (top < 1 || top > ADAPTERS_MAX_TOP) return 3;
    if (dtype != ADAPTERS_F32 && dtype != ADAPTERS_BF16 && dtype != ADAPTERS_F16) return 4;
    const int es = size_of(dtype);
    if (bad_ptr(logits, t > 0 && v > 0, es)) return 5;
    if (ldz < imax(1, v)) return 6;
    if (bad_ptr(teacher, t > 0, 4)) return 7;
    if (bad_ptr(index, t > 0, 4)) return 8;
    if (bad_ptr(weight, false, 4)) return 9;
    if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.44269504088896341f / temperature)) return 10;
    if (bad_ptr(loss, t > 0, 4)) return 11;
    if (!aligned(grad, es)) return 12;
    if (ldg < imax(1, v)) return 13;
    if (t == 0) return SGEMM_STATUS_OK;
    DeviceState *d;
    int st = device_state(&d);
    if (st) return st;
    rowloss::Args a = {};
    a.z = logits;
    a.grad = grad;
    a.ldz = ldz;
    a.ldg = ldg;
    a.t = t;
    a.v = v;
    a.c = 1.44269504088896341f / temperature;
    a.weight = weight;
    a.loss = loss;
    a.teacher = teacher;
    a.index = index;
    a.top = top;
    a.tau = temperature;
    const cudaError_t e = units::distill_launch(a, dtype, d->sms, (int)(d - g_dev), stream);
    return e != cudaSuccess ? fail_cuda(e) : SGEMM_STATUS_OK;
}

int policy_loss(int t, int v, int dtype, const void *logits, int ldz, const int *labels, const float *old_logp,
                const float *advantage, const float *ref, const float *weight, float clip_low, float clip_high,
                float kl_coef, float *loss, float *logp, void *grad, int ldg, cudaStream_t stream) {
    if (t < 0) return 1;
    if (v < 0) return 2;
    if (dtype != ADAPTERS_F32 && dtype != ADAPTERS_BF16 && dtype != ADAPTERS_F16) return 3;
    const int es = size_of(dtype);
    if (bad_ptr(logits, t > 0 && v > 0, es)) return 4;
    if (ldz < imax(1, v)) return 5;
    if (bad_ptr(labels, t > 0, 4)) return 6;
    if (bad_ptr(old_logp, t > 0, 4)) return 7;
    if (bad_ptr(advantage, t > 0, 4)) return 8;
    if (bad_ptr(ref, t > 0 && kl_coef != 0.f, 4)) return 9;
    if (bad_ptr(weight, false, 4)) return 10;
    if (!(clip_low >= 0.f)) return 11;
    if (!(clip_high >= 0.f)) return 12;
    if (!std::isfinite(kl_coef)) return 13;
    if (bad_ptr(loss, t > 0, 4)) return 14;
    if (bad_ptr(logp, false, 4)) return 15;
    if (!aligned(grad, es)) return 16;
    if (ldg < imax(1, v)) return 17;
    if (t == 0) return SGEMM_STATUS_OK;
    DeviceState *d;
    int st = device_state(&d);
    if (st) return st;
    rowloss::Args a = {};
    a.z = logits;
    a.grad = grad;
    a.ldz = ldz;
    a.ldg = ldg;
    a.t = t;
    a.v = v;
    a.c = 1.44269504088896341f;
    a.weight = weight;
    a.loss = loss;
    a.label = labels;
    a.old_logp = old_logp;
    a.adv = advantage;
    a.ref = ref;
    a.clip_low = clip_low;
    a.clip_high = clip_high;
    a.kl = kl_coef;
    a.logp = logp;
    const cudaError_t e = units::policy_launch(a, dtype, d->sms, (int)(d - g_dev), stream);
    return e != cudaSuccess ? fail_cuda(e) : SGEMM_STATUS_OK;
}

const char *adapters_status_string(int status) {
    static const char *const arg[] = {
        "invalid argument 1",  "invalid argument 2",  "invalid argument 3",  "invalid argument 4",  "invalid argument 5",
        "invalid argument 6",  "invalid argument 7",  "invalid argument 8",  "invalid argument 9",  "invalid argument 10",
        "invalid argument 11", "invalid argument 12", "invalid argument 13", "invalid argument 14", "invalid argument 15",
        "invalid argument 16", "invalid argument 17", "invalid argument 18", "invalid argument 19", "invalid argument 20",
        "invalid argument 21", "invalid argument 22"};
    if (status >= 1 && status <= (int)(sizeof(arg) / sizeof(arg[0]))) return arg[status - 1];
    return sgemm_status_string(status);
}

int adapters_last_cuda_error(void) { return g_last_cuda_error; }

int adapters_plan_for(int t, int k, int n, adapters_plan *plan) {
    if (t < 1) return 1;
    if (k < 1) return 2;
    if (n < 1) return 3;
    if (plan == nullptr) return 4;
    DeviceState *d;
    if (const int st = device_state(&d)) return st;
    const units::TcPlan p = units::lora_tc_plan(t, n, k, d->tc);
    const units::TcGrid g = units::lora_tc_grid(p, t, n, d->tc);
    *plan = {p.bn, p.split, p.pair, (int)((g.tiles + g.clusters - 1) / g.clusters)};
    return SGEMM_STATUS_OK;
}

int adapters_device_status(int *flag, int clear) {
    if (flag == nullptr) return 1;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return fail_cuda(e);
    *flag = 0;
    cudaError_t (*const parts[])(int *, int *, bool) = {units::row_loss_status, units::lora_simt_status, units::lora_tc_status,
                                                        units::lora_skinny_status};
    for (auto part : parts) {
        int one = 0;
        if ((e = part(&one, nullptr, clear != 0)) != cudaSuccess) return fail_cuda(e);
        if (*flag == 0) *flag = one;
    }
    return SGEMM_STATUS_OK;
}

}  // extern "C"
