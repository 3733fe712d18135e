/*
 * adapters_gb300.h -- C ABI of the adapter and loss operators of the GB300
 * GEMM library (sm_103a): low-rank adapters of many requests beside a shared
 * projection, and two losses over the logits such a projection makes.
 *
 *   lora_forward    Y_t = X_t W + H_t B_a,      H_t = s_a X_t A_a^T,  a = ids[t]
 *   lora_backward   dX_t = dY_t W^T + U_t A_a,  U_t = s_a dY_t B_a^T,
 *                   dA_a = sum_{t: ids[t]=a} U_t^T X_t,
 *                   dB_a = sum_{t: ids[t]=a} H_t^T dY_t
 *   distill_topk    loss_t = w_t tau^2 sum_j q_tj (log q_tj - log p_t[index_tj]),
 *                   p_t = softmax(z_t / tau), q_t = softmax(teacher_t / tau)
 *   policy_loss     loss_t = w_t (-min(r A_t, clip(r, 1 - lo, 1 + hi) A_t)
 *                                 + c (exp(ref_t - lp) - (ref_t - lp) - 1)),
 *                   lp = log softmax(z_t)[label_t], r = exp(lp - old_t)
 *
 * Types.  `dtype` is the type of the matrices (ADAPTERS_F32, ADAPTERS_BF16;
 * the losses also ADAPTERS_F16); every sum, softmax statistic and H is held
 * in FP32, every output is rounded once.  The FP32 projection is the
 * library's sgemm (3xTF32 or FFMA, its own choice); on bfloat16 matrices the
 * products run on the tensor cores with FP32 accumulators, and H and U enter
 * the projection and the gradients as two bfloat16 parts (16 bits).  A call's FP32 products are exact FP32 FMAs up to 32 rows or
 * 2^28 multiply-adds; above, the projection has sgemm's FP32 bound.
 *
 * Layout.  Row-major with leading dimensions in elements, offsets in 64
 * bits, any element-aligned pointers.  X is t x k, Y is t x n; W is k x n
 * (op_w = SGEMM_OP_N) or stored n x k (SGEMM_OP_T).  The adapters are two
 * contiguous stacks with the rank outside: A is l x r x k and B is l x r x n
 * (an adapter's "down" matrix as a linear layer stores it, and its "up"
 * matrix transposed), so that every product reads rows of consecutive k or
 * n.  Ranks below r are stored with rows of zeros.  ids[t] is row t's
 * adapter; a row whose id is outside 0 .. l-1 (say -1) has none: its H, U
 * and contribution to the gradients are zero.  scale (l values) may be
 * NULL: 1.  H, where given, is t x r FP32, contiguous; it includes the scale.
 *
 * Losses.  logits z is t x v with row pitch ldz; grad has z's type and
 * receives d(sum of loss)/dz; it may be NULL (no gradient), and it may be z
 * itself (same pointer and pitch), but must not overlap z otherwise.
 * weight (t values) may be NULL: 1.  A row counts for nothing -- loss 0,
 * gradient 0, whatever it holds -- when its weight is 0, when its label is
 * outside 0 .. v-1 (policy_loss), when none of its teacher places is usable
 * (distill_topk; a place is usable when its index is in 0 .. v-1 and its
 * teacher logit is not -inf), or when all of its logits are -inf.  Places of
 * one row may name an index twice: their q add up.
 *
 * Ownership, execution, streams.  As in sgemm_gb300.h: caller-owned device
 * pointers, everything enqueued on `stream` of the current device without
 * synchronising, thread-safe, capturable into a CUDA graph after a first
 * call has done the device's one-time set-up.  Scratch (H where it is not
 * given, U, partial sums, copies of matrices whose rows TMA cannot read)
 * comes from a stream-ordered pool of its own per device, which keeps up to
 * 256 MiB mapped between calls; the losses take none.  Outputs must not
 * overlap inputs (but for grad, above).  Results do not depend on the order
 * in which blocks run: the same call gives the same bits.
 *
 * Errors.  0, the 1-based position of the first invalid argument (sizes < 0;
 * a pointer NULL while it is needed, or not aligned to its elements; a
 * leading dimension below the row; an unknown dtype or op), or
 * SGEMM_STATUS_CUDA_ERROR (adapters_last_cuda_error() has the code, per
 * thread).  Argument errors and failed allocations return before anything is
 * enqueued.
 */
#ifndef ADAPTERS_GB300_H
#define ADAPTERS_GB300_H

#include "sgemm_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif

#define ADAPTERS_F32 0
#define ADAPTERS_BF16 1
#define ADAPTERS_F16 2 /* losses only */

#define ADAPTERS_MAX_RANK 256
#define ADAPTERS_MAX_TOP 1024

/*
 * lora_forward -- see the file comment.  H (argument 18) may be NULL; a
 * training step keeps it for lora_backward.  Rank 0 or l = 0: Y = X W.
 * k = 0: Y = 0.  ids may be NULL when r or l is 0.
 */
int lora_forward(int t, int k, int n, int l, int r, int dtype, const void *X, int ldx, int op_w, const void *W,
                 int ldw, const void *A, const void *B, const int *ids, const float *scale, void *Y, int ldy, float *H,
                 cudaStream_t stream);

/*
 * lora_backward -- W is frozen: the gradients by X and by the adapters.  dX,
 * dA and dB may each be NULL (not wanted); H is read only for dB, X only
 * for dA, W only for dX.  dA and dB are written whole (an adapter without
 * rows gets zeros) and have the matrices' type.
 */
int lora_backward(int t, int k, int n, int l, int r, int dtype, const void *dY, int lddy, const void *X, int ldx,
                  int op_w, const void *W, int ldw, const void *A, const void *B, const int *ids, const float *scale,
                  const float *H, void *dX, int lddx, void *dA, void *dB, cudaStream_t stream);

/*
 * distill_topk -- teacher and index are t x top, contiguous; top is 1 ..
 * ADAPTERS_MAX_TOP; temperature tau > 0 and finite, log2(e) / tau finite too
 * (tau above 4.24e-39).  loss: t values.
 */
int distill_topk(int t, int v, int top, int dtype, const void *logits, int ldz, const float *teacher,
                 const int *index, const float *weight, float temperature, float *loss, void *grad, int ldg,
                 cudaStream_t stream);

/*
 * policy_loss -- labels, old_logp, advantage and loss hold t values; ref and
 * weight may be NULL (no KL term; weight 1); kl_coef needs ref unless it is
 * 0.  logp, where given, receives lp of every row whose label is in range
 * (of weight 0 too), and 0 for the others.  clip_low and clip_high >= 0.  A
 * row whose min(r A, clip(r) A) is not a number (a NaN, or a ratio that
 * overflows beside an advantage of 0) has a loss and a gradient that are not.
 */
int policy_loss(int t, int v, int dtype, const void *logits, int ldz, const int *labels, const float *old_logp,
                const float *advantage, const float *ref, const float *weight, float clip_low, float clip_high,
                float kl_coef, float *loss, float *logp, void *grad, int ldg, cudaStream_t stream);

/* Static description of a status of these calls. */
const char *adapters_status_string(int status);

/* cudaError_t value of the last SGEMM_STATUS_CUDA_ERROR of these calls on this thread. */
int adapters_last_cuda_error(void);

/*
 * How the current device runs the bfloat16 projection of t rows from k to n
 * features (all at least 1): rows of an output tile, CTAs that share a
 * tile's contraction, whether tiles are CTA pairs', and the most tiles that
 * one of them takes in turn.
 */
typedef struct {
    int rows, split, pair, tiles;
} adapters_plan;
int adapters_plan_for(int t, int k, int n, adapters_plan *plan);

/*
 * The bounded waits of the tensor-core kernels of these calls, as
 * sgemm_device_status: synchronises the device, copies the first recorded
 * code (0: none) to *flag and resets it when `clear` is non-zero.
 */
int adapters_device_status(int *flag, int clear);

#ifdef __cplusplus
}
#endif

#endif /* ADAPTERS_GB300_H */
