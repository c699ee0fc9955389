/*
 * lp_tune.h: C ABI of liblp's fine-tuning operators on GB300 (sm_103a), beside
 * the training-step operators of lp_train.h:
 *
 *   layer norm       the sum of a residual stream and a block's output, and its
 *                    layer norm (the H of lp_linear_logprob for models whose
 *                    head is fed by one), in one pass; and its backward pass.
 *   preference loss  the loss of pairs of a chosen and a rejected sequence, from
 *                    the selected tokens' log-probabilities, with the grad_logp
 *                    that lp_linear_logprob_backward takes.
 *   Muon             one optimizer step over many matrices, whose momentum is
 *                    orthogonalised by Newton-Schulz products.
 *
 * The conventions are those of lp.h and lp_train.h: pointers are device memory
 * owned by the caller unless a comment says host, nothing is allocated, all work
 * is enqueued on `stream` without synchronising with the host, argument errors
 * are returned before anything is enqueued, and the current device must be of
 * compute capability 10.3.  Strides are in elements.  Data on the device (row
 * offsets, masks, NaN or infinities) never makes a call fault.
 */
#ifndef LP_TUNE_H_
#define LP_TUNE_H_

#include "lp_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Layer norm.  Per row of d channels, with residual stream r and block output
 * (branch) y:
 *
 *     r' = r + y
 *     h  = (r' - mean) * rstd * weight + bias,  rstd = rsqrt(mean((r' - mean)^2) + eps)
 *
 * branch, weight and bias are optional (without branch r' = r).  All arithmetic
 * and the sums are float32; the squares are of the deviations from the row's
 * mean, h is formed from the unrounded r', and each output is rounded once.  A
 * row's results do not depend on the other rows, on T or on the row's place.
 * ------------------------------------------------------------------------ */

/*
 * lp_layer_norm:
 *   residual      [T, d] residual_dtype, row stride ld_residual >= d.
 *   branch        [T, d] act_dtype, row stride ld_branch >= d, or NULL.
 *   weight, bias  [d] weight_dtype, or NULL.
 *   T >= 0 (0 enqueues nothing), 1 <= d <= 16384, eps >= 0 and finite.
 *   residual_out  [T, d] residual_dtype, required with branch and NULL without;
 *                 it may be `residual` itself (same pointer and stride).
 *   normed        [T, d] act_dtype, required.
 *   mean, rstd    [T] float32, or NULL: for the backward pass.
 * Pointers are aligned to their element; rows that all start on multiples of 8
 * elements, in memory and by their strides, with d a multiple of 8, are read and
 * written 8 columns at a time; others are slower, with the same results.  Outputs
 * must not overlap the inputs or one another, other than residual_out in place
 * (LP_ERR_INVALID_ARGUMENT).
 */
LP_API lp_status lp_layer_norm(const void* residual, int64_t ld_residual, int residual_dtype,
                               const void* branch, int64_t ld_branch, int act_dtype,
                               const void* weight, const void* bias, int weight_dtype, int64_t T,
                               int64_t d, float eps, void* residual_out, int64_t ld_residual_out,
                               void* normed, int64_t ld_normed, float* mean, float* rstd,
                               void* stream);

/* Workspace bytes of lp_layer_norm_backward; 0 for invalid sizes. */
LP_API size_t lp_layer_norm_backward_workspace_size(int64_t T, int64_t d);

/*
 * lp_layer_norm_backward: the gradients of lp_layer_norm from those of its
 * outputs.  With x = (r' - mean) * rstd and dx = grad_normed * weight:
 *     D = grad_residual_out + rstd * (dx - mean(dx) - x * mean(dx * x))
 *     grad_residual = grad_branch = D
 *     grad_weight = sum_t grad_normed * x;   grad_bias = sum_t grad_normed
 *
 *   residual_out  [T, d] residual_dtype: the forward's residual_out (its
 *                 `residual` when it had no branch).
 *   weight        the forward's, or NULL.
 *   mean, rstd    [T] float32 from the forward.
 *   grad_normed   [T, d] act_dtype.
 *   grad_residual_out  [T, d] residual_dtype, or NULL (zero).
 *   grad_residual [T, d] residual_dtype; may be grad_residual_out itself.
 *   grad_branch   [T, d] act_dtype: the same gradient in the branch's type, or
 *                 NULL to skip (it is grad_residual where the types are equal).
 *   grad_weight, grad_bias  [d] float32, each NULL to skip.
 *   workspace     256-byte aligned, lp_layer_norm_backward_workspace_size(T, d)
 *                 bytes; its contents on entry do not matter.  NULL when neither
 *                 sum is asked for.
 * T >= 1 rows are summed in a fixed order (float32), so repeated calls give the
 * same bits; T == 0 writes zeros to the summed gradients.
 */
LP_API lp_status lp_layer_norm_backward(
    const void* residual_out, int64_t ld_residual_out, int residual_dtype, int act_dtype,
    const void* weight, int weight_dtype, int64_t T, int64_t d, const float* mean,
    const float* rstd, const void* grad_normed, int64_t ld_grad_normed,
    const void* grad_residual_out, int64_t ld_grad_residual_out, void* grad_residual,
    int64_t ld_grad_residual, void* grad_branch, int64_t ld_grad_branch, float* grad_weight,
    float* grad_bias, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Preference loss.  Sequence i has the rows [cu_seqlens[i], cu_seqlens[i + 1]),
 * of which those count whose mask is not zero, n_i of them.  Its score is
 *
 *     s_i = sum over its counted rows of (logp - ref_logp)      (divided by n_i with `average`)
 *
 * and a pair of a chosen sequence c and a rejected one r, which counts when both
 * have a counted row, has z = beta (s_c - s_r) - margin and the loss
 *
 *     SIGMOID  (1 - e) log(1 + exp(-z)) + e log(1 + exp(z)),  e = label_smoothing
 *     HINGE    max(0, 1 - z)
 *     SQUARE   ((z - 1/2) / beta)^2
 *
 * plus nll_coef times the chosen sequence's mean of -logp.  The call's loss is
 * the mean over the counted pairs; without one everything is 0.  Rows that do
 * not count have no gradient whatever they hold (their logp is NaN where the
 * target is padding), and neither do the rows of pairs that do not count.
 *
 * Sums, scores, means and z are held as pairs of float32, 48 bits less what a sum's chain of
 * additions loses: 2^-37 of the terms' size for 10^5 rows, 2^-35 for 10^6.  So differences
 * of such sums keep float32's precision.  The sums are taken in a fixed order.
 * ------------------------------------------------------------------------ */

typedef enum lp_preference {
  LP_PREFERENCE_SIGMOID = 0,
  LP_PREFERENCE_HINGE = 1,
  LP_PREFERENCE_SQUARE = 2
} lp_preference;

/* Workspace bytes of lp_preference_loss for T rows in n_sequences; 0 for invalid sizes. */
LP_API size_t lp_preference_loss_workspace_size(int64_t T, int64_t n_sequences);

/*
 * lp_preference_loss:
 *   logp            [T] float32.
 *   ref_logp        [T] float32, or NULL (zero: no reference).
 *   mask            [T] bytes (0: the row does not count), or NULL (all count).
 *   cu_seqlens      [n_sequences + 1] int64 ascending row offsets; rows in no sequence
 *                   do not count.
 *   n_sequences     even.  Pair i is of the sequences 2 i (chosen) and 2 i + 1
 *                   (rejected), or with `halves` of i and i + n_sequences / 2.
 *   kind            an lp_preference.
 *   beta > 0, margin, 0 <= label_smoothing <= 1 (0 unless SIGMOID), nll_coef: finite in
 *                   float32, beta and 1 / beta no subnormals; with an nll_coef of 0 the
 *                   term is in the stats alone, whatever it holds.
 *   stats           [6] float32: the loss, and the means over the counted pairs of the
 *                   loss without the nll term, of the chosen's -logp, of s_c > s_r, and of
 *                   beta s_c and beta s_r.
 *   rewards         [n_sequences] float32: beta s_i, 0 for a sequence without a counted row.
 *   grad_logp       [T] float32, d loss / d logp.
 *   workspace       256-byte aligned, lp_preference_loss_workspace_size(T, n_sequences)
 *                   bytes; its contents on entry do not matter.
 * 0 <= T < 2^31, 0 <= n_sequences < 2^31.
 */
LP_API lp_status lp_preference_loss(const float* logp, const float* ref_logp, const uint8_t* mask,
                                    const int64_t* cu_seqlens, int64_t T, int64_t n_sequences,
                                    int kind, int average, int halves, double beta, double margin,
                                    double label_smoothing, double nll_coef, float* stats,
                                    float* rewards, float* grad_logp, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Muon over many matrices.  Per matrix, with gradient g and momentum M:
 *
 *     M = momentum M + g;   u = g + momentum M  (nesterov), or u = M
 *     X = u / (|u| + eps),  |u| the Frobenius norm
 *     steps times:  X = a X + b (X X^T) X + c (X X^T)^2 X,  a, b, c = 3.4445, -4.7750, 2.0315
 *     p = p (1 - l weight_decay) - l update_scale X,  l = lr * lr_scale
 *
 * which takes the singular values of X towards 1 and leaves its directions.  p and
 * M are float32; a bfloat16 copy of p is written in the same pass when asked.  The
 * products are taken on the tensor cores with operands of 22 bits (pairs of
 * float16) and float32 sums, on the smaller side of the matrix.  The 22 bits are those of
 * elements of X above 2^-16 of its norm; smaller ones keep an absolute 2^-39 of it.  (X is
 * held by a power of two that an eps above |u| does not take from it.)  The tensor core cuts sums off
 * where float32 rounds, for 512 of K at a time.  |u| is a float32 sum of squares: elements
 * below 2^-63 lose theirs, which shows beside an eps of less than 1e-14.
 *
 * A matrix whose |u| is not finite in float32 (a NaN or an infinity, or squares
 * past its range) keeps its p, its copy and its M; the others are not touched by it.
 * ------------------------------------------------------------------------ */

typedef struct lp_muon_tensor {
  float* param;        /* [rows, cols] float32, contiguous */
  void* copy;          /* bfloat16 copy of param to write, or NULL */
  const void* grad;    /* [rows, cols] grad_dtype, contiguous */
  float* momentum;     /* [rows, cols] float32, contiguous; zero before the first step */
  int64_t rows, cols;  /* 0 .. 65536 each */
  float lr_scale;      /* finite, >= 0 */
  float weight_decay;  /* finite, >= 0 */
  float update_scale;  /* finite, >= 0: the factor that the shape gives, such as
                          sqrt(max(1, rows / cols)) or 0.2 sqrt(max(rows, cols)) */
  int grad_dtype;      /* an lp_dtype */
} lp_muon_tensor;

/* Bytes of the plan of these matrices; 0 for invalid arguments.  Host function;
 * `tensors` is host memory. */
LP_API size_t lp_muon_plan_size(const lp_muon_tensor* tensors, int64_t n_tensors);

/*
 * lp_muon_plan: lay out the plan of a step over `tensors` (host memory) in `plan_host`
 * (host memory, 8-byte aligned, lp_muon_plan_size bytes).  Keep it, copy it to
 * 256-byte aligned device memory once, and pass both to lp_muon_step; lay it out
 * again when a pointer, shape or factor changes.  Pointers are aligned to their
 * element; matrices whose pointers are multiples of 16 bytes and whose cols are a
 * multiple of 4 go 16 bytes at a time, with the same results.  A matrix must not
 * appear twice, and what a step writes (params, copies, momenta) may not share memory
 * with another matrix's tensors: a matrix's own are compared here, those of others
 * are the caller's to keep apart.  Host function.
 */
LP_API lp_status lp_muon_plan(const lp_muon_tensor* tensors, int64_t n_tensors, void* plan_host,
                              size_t plan_bytes);

/* Workspace bytes of lp_muon_step; 0 when plan_host is no plan.  Host function. */
LP_API size_t lp_muon_workspace_size(const void* plan_host);

/*
 * lp_muon_step: one step over every matrix of the plan.
 *   plan_host      host memory, as laid out by lp_muon_plan; read during the call only.
 *   plan           device memory, 256-byte aligned: its copy.
 *   lr >= 0, 0 <= momentum < 1, 1e-16 <= eps, all finite; 1 <= steps <= 32.
 *   workspace      256-byte aligned, lp_muon_workspace_size(plan_host) bytes; its
 *                  contents on entry do not matter.
 * lr and momentum are arguments of the launch: a captured call keeps them at every
 * replay.  The matrices go through the workspace in batches, in their order, of up to 2^26
 * elements (each side rounded up to 128) or of one matrix.  If a device-side wait gives up,
 * the params of its batch are NaN, whichever matrix it was for, those of the other batches
 * are not, and lp_get_device_error on the workspace says so.
 */
LP_API lp_status lp_muon_step(const void* plan_host, const void* plan, double lr, double momentum,
                              int nesterov, int steps, double eps, void* workspace,
                              size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LP_TUNE_H_ */
