/*
 * lp_train.h: C ABI of liblp's training-step operators on GB300 (sm_103a),
 * the calls on either side of the selected-token log-probabilities of lp.h:
 *
 *   residual norm  the norm of a block's output, its gate and residual scale,
 *                  and the norm of the new residual stream that feeds the next
 *                  block or the LM head (the H of lp_linear_logprob), in one
 *                  pass; and its backward pass.
 *   policy loss    the clipped policy-gradient loss of the log-probabilities,
 *                  with the grad_logp and grad_entropy that
 *                  lp_linear_logprob_backward takes.
 *   AdamW          one optimizer step over many tensors at once, with moments
 *                  in 32 bits or in 8, and the clip of the global gradient norm.
 *
 * The conventions are those of lp.h: pointers are device memory owned by the
 * caller unless a comment says host, nothing is allocated, all work is
 * enqueued on `stream` without synchronising with the host, argument errors
 * are returned before anything is enqueued, and the current device must be of
 * compute capability 10.3.  Strides are in elements.  Data on the device (row
 * offsets, masks, NaN or infinities) never makes a call fault.
 */
#ifndef LP_TRAIN_H_
#define LP_TRAIN_H_

#include "lp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
typedef enum lp_dtype { LP_FLOAT32 = 0, LP_BFLOAT16 = 1 } lp_dtype;

/* ------------------------------------------------------------------------
 * Residual norm.  Per row of d channels, with residual stream r, block output
 * (branch) y, gate g, scales a = residual_scale and b = branch_scale:
 *
 *     n  = y * rsqrt(mean(y^2) + eps) * branch_weight     (norm after the block)
 *     r' = a * r + b * g * n
 *     h  = r' * rsqrt(mean(r'^2) + eps) * weight          (norm before the next)
 *
 * Every part is optional: without branch_weight n = y, without gate g = 1,
 * without weight there is no h, and without branch r' = r (a must be 1).  All
 * arithmetic and both sums are float32; h is formed from the unrounded r', and
 * each output is rounded once.  A row's results do not depend on the other
 * rows, on T or on the row's place.
 * ------------------------------------------------------------------------ */

/*
 * lp_residual_norm:
 *   residual      [T, d] residual_dtype, row stride ld_residual >= d.
 *   branch        [T, d] act_dtype, row stride ld_branch >= d, or NULL.
 *   gate          act_dtype: [T, d] with row stride ld_gate >= d, or one row [d]
 *                 for all (ld_gate == 0), or NULL; needs branch.
 *   branch_weight, weight  [d] weight_dtype or NULL; branch_weight needs branch,
 *                 and one of branch and weight must be given.
 *   T >= 0 (0 enqueues nothing), 1 <= d <= 16384, eps >= 0 and finite.
 *   residual_out  [T, d] residual_dtype, required with branch and NULL without;
 *                 it may be `residual` itself (same pointer and stride).
 *   normed        [T, d] act_dtype, required with weight and NULL without.
 *   branch_rstd, rstd  [T] float32, or NULL: the reciprocal roots
 *                 rsqrt(mean + eps) of the two norms, for the backward pass;
 *                 branch_rstd needs branch_weight and rstd needs weight.
 * Pointers are aligned to their element; rows that all start on multiples of 8
 * elements, in memory and by their strides, with d a multiple of 8, are read and
 * written 8 columns at a time; others are slower, with the same results.  Outputs
 * must not overlap the inputs or one another, other than residual_out in place
 * (LP_ERR_INVALID_ARGUMENT).
 */
LP_API lp_status lp_residual_norm(const void* residual, int64_t ld_residual, int residual_dtype,
                                  const void* branch, int64_t ld_branch, const void* gate,
                                  int64_t ld_gate, int act_dtype, const void* branch_weight,
                                  const void* weight, int weight_dtype, int64_t T, int64_t d,
                                  float residual_scale, float branch_scale, float eps,
                                  void* residual_out, int64_t ld_residual_out, void* normed,
                                  int64_t ld_normed, float* branch_rstd, float* rstd,
                                  void* stream);

/* Workspace bytes of lp_residual_norm_backward; 0 for invalid sizes. */
LP_API size_t lp_residual_norm_backward_workspace_size(int64_t T, int64_t d);

/*
 * lp_residual_norm_backward: the gradients of lp_residual_norm from those of
 * its outputs.  With x = r' * rstd, yh = y * branch_rstd, dx = grad_normed *
 * weight:
 *     D = grad_residual_out + rstd * (dx - x * mean(dx * x))
 *     grad_residual = a * D;   grad_gate = b * D * n  (summed over the rows for one row [d])
 *     grad_weight = sum_t grad_normed * x;   grad_branch_weight = sum_t b * g * D * yh
 *     grad_branch = branch_rstd * (e - yh * mean(e * yh)),  e = b * g * D * branch_weight
 * (without branch_weight grad_branch = b * g * D).  mean(e * yh) is taken with
 * mean(dx * x) in one round of float32 sums, as mean(f * (grad_residual_out + rstd *
 * dx)) - rstd * mean(dx * x) * mean(f * x) with f = b * g * branch_weight * yh.
 *
 *   residual_out  [T, d] residual_dtype: the forward's residual_out (its
 *                 `residual` when it had no branch).  NULL when weight is NULL.
 *   branch, gate, branch_weight, weight, T, d, scales: the forward's.
 *   branch_rstd, rstd  [T] float32 from the forward; required with
 *                 branch_weight and weight.
 *   grad_normed   [T, d] act_dtype, required with weight and NULL without.
 *   grad_residual_out  [T, d] residual_dtype, or NULL (zero) when weight is given.
 *   grad_residual [T, d] residual_dtype; may be grad_residual_out itself.
 *   grad_branch   [T, d] act_dtype, required with branch.
 *   grad_gate     NULL to skip; [T, d] act_dtype (row stride ld_grad_gate) for a
 *                 gate of T rows, [d] float32 for a gate of one row.
 *   grad_branch_weight, grad_weight  [d] float32, each NULL to skip.
 *   workspace     256-byte aligned, lp_residual_norm_backward_workspace_size(T, d)
 *                 bytes; its contents on entry do not matter.
 * T >= 1 rows are summed in a fixed order (float32), so repeated calls give the
 * same bits; T == 0 writes zeros to the summed gradients.
 */
LP_API lp_status lp_residual_norm_backward(
    const void* residual_out, int64_t ld_residual_out, int residual_dtype, const void* branch,
    int64_t ld_branch, const void* gate, int64_t ld_gate, int act_dtype, const void* branch_weight,
    const void* weight, int weight_dtype, int64_t T, int64_t d, float residual_scale,
    float branch_scale, const float* branch_rstd, const float* rstd, const void* grad_normed,
    int64_t ld_grad_normed, const void* grad_residual_out, int64_t ld_grad_residual_out,
    void* grad_residual, int64_t ld_grad_residual, void* grad_branch, int64_t ld_grad_branch,
    void* grad_gate, int64_t ld_grad_gate, float* grad_branch_weight, float* grad_weight,
    void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Policy loss.  Per row t that counts (mask[t] != 0), with advantage A, delta =
 * logp - old_logp (the float32 difference) and rho = exp(delta):
 *
 *     policy = -min(rho * A, clip(rho, 1 - clip_low, 1 + clip_high) * A)
 *     kl     = exp(r) - r - 1,  r = ref_logp - logp
 *     loss   = sum_t w_t (policy + kl_coef * kl - entropy_coef * entropy)
 *
 * A row is clipped when A > 0 and delta > log1p(clip_high), or A < 0 and
 * delta < log1p(-clip_low) (limits rounded to float32); its policy term then
 * has no gradient.  The weights are w = 1 / N for N counted rows in all
 * (LP_REDUCE_TOKEN), or w = 1 / (n_i S) for a row of sequence i with n_i counted
 * rows among S sequences that have any (LP_REDUCE_SEQUENCE).  Rows that do not
 * count have weight 0 whatever they hold (their logp is NaN where the target is
 * padding), and without any counted row everything is 0.
 * ------------------------------------------------------------------------ */

typedef enum lp_reduction { LP_REDUCE_TOKEN = 0, LP_REDUCE_SEQUENCE = 1 } lp_reduction;

/* Workspace bytes of lp_policy_loss for T rows in n_sequences; 0 for invalid sizes. */
LP_API size_t lp_policy_loss_workspace_size(int64_t T, int64_t n_sequences);

/*
 * lp_policy_loss:
 *   logp, old_logp  [T] float32.
 *   ref_logp        [T] float32, or NULL (no kl term; kl_coef is not used).
 *   entropy         [T] float32, or NULL (no entropy term).
 *   kl_coef, entropy_coef  finite; with 0 the term is in the stats alone, whatever it holds.
 *   advantages      [T] float32, or [n_sequences] when advantages_per_sequence != 0.
 *   mask            [T] bytes (0: the row does not count), or NULL (all count).
 *   cu_seqlens      [n_sequences + 1] int64 ascending row offsets: sequence i is the
 *                   rows [cu_seqlens[i], cu_seqlens[i + 1]); rows in no sequence do not
 *                   count.  NULL (and not read) when reduction is LP_REDUCE_TOKEN and
 *                   advantages are per row.
 *   clip_low in [0, 1), clip_high >= 0.
 *   stats           [5] float32: loss, the sums over t of w policy, w kl and w entropy,
 *                   and the weight of the clipped rows.
 *   grad_logp       [T] float32, d loss / d logp; grad_entropy [T] float32,
 *                   d loss / d entropy, required with entropy and NULL without.
 *   workspace       256-byte aligned, lp_policy_loss_workspace_size(T, n_sequences) bytes.
 * 0 <= T < 2^31, 0 <= n_sequences < 2^31.  The sums are taken in a fixed order.
 */
LP_API lp_status lp_policy_loss(const float* logp, const float* old_logp, const float* ref_logp,
                                const float* entropy, const float* advantages,
                                int advantages_per_sequence, const uint8_t* mask,
                                const int64_t* cu_seqlens, int64_t T, int64_t n_sequences,
                                int reduction, double clip_low, double clip_high, double kl_coef,
                                double entropy_coef, float* stats, float* grad_logp,
                                float* grad_entropy, void* workspace, size_t workspace_bytes,
                                void* stream);

/* ------------------------------------------------------------------------
 * AdamW over many tensors.  Per element, with gradient g (scaled by the clip
 * coefficient when there is one), float32 throughout:
 *
 *     m = beta1 m + (1 - beta1) g;   v = beta2 v + (1 - beta2) g^2
 *     p = p (1 - l weight_decay) - (l / (1 - beta1^t)) m / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * with l = lr * lr_scale of the tensor.  p is float32; a bfloat16 copy of it
 * (the weights the forward pass reads) is written in the same pass when asked.
 * The moments' products and sums are each rounded once; the change of p divides by
 * way of an approximate reciprocal, within 3 units in the last place of the change.
 *
 * The moments of all tensors lie in flat buffers: tensor i's start at the sum
 * over the tensors before it of their lengths rounded up to
 * LP_ADAMW_ALIGN.  Set them to zero before the first step.
 *
 * 8-bit moments hold m and u = sqrt(v) in one byte each, with one float32
 * scale for LP_ADAMW_BLOCK consecutive elements of a tensor: the block's
 * largest magnitude (0 when below 2^-100).  A magnitude relative to the scale
 * is held as a code c: 0 for zero, else the float whose bits are
 * (c + 889) << 20 for m (7 bits, 8 steps an octave, bit 7 the sign) or
 * (c + 1777) << 19 for u (8 bits, 16 steps an octave): 1 at the largest code
 * down to about 2^-16.  They are rounded up with the probability of the part
 * cut off (to 16 bits), so that a decay of 0.1% a step, far less than a step of
 * the code, is kept on average: m and u come out without bias, and v = u^2 2 to 3%
 * high on average (u itself under 1% over the root of the averaged squares).  A
 * magnitude below code 1 becomes zero or code 1.  Where that leaves a u of zero
 * beside an m that is not, the next step divides that m by the root of its own
 * gradient's square alone, or by eps where that is zero: tensors whose blocks mix
 * magnitudes of 2^16 and more apart want 32 bits, or an eps of that part of their
 * largest gradients.  The random bits are those of Philox 4x32 with
 * 7 rounds (Salmon et al., SC11) at counter (flat index / 4, t) and key seed;
 * the low half of word (flat index mod 4) rounds m, the high half u.  The
 * update itself uses the moments before they are rounded.  A block with a NaN
 * or an infinity reads back as NaN.
 * ------------------------------------------------------------------------ */

#define LP_ADAMW_ALIGN 2048
#define LP_ADAMW_BLOCK 256

typedef struct lp_adamw_tensor {
  float* param;        /* [n] float32 */
  void* copy;          /* [n] bfloat16 copy of param to write, or NULL */
  const void* grad;    /* [n] grad_dtype */
  int64_t n;           /* elements, >= 0 */
  float lr_scale;      /* finite, >= 0 */
  float weight_decay;  /* finite, >= 0 */
  int grad_dtype;      /* an lp_dtype */
  int reserved;        /* 0 */
} lp_adamw_tensor;

/* Elements of each flat moment buffer; -1 for invalid arguments.  Host function;
 * `tensors` is host memory. */
LP_API int64_t lp_adamw_state_elements(const lp_adamw_tensor* tensors, int64_t n_tensors);

/* Bytes of the plan of these tensors; 0 for invalid arguments.  Host function. */
LP_API size_t lp_adamw_plan_size(const lp_adamw_tensor* tensors, int64_t n_tensors);

/*
 * lp_adamw_plan: lay out the plan of a step over `tensors` (host memory) in
 * `plan_host` (host memory, lp_adamw_plan_size bytes).  Copy it to 256-byte
 * aligned device memory once and pass it to the calls below; lay it out again
 * when a pointer, length or factor changes.  Pointers are aligned to their
 * element; tensors whose pointers are multiples of 16 bytes go 16 bytes at a
 * time, with the same results.  A tensor must not appear twice, and no param or copy
 * may share memory with another tensor's param, copy or gradient: a tensor's own are
 * compared here, those of others are the caller's to keep apart.  Host function.
 */
LP_API lp_status lp_adamw_plan(const lp_adamw_tensor* tensors, int64_t n_tensors, void* plan_host,
                               size_t plan_bytes);

/* Workspace bytes of lp_adamw_grad_norm; 0 for invalid sizes. */
LP_API size_t lp_adamw_grad_norm_workspace_size(int64_t state_elements);

/*
 * lp_adamw_grad_norm: norm_out[0] = the 2-norm of all gradients of the plan
 * (float32 within 2048 elements, float pairs across them, in a fixed order; an
 * infinity where the sum of the squares is none) and
 * norm_out[1] = min(1, max_norm / (norm + 1e-6)), NaN when the norm is not
 * finite.  plan, n_tensors and state_elements as in lp_adamw_step; max_norm > 0;
 * workspace 256-byte aligned.
 */
LP_API lp_status lp_adamw_grad_norm(const void* plan, int64_t n_tensors, int64_t state_elements,
                                    float max_norm, float* norm_out, void* workspace,
                                    size_t workspace_bytes, void* stream);

/*
 * lp_adamw_step: one step over every tensor of the plan.
 *   plan           device memory, 256-byte aligned, as laid out by lp_adamw_plan for
 *                  n_tensors tensors; state_elements is lp_adamw_state_elements of them.
 *   state_bits     32 or 8.
 *   exp_avg, exp_avg_sq  the moments: float32, or bytes of m and sqrt(v); 16-byte aligned.
 *   exp_avg_scale, exp_avg_sq_scale  [state_elements / LP_ADAMW_BLOCK] float32 for 8
 *                  bits, NULL for 32.
 *   grad_scale     [1] float32 that every gradient is multiplied by (norm_out + 1 of
 *                  lp_adamw_grad_norm), or NULL.  When it is NaN the step changes nothing.
 *   step           t >= 1, the number of this step; seed: of the 8-bit rounding.
 *                  step, lr and the betas are arguments of the launch: a captured call
 *                  repeats this step at every replay, with the same random bits.
 *   lr >= 0, 0 <= beta1, beta2 < 1, eps >= 2^-126 (as a float32), all finite.
 */
LP_API lp_status lp_adamw_step(const void* plan, int64_t n_tensors, int64_t state_elements,
                               int state_bits, void* exp_avg, void* exp_avg_sq,
                               float* exp_avg_scale, float* exp_avg_sq_scale, double lr,
                               double beta1, double beta2, double eps, int64_t step, uint64_t seed,
                               const float* grad_scale, void* stream);

/*
 * lp_adamw_state_values: the values 8-bit moments stand for, exp_avg_out = m and
 * exp_avg_sq_out = v = u^2, [state_elements] float32 each (16-byte aligned).
 */
LP_API lp_status lp_adamw_state_values(const void* exp_avg, const void* exp_avg_sq,
                                       const float* exp_avg_scale, const float* exp_avg_sq_scale,
                                       int64_t state_elements, float* exp_avg_out,
                                       float* exp_avg_sq_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LP_TRAIN_H_ */
