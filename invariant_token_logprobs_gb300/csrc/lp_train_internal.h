// lp_train_internal.h: launchers of the training-step operators, shared between
// their C-ABI front end (lp_train_api.cu) and the kernel translation units.
// Arguments reaching these functions have already been validated.
#pragma once

#include "../../include/lp_train.h"
#include <cuda_bf16.h>

#include "lp_internal.h"

namespace lp {

// ---------------------------------------------------------------- residual norm

constexpr int64_t kNormMaxDim = 16384;

// A row operand: its base and row stride in elements.
struct Rows {
  void* p;
  int64_t ld;
};

struct NormArgs {
  Rows residual, branch, gate;  // branch.p / gate.p may be null; gate.ld == 0: one row
  const void* branch_weight;    // may be null
  const void* weight;           // may be null
  bool residual_bf16, act_bf16, weight_bf16;
  int64_t T, d;
  float residual_scale, branch_scale, eps;
  Rows residual_out, normed;    // null where absent
  float* branch_rstd;           // may be null
  float* rstd;                  // may be null
};
lp_status launch_residual_norm(const Device& dev, const NormArgs& a, cudaStream_t stream);

struct NormGradArgs {
  Rows residual_out, branch, gate;
  const void* branch_weight;
  const void* weight;
  bool residual_bf16, act_bf16, weight_bf16;
  int64_t T, d;
  float residual_scale, branch_scale;
  const float* branch_rstd;
  const float* rstd;
  Rows grad_normed, grad_residual_out;  // null where absent
  Rows grad_residual, grad_branch;
  Rows grad_gate;               // null to skip; float32 [d] when gate.ld == 0
  float* grad_branch_weight;    // null to skip
  float* grad_weight;           // null to skip
  float* partials;              // workspace; null when no sum is asked for
};
size_t residual_norm_backward_workspace(int64_t T, int64_t d);
lp_status launch_residual_norm_backward(const Device& dev, const NormGradArgs& a,
                                        cudaStream_t stream);

// ------------------------------------------------------------------ policy loss

struct PolicyArgs {
  const float *logp, *old_logp, *ref_logp, *entropy, *advantages;
  bool per_sequence, by_sequence;
  const uint8_t* mask;
  const int64_t* cu_seqlens;  // null when neither flag above is set
  int64_t T, n_sequences;
  float low, high;            // the clip's limits on delta
  float ratio_low, ratio_high;
  float kl_coef, entropy_coef;
  bool wide;                  // set by the launcher: rows may go 16 bytes at a time
  float *stats, *grad_logp, *grad_entropy;
  void* workspace;
};
size_t policy_loss_workspace(int64_t T, int64_t n_sequences);
lp_status launch_policy_loss(const PolicyArgs& a, cudaStream_t stream);

// ------------------------------------------------------------------------ AdamW

// One tensor's record in the device plan.
struct AdamwRecord {
  float* param;
  __nv_bfloat16* copy;
  const void* grad;
  int64_t n;
  int64_t first_row;  // its first row of LP_ADAMW_ALIGN elements in the flat buffers
  float lr_scale;
  float weight_decay;
  int32_t grad_bf16;
  int32_t wide;  // every pointer is 16-byte aligned (8-byte for bfloat16 ones)
};
static_assert(sizeof(AdamwRecord) == 56, "plan layout");

// The plan: the records, then one int32 tensor index for each row.
inline size_t adamw_table_offset(int64_t n_tensors) {
  return (static_cast<size_t>(n_tensors) * sizeof(AdamwRecord) + 255) / 256 * 256;
}

struct AdamwArgs {
  const AdamwRecord* records;
  const int32_t* table;
  int64_t n_tensors, rows;  // rows of LP_ADAMW_ALIGN state elements
  void *exp_avg, *exp_avg_sq;
  float *exp_avg_scale, *exp_avg_sq_scale;  // null: 32-bit moments
  float lr, step_size, beta1, beta2, rest1, rest2, root_scale, eps;
  uint64_t step, seed;
  uint32_t round_keys[7][2];  // of the random words, set by the launcher from seed
  const float* grad_scale;
};
lp_status launch_adamw_step(const AdamwArgs& a, cudaStream_t stream);
size_t adamw_grad_norm_workspace(int64_t rows);
lp_status launch_adamw_grad_norm(const AdamwRecord* records, const int32_t* table,
                                 int64_t n_tensors, int64_t rows, float max_norm, float* norm_out,
                                 void* workspace, cudaStream_t stream);
lp_status launch_adamw_state_values(const void* exp_avg, const void* exp_avg_sq,
                                    const float* exp_avg_scale, const float* exp_avg_sq_scale,
                                    int64_t rows, float* m_out, float* v_out, cudaStream_t stream);

// Read and clear the check words of these translation units (lp_check.cuh).
cudaError_t take_check_word_norm(uint32_t* out);
cudaError_t take_check_word_norm_backward(uint32_t* out);
cudaError_t take_check_word_policy(uint32_t* out);
cudaError_t take_check_word_adamw(uint32_t* out);

}  // namespace lp
