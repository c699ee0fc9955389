// lp_tune_internal.h: launchers of the fine-tuning operators, shared between their
// C-ABI front end (lp_tune_api.cu) and the kernel translation units.  Arguments
// reaching these functions have already been validated.
#pragma once

#include "../../include/lp_tune.h"

#include "lp_train_internal.h"

namespace lp {

// ------------------------------------------------------------------- layer norm

struct LayerNormArgs {
  Rows residual, branch;     // branch.p may be null
  const void *weight, *bias; // may be null
  bool residual_bf16, act_bf16, weight_bf16;
  int64_t T, d;
  float eps;
  Rows residual_out, normed; // residual_out.p null without branch
  float *mean, *rstd;        // may be null
};
lp_status launch_layer_norm(const Device& dev, const LayerNormArgs& a, cudaStream_t stream);

struct LayerNormGradArgs {
  Rows residual_out;
  const void* weight;        // may be null
  bool residual_bf16, act_bf16, weight_bf16;
  int64_t T, d;
  const float *mean, *rstd;
  Rows grad_normed, grad_residual_out;  // grad_residual_out.p may be null
  Rows grad_residual, grad_branch;      // grad_branch.p null to skip
  float *grad_weight, *grad_bias;       // null to skip
  float* partials;                      // workspace; null when no sum is asked for
};
size_t layer_norm_backward_workspace(int64_t T, int64_t d);
lp_status launch_layer_norm_backward(const Device& dev, const LayerNormGradArgs& a,
                                     cudaStream_t stream);

// -------------------------------------------------------------- preference loss

struct PreferenceArgs {
  const float *logp, *ref_logp;  // ref_logp may be null
  const uint8_t* mask;           // may be null
  const int64_t* cu_seqlens;
  int64_t T, n_sequences;
  int kind;                      // lp_preference
  bool average, halves;
  bool wide;                     // set by the launcher: rows may go 16 bytes at a time
  double beta, inverse_beta, margin, smoothing, nll_coef;
  float *stats, *rewards, *grad_logp;
  void* workspace;
};
size_t preference_loss_workspace(int64_t T, int64_t n_sequences);
lp_status launch_preference_loss(const PreferenceArgs& a, cudaStream_t stream);

// Read and clear the check words of these translation units (lp_check.cuh).
cudaError_t take_check_word_layer_norm(uint32_t* out);
cudaError_t take_check_word_layer_norm_backward(uint32_t* out);
cudaError_t take_check_word_preference(uint32_t* out);

}  // namespace lp
