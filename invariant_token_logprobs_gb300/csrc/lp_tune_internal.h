// lp_tune_internal.h: launchers of the fine-tuning operators, shared between their
// C-ABI front end (lp_tune_api.cu) and the kernel translation units.  Arguments
// reaching these functions have already been validated.
#pragma once

#include <cuda.h>

#include "../../include/lp_tune.h"

#include "lp_train_internal.h"

namespace lp {

// The workspace as `rows` rows of 128 bytes, in boxes of box_rows whole rows, without a swizzle.  Returns
// false if the CUDA driver rejects it.
bool encode_rows128(CUtensorMap* map, const void* base, int64_t rows, int box_rows);

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

// A float64 as the sum of two float32.
struct Pair32 {
  float high, low;
};
inline Pair32 pair32(double v) {
  Pair32 p;
  p.high = static_cast<float>(v);
  p.low = static_cast<float>(v - static_cast<double>(p.high));
  return p;
}

struct PreferenceArgs {
  const float *logp, *ref_logp;  // ref_logp may be null
  const uint8_t* mask;           // may be null
  const int64_t* cu_seqlens;
  int64_t T, n_sequences;
  int kind;                      // lp_preference
  bool average, halves;
  bool wide;                     // set by the launcher: rows may go 16 bytes at a time
  Pair32 beta, inverse_beta, margin;
  float smoothing, nll_coef;
  float *stats, *rewards, *grad_logp;
  void* workspace;
};
size_t preference_loss_workspace(int64_t T, int64_t n_sequences);
lp_status launch_preference_loss(const PreferenceArgs& a, cudaStream_t stream);

// ------------------------------------------------------------------------- Muon

constexpr int64_t kMuonMagic = 0x6e6f756d2d706cll;  // of a plan's header
constexpr int64_t kMuonMaxDim = 65536;
constexpr int64_t kMuonPart = 4096;  // elements of a partial sum of the norm, at least

// One matrix's record in the plan.  x, g, p: byte offsets of its buffers in the workspace.
struct MuonRecord {
  float* param;
  __nv_bfloat16* copy;
  const void* grad;
  float* momentum;
  int64_t rows, cols, m, n;  // m <= n: the X that is orthogonalised, transposed when tall
  int64_t x[2], g, p;
  int64_t first_part, parts, part;  // its partial sums: the first, how many, of how many elements
  float lr_scale, weight_decay, update_scale;
  int32_t grad_bf16, tall, wide;
};
// A CTA's work: a partial sum, or a block or tile (i, j) of a matrix.
struct MuonUnit {
  int32_t tensor, part;
  int16_t i, j;
};
// Matrices that go through the launches together; where their units begin, and how many.
struct MuonBatch {
  int64_t first_part, parts, first_block, blocks, first_gram, grams, first_apply, applies;
  int64_t partials_at;       // in the workspace
  int64_t most_m, most_n;    // of its matrices
};
struct MuonHeader {
  int64_t magic, bytes, n_tensors, n_batches, workspace;
  int64_t batches_at, records_at, parts_at, blocks_at, gram_at, apply_at;
};
struct MuonArgs {
  const MuonRecord* records;  // set by the launcher, as n_tensors, err and levels
  int64_t n_tensors;
  unsigned char* workspace;
  uint32_t* err;
  int32_t* levels;            // of a matrix: 0 where its norm is not finite, else 1 + its X's exponent
  double lr;
  float momentum, eps;
  int nesterov;
};
// Both allocate on the host: std::bad_alloc is the caller's to catch.
size_t muon_plan_bytes(const lp_muon_tensor* tensors, int64_t n_tensors);
void write_muon_plan(const lp_muon_tensor* tensors, int64_t n_tensors, void* plan, size_t bytes);
lp_status launch_muon_step(const Device& dev, const void* plan_host, const void* plan, const MuonArgs& a,
                           int steps, cudaStream_t stream);

// Read and clear the check words of these translation units (lp_check.cuh).
cudaError_t take_check_word_layer_norm(uint32_t* out);
cudaError_t take_check_word_layer_norm_backward(uint32_t* out);
cudaError_t take_check_word_preference(uint32_t* out);
cudaError_t take_check_word_muon(uint32_t* out);

}  // namespace lp
