// lp_tune_api.cu: the C-ABI front end of the fine-tuning operators (declared in
// include/lp_tune.h).  As in lp_api.cu, every entry point validates its arguments
// on the host in the order sizes and null pointers, alignment, workspace, device,
// and enqueues nothing before all checks pass.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "lp_args.h"
#include "lp_tune_internal.h"

extern "C" {

lp_status lp_layer_norm(const void* residual, int64_t ld_residual, int residual_dtype,
                        const void* branch, int64_t ld_branch, int act_dtype, const void* weight,
                        const void* bias, int weight_dtype, int64_t T, int64_t d, float eps,
                        void* residual_out, int64_t ld_residual_out, void* normed,
                        int64_t ld_normed, float* mean, float* rstd, void* stream) {
  using namespace lp;
  if (T < 0 || T > kMaxRows || d < 1 || d > kNormMaxDim || !is_dtype(residual_dtype) ||
      !is_dtype(act_dtype) || !is_dtype(weight_dtype) || !(eps >= 0.0f) || !std::isfinite(eps))
    return LP_ERR_INVALID_ARGUMENT;
  if (T == 0) return LP_OK;  // operands without rows may be null
  if (residual == nullptr || normed == nullptr || mismatch(residual_out, branch != nullptr))
    return LP_ERR_INVALID_ARGUMENT;
  if (bad_rows(ld_residual, d) || bad_rows(ld_normed, d) ||
      (branch != nullptr && (bad_rows(ld_branch, d) || bad_rows(ld_residual_out, d))))
    return LP_ERR_INVALID_ARGUMENT;
  const bool rb = residual_dtype == LP_BFLOAT16, ab = act_dtype == LP_BFLOAT16,
             wb = weight_dtype == LP_BFLOAT16;
  const int64_t rs = size_of(rb), as = size_of(ab), ws = size_of(wb);
  const Extent in[4] = {extent(residual, T, ld_residual, d, rs), extent(branch, T, ld_branch, d, as),
                        extent(weight, 1, d, d, ws), extent(bias, 1, d, d, ws)};
  const Extent out[4] = {extent(residual_out, T, ld_residual_out, d, rs),
                         extent(normed, T, ld_normed, d, as), extent(mean, T, 1, 1, 4),
                         extent(rstd, T, 1, 1, 4)};
  const bool in_place = residual_out == residual && ld_residual_out == ld_residual;
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j)
      if (overlap(out[i], in[j]) && !(i == 0 && j == 0 && in_place)) return LP_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return LP_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(residual, rs) || !aligned(residual_out, rs) || !aligned(branch, as) ||
      !aligned(normed, as) || !aligned(weight, ws) || !aligned(bias, ws) || !aligned(mean, 4) ||
      !aligned(rstd, 4))
    return LP_ERR_MISALIGNED;
  Device dev;
  const lp_status st = current_device(&dev);
  if (st != LP_OK) return st;
  LayerNormArgs a{};
  a.residual = {const_cast<void*>(residual), ld_residual};
  a.branch = {const_cast<void*>(branch), ld_branch};
  a.weight = weight;
  a.bias = bias;
  a.residual_bf16 = rb;
  a.act_bf16 = ab;
  a.weight_bf16 = wb;
  a.T = T;
  a.d = d;
  a.eps = eps;
  a.residual_out = {residual_out, ld_residual_out};
  a.normed = {normed, ld_normed};
  a.mean = mean;
  a.rstd = rstd;
  return launch_layer_norm(dev, a, static_cast<cudaStream_t>(stream));
}

size_t lp_layer_norm_backward_workspace_size(int64_t T, int64_t d) {
  if (T < 0 || T > lp::kMaxRows || d < 1 || d > lp::kNormMaxDim) return 0;
  return lp::layer_norm_backward_workspace(T, d);
}

lp_status lp_layer_norm_backward(
    const void* residual_out, int64_t ld_residual_out, int residual_dtype, int act_dtype,
    const void* weight, int weight_dtype, int64_t T, int64_t d, const float* mean,
    const float* rstd, const void* grad_normed, int64_t ld_grad_normed,
    const void* grad_residual_out, int64_t ld_grad_residual_out, void* grad_residual,
    int64_t ld_grad_residual, void* grad_branch, int64_t ld_grad_branch, float* grad_weight,
    float* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace lp;
  if (T < 0 || T > kMaxRows || d < 1 || d > kNormMaxDim || !is_dtype(residual_dtype) ||
      !is_dtype(act_dtype) || !is_dtype(weight_dtype))
    return LP_ERR_INVALID_ARGUMENT;
  const bool sums = grad_weight != nullptr || grad_bias != nullptr;
  if (T == 0 && !sums) return LP_OK;
  if (sums && workspace == nullptr) return LP_ERR_INVALID_ARGUMENT;
  if (T > 0) {  // operands without rows may be null
    if (residual_out == nullptr || mean == nullptr || rstd == nullptr || grad_normed == nullptr ||
        grad_residual == nullptr)
      return LP_ERR_INVALID_ARGUMENT;
    if (bad_rows(ld_residual_out, d) || bad_rows(ld_grad_normed, d) ||
        bad_rows(ld_grad_residual, d) ||
        (grad_residual_out != nullptr && bad_rows(ld_grad_residual_out, d)) ||
        (grad_branch != nullptr && bad_rows(ld_grad_branch, d)))
      return LP_ERR_INVALID_ARGUMENT;
  }
  const bool rb = residual_dtype == LP_BFLOAT16, ab = act_dtype == LP_BFLOAT16,
             wb = weight_dtype == LP_BFLOAT16;
  const int64_t rs = size_of(rb), as = size_of(ab), ws = size_of(wb);
  const Extent in[6] = {extent(residual_out, T, ld_residual_out, d, rs),
                        extent(weight, 1, d, d, ws),
                        extent(mean, T, 1, 1, 4),
                        extent(rstd, T, 1, 1, 4),
                        extent(grad_normed, T, ld_grad_normed, d, as),
                        extent(grad_residual_out, T, ld_grad_residual_out, d, rs)};
  const Extent out[5] = {extent(grad_residual, T, ld_grad_residual, d, rs),
                         extent(grad_branch, T, ld_grad_branch, d, as),
                         extent(grad_weight, 1, d, d, 4), extent(grad_bias, 1, d, d, 4),
                         extent(sums ? workspace : nullptr, 1, 0,
                                static_cast<int64_t>(layer_norm_backward_workspace(T, d)), 1)};
  const bool in_place =
      grad_residual == grad_residual_out && ld_grad_residual == ld_grad_residual_out;
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 6; ++j)
      if (overlap(out[i], in[j]) && !(i == 0 && j == 5 && in_place)) return LP_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return LP_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(residual_out, rs) || !aligned(grad_residual_out, rs) ||
      !aligned(grad_residual, rs) || !aligned(grad_normed, as) || !aligned(grad_branch, as) ||
      !aligned(weight, ws) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(grad_weight, 4) ||
      !aligned(grad_bias, 4) || (sums && !aligned(workspace, 256)))
    return LP_ERR_MISALIGNED;
  if (sums && workspace_bytes < layer_norm_backward_workspace(T, d))
    return LP_ERR_WORKSPACE_TOO_SMALL;
  Device dev;
  const lp_status st = current_device(&dev);
  if (st != LP_OK) return st;
  LayerNormGradArgs a{};
  a.residual_out = {const_cast<void*>(residual_out), ld_residual_out};
  a.weight = weight;
  a.residual_bf16 = rb;
  a.act_bf16 = ab;
  a.weight_bf16 = wb;
  a.T = T;
  a.d = d;
  a.mean = mean;
  a.rstd = rstd;
  a.grad_normed = {const_cast<void*>(grad_normed), ld_grad_normed};
  a.grad_residual_out = {const_cast<void*>(grad_residual_out), ld_grad_residual_out};
  a.grad_residual = {grad_residual, ld_grad_residual};
  a.grad_branch = {grad_branch, ld_grad_branch};
  a.grad_weight = grad_weight;
  a.grad_bias = grad_bias;
  a.partials = sums ? static_cast<float*>(workspace) : nullptr;
  return launch_layer_norm_backward(dev, a, static_cast<cudaStream_t>(stream));
}

size_t lp_preference_loss_workspace_size(int64_t T, int64_t n_sequences) {
  if (T < 0 || T > lp::kMaxRows || n_sequences < 0 || n_sequences > lp::kMaxRows) return 0;
  return lp::preference_loss_workspace(T, n_sequences);
}

lp_status lp_preference_loss(const float* logp, const float* ref_logp, const uint8_t* mask,
                             const int64_t* cu_seqlens, int64_t T, int64_t n_sequences, int kind,
                             int average, int halves, double beta, double margin,
                             double label_smoothing, double nll_coef, float* stats, float* rewards,
                             float* grad_logp, void* workspace, size_t workspace_bytes,
                             void* stream) {
  using namespace lp;
  if (T < 0 || T > kMaxRows || n_sequences < 0 || n_sequences > kMaxRows || n_sequences % 2 != 0)
    return LP_ERR_INVALID_ARGUMENT;
  if (kind != LP_PREFERENCE_SIGMOID && kind != LP_PREFERENCE_HINGE && kind != LP_PREFERENCE_SQUARE)
    return LP_ERR_INVALID_ARGUMENT;
  // what the kernels take as float32 has to be one; beta and its reciprocal normal ones
  const auto fits = [](double v) { return std::isfinite(static_cast<float>(v)); };
  if (!(static_cast<float>(beta) >= FLT_MIN) || !(static_cast<float>(1.0 / beta) >= FLT_MIN) ||
      !fits(beta) || !fits(1.0 / beta) || !fits(margin) || !fits(nll_coef) ||
      !(label_smoothing >= 0.0 && label_smoothing <= 1.0) ||
      (label_smoothing != 0.0 && kind != LP_PREFERENCE_SIGMOID))
    return LP_ERR_INVALID_ARGUMENT;
  if (cu_seqlens == nullptr || stats == nullptr || workspace == nullptr ||
      (n_sequences > 0 && rewards == nullptr) ||
      (T > 0 && (logp == nullptr || grad_logp == nullptr)))
    return LP_ERR_INVALID_ARGUMENT;
  const Extent in[4] = {extent(logp, T, 1, 1, 4), extent(ref_logp, T, 1, 1, 4),
                        extent(mask, T, 1, 1, 1), extent(cu_seqlens, n_sequences + 1, 1, 1, 8)};
  const Extent out[4] = {
      extent(stats, 6, 1, 1, 4), extent(rewards, n_sequences, 1, 1, 4), extent(grad_logp, T, 1, 1, 4),
      extent(workspace, 1, 0, static_cast<int64_t>(preference_loss_workspace(T, n_sequences)), 1)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j)
      if (overlap(out[i], in[j])) return LP_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return LP_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(logp, 4) || !aligned(ref_logp, 4) || !aligned(cu_seqlens, 8) || !aligned(stats, 4) ||
      !aligned(rewards, 4) || !aligned(grad_logp, 4) || !aligned(workspace, 256))
    return LP_ERR_MISALIGNED;
  if (workspace_bytes < preference_loss_workspace(T, n_sequences)) return LP_ERR_WORKSPACE_TOO_SMALL;
  Device dev;
  const lp_status st = current_device(&dev);
  if (st != LP_OK) return st;
  PreferenceArgs a{};
  a.logp = logp;
  a.ref_logp = ref_logp;
  a.mask = mask;
  a.cu_seqlens = cu_seqlens;
  a.T = T;
  a.n_sequences = n_sequences;
  a.kind = kind;
  a.average = average != 0;
  a.halves = halves != 0;
  a.beta = pair32(beta);
  a.inverse_beta = pair32(1.0 / beta);
  a.margin = pair32(margin);
  a.smoothing = static_cast<float>(label_smoothing);
  a.nll_coef = static_cast<float>(nll_coef);
  a.stats = stats;
  a.rewards = rewards;
  a.grad_logp = grad_logp;
  a.workspace = workspace;
  return launch_preference_loss(a, static_cast<cudaStream_t>(stream));
}

namespace {
bool bad_matrices(const lp_muon_tensor* tensors, int64_t n_tensors) {
  using namespace lp;
  if (n_tensors < 0 || n_tensors > kMaxRows || (tensors == nullptr && n_tensors > 0)) return true;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const lp_muon_tensor& t = tensors[i];
    if (t.rows < 0 || t.rows > kMuonMaxDim || t.cols < 0 || t.cols > kMuonMaxDim) return true;
  }
  return false;
}
const lp::MuonHeader* muon_header(const void* plan_host) {
  if (plan_host == nullptr || !lp::aligned(plan_host, 8)) return nullptr;
  const auto* h = static_cast<const lp::MuonHeader*>(plan_host);
  return h->magic == lp::kMuonMagic ? h : nullptr;
}
}  // namespace

size_t lp_muon_plan_size(const lp_muon_tensor* tensors, int64_t n_tensors) {
  if (bad_matrices(tensors, n_tensors)) return 0;
  try {
    return lp::muon_plan_bytes(tensors, n_tensors);
  } catch (...) {  // out of host memory
    return 0;
  }
}

lp_status lp_muon_plan(const lp_muon_tensor* tensors, int64_t n_tensors, void* plan_host,
                       size_t plan_bytes) {
  using namespace lp;
  if (bad_matrices(tensors, n_tensors) || plan_host == nullptr) return LP_ERR_INVALID_ARGUMENT;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const lp_muon_tensor& t = tensors[i];
    if (!is_dtype(t.grad_dtype)) return LP_ERR_INVALID_ARGUMENT;
    for (float f : {t.lr_scale, t.weight_decay, t.update_scale})
      if (!(f >= 0.0f) || !std::isfinite(f)) return LP_ERR_INVALID_ARGUMENT;
    const int64_t n = t.rows * t.cols;
    if (n > 0 && (t.param == nullptr || t.grad == nullptr || t.momentum == nullptr))
      return LP_ERR_INVALID_ARGUMENT;
    const Extent e[4] = {extent(t.param, n, 1, 1, 4), extent(t.copy, n, 1, 1, 2),
                         extent(t.momentum, n, 1, 1, 4),
                         extent(t.grad, n, 1, 1, size_of(t.grad_dtype == LP_BFLOAT16))};
    for (int j = 0; j < 4; ++j)
      for (int k = 0; k < j; ++k)
        if (overlap(e[j], e[k])) return LP_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(plan_host, 8)) return LP_ERR_MISALIGNED;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const lp_muon_tensor& t = tensors[i];
    if (!aligned(t.param, 4) || !aligned(t.copy, 2) || !aligned(t.momentum, 4) ||
        !aligned(t.grad, size_of(t.grad_dtype == LP_BFLOAT16)))
      return LP_ERR_MISALIGNED;
  }
  try {
    if (plan_bytes < muon_plan_bytes(tensors, n_tensors)) return LP_ERR_WORKSPACE_TOO_SMALL;
    write_muon_plan(tensors, n_tensors, plan_host, plan_bytes);
  } catch (...) {  // out of host memory
    return LP_ERR_WORKSPACE_TOO_SMALL;
  }
  return LP_OK;
}

size_t lp_muon_workspace_size(const void* plan_host) {
  const lp::MuonHeader* h = muon_header(plan_host);
  return h == nullptr ? 0 : static_cast<size_t>(h->workspace);
}

lp_status lp_muon_step(const void* plan_host, const void* plan, double lr, double momentum,
                       int nesterov, int steps, double eps, void* workspace,
                       size_t workspace_bytes, void* stream) {
  using namespace lp;
  if (!(lr >= 0.0) || !std::isfinite(lr) || !(momentum >= 0.0 && momentum < 1.0) ||
      !(eps >= 1e-16) || !std::isfinite(static_cast<float>(eps)) || steps < 1 || steps > 32)
    return LP_ERR_INVALID_ARGUMENT;
  const MuonHeader* h = muon_header(plan_host);
  if (h == nullptr) return LP_ERR_INVALID_ARGUMENT;
  if (h->n_batches == 0) return LP_OK;
  if (plan == nullptr || workspace == nullptr) return LP_ERR_INVALID_ARGUMENT;
  if (!aligned(plan, 256) || !aligned(workspace, 256)) return LP_ERR_MISALIGNED;
  if (workspace_bytes < static_cast<size_t>(h->workspace)) return LP_ERR_WORKSPACE_TOO_SMALL;
  Device dev;
  const lp_status st = current_device(&dev);
  if (st != LP_OK) return st;
  MuonArgs a{};
  a.workspace = static_cast<unsigned char*>(workspace);
  a.lr = lr;
  a.momentum = static_cast<float>(momentum);
  a.eps = static_cast<float>(eps);
  a.nesterov = nesterov != 0;
  return launch_muon_step(dev, plan_host, plan, a, steps, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
