// lp_train_api.cu: the C-ABI front end of the training-step operators (declared
// in include/lp_train.h).  As in lp_api.cu, every entry point validates its
// arguments on the host in the order sizes and null pointers, alignment,
// workspace, device, and enqueues nothing before all checks pass.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "lp_args.h"
#include "lp_train_internal.h"

extern "C" {

lp_status lp_residual_norm(const void* residual, int64_t ld_residual, int residual_dtype,
                           const void* branch, int64_t ld_branch, const void* gate,
                           int64_t ld_gate, int act_dtype, const void* branch_weight,
                           const void* weight, int weight_dtype, int64_t T, int64_t d,
                           float residual_scale, float branch_scale, float eps,
                           void* residual_out, int64_t ld_residual_out, void* normed,
                           int64_t ld_normed, float* branch_rstd, float* rstd, void* stream) {
  using namespace lp;
  if (T < 0 || T > kMaxRows || d < 1 || d > kNormMaxDim || !is_dtype(residual_dtype) ||
      !is_dtype(act_dtype) || !is_dtype(weight_dtype))
    return LP_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(residual_scale) || !std::isfinite(branch_scale) || !(eps >= 0.0f) ||
      !std::isfinite(eps))
    return LP_ERR_INVALID_ARGUMENT;
  if (T == 0) return LP_OK;  // operands without rows may be null
  if (branch == nullptr && (weight == nullptr || residual_scale != 1.0f))
    return LP_ERR_INVALID_ARGUMENT;
  if (branch == nullptr && (gate != nullptr || branch_weight != nullptr))
    return LP_ERR_INVALID_ARGUMENT;
  if ((branch_weight == nullptr && branch_rstd != nullptr) ||
      (weight == nullptr && rstd != nullptr))
    return LP_ERR_INVALID_ARGUMENT;
  if (bad_rows(ld_residual, d) || (branch != nullptr && bad_rows(ld_branch, d)) ||
      (gate != nullptr && ld_gate != 0 && bad_rows(ld_gate, d)))
    return LP_ERR_INVALID_ARGUMENT;
  if (residual == nullptr || mismatch(residual_out, branch != nullptr) ||
      mismatch(normed, weight != nullptr))
    return LP_ERR_INVALID_ARGUMENT;
  if ((residual_out != nullptr && bad_rows(ld_residual_out, d)) ||
      (normed != nullptr && bad_rows(ld_normed, d)))
    return LP_ERR_INVALID_ARGUMENT;
  const bool rb = residual_dtype == LP_BFLOAT16, ab = act_dtype == LP_BFLOAT16,
             wb = weight_dtype == LP_BFLOAT16;
  const int64_t rs = size_of(rb), as = size_of(ab), ws = size_of(wb);
  const Extent in[5] = {extent(residual, T, ld_residual, d, rs),
                        extent(branch, T, ld_branch, d, as),
                        extent(gate, ld_gate == 0 ? 1 : T, ld_gate, d, as),
                        extent(branch_weight, 1, d, d, ws), extent(weight, 1, d, d, ws)};
  const Extent out[4] = {extent(residual_out, T, ld_residual_out, d, rs),
                         extent(normed, T, ld_normed, d, as), extent(branch_rstd, T, 1, 1, 4),
                         extent(rstd, T, 1, 1, 4)};
  const bool in_place = residual_out == residual && ld_residual_out == ld_residual;
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 5; ++j)
      if (overlap(out[i], in[j]) && !(i == 0 && j == 0 && in_place)) return LP_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return LP_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(residual, rs) || !aligned(residual_out, rs) || !aligned(branch, as) ||
      !aligned(gate, as) || !aligned(normed, as) || !aligned(branch_weight, ws) ||
      !aligned(weight, ws) || !aligned(branch_rstd, 4) || !aligned(rstd, 4))
    return LP_ERR_MISALIGNED;
  Device dev;
  const lp_status st = current_device(&dev);
  if (st != LP_OK) return st;
  NormArgs a{};
  a.residual = {const_cast<void*>(residual), ld_residual};
  a.branch = {const_cast<void*>(branch), ld_branch};
  a.gate = {const_cast<void*>(gate), ld_gate};
  a.branch_weight = branch_weight;
  a.weight = weight;
  a.residual_bf16 = rb;
  a.act_bf16 = ab;
  a.weight_bf16 = wb;
  a.T = T;
  a.d = d;
  a.residual_scale = residual_scale;
  a.branch_scale = branch_scale;
  a.eps = eps;
  a.residual_out = {residual_out, ld_residual_out};
  a.normed = {normed, ld_normed};
  a.branch_rstd = branch_rstd;
  a.rstd = rstd;
  return launch_residual_norm(dev, a, static_cast<cudaStream_t>(stream));
}

size_t lp_residual_norm_backward_workspace_size(int64_t T, int64_t d) {
  if (T < 0 || T > lp::kMaxRows || d < 1 || d > lp::kNormMaxDim) return 0;
  return lp::residual_norm_backward_workspace(T, d);
}

lp_status lp_residual_norm_backward(
    const void* residual_out, int64_t ld_residual_out, int residual_dtype, const void* branch,
    int64_t ld_branch, const void* gate, int64_t ld_gate, int act_dtype, const void* branch_weight,
    const void* weight, int weight_dtype, int64_t T, int64_t d, float residual_scale,
    float branch_scale, const float* branch_rstd, const float* rstd, const void* grad_normed,
    int64_t ld_grad_normed, const void* grad_residual_out, int64_t ld_grad_residual_out,
    void* grad_residual, int64_t ld_grad_residual, void* grad_branch, int64_t ld_grad_branch,
    void* grad_gate, int64_t ld_grad_gate, float* grad_branch_weight, float* grad_weight,
    void* workspace, size_t workspace_bytes, void* stream) {
  using namespace lp;
  if (T < 0 || T > kMaxRows || d < 1 || d > kNormMaxDim || !is_dtype(residual_dtype) ||
      !is_dtype(act_dtype) || !is_dtype(weight_dtype))
    return LP_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(residual_scale) || !std::isfinite(branch_scale))
    return LP_ERR_INVALID_ARGUMENT;
  const bool gate_row = gate != nullptr && ld_gate == 0;
  const bool sums = grad_weight != nullptr || grad_branch_weight != nullptr ||
                    (gate_row && grad_gate != nullptr);
  if (T == 0 && !sums) return LP_OK;
  if (sums && workspace == nullptr) return LP_ERR_INVALID_ARGUMENT;
  const bool has_branch = branch != nullptr, has_weight = weight != nullptr;
  if (T > 0) {  // operands without rows may be null
    if (!has_branch && (!has_weight || residual_scale != 1.0f)) return LP_ERR_INVALID_ARGUMENT;
    if (!has_branch && (gate != nullptr || branch_weight != nullptr))
      return LP_ERR_INVALID_ARGUMENT;
    if ((grad_gate != nullptr && gate == nullptr) ||
        (grad_branch_weight != nullptr && branch_weight == nullptr) ||
        (grad_weight != nullptr && !has_weight))
      return LP_ERR_INVALID_ARGUMENT;
    if ((has_weight && bad_rows(ld_residual_out, d)) || (has_branch && bad_rows(ld_branch, d)) ||
        (gate != nullptr && ld_gate != 0 && bad_rows(ld_gate, d)) ||
        (has_weight && bad_rows(ld_grad_normed, d)) ||
        (grad_residual_out != nullptr && bad_rows(ld_grad_residual_out, d)) ||
        bad_rows(ld_grad_residual, d) || (has_branch && bad_rows(ld_grad_branch, d)) ||
        (grad_gate != nullptr && ld_gate != 0 && bad_rows(ld_grad_gate, d)))
      return LP_ERR_INVALID_ARGUMENT;
    if (mismatch(residual_out, has_weight) || mismatch(grad_normed, has_weight) ||
        (!has_weight && grad_residual_out == nullptr) || grad_residual == nullptr ||
        mismatch(grad_branch, has_branch) || (has_weight && rstd == nullptr) ||
        (branch_weight != nullptr && branch_rstd == nullptr))
      return LP_ERR_INVALID_ARGUMENT;
  }
  const bool rb = residual_dtype == LP_BFLOAT16, ab = act_dtype == LP_BFLOAT16,
             wb = weight_dtype == LP_BFLOAT16;
  const int64_t rs = size_of(rb), as = size_of(ab), ws = size_of(wb);
  const int64_t gate_rows = gate_row ? 1 : T;
  const Extent in[9] = {extent(residual_out, T, ld_residual_out, d, rs),
                        extent(branch, T, ld_branch, d, as),
                        extent(gate, gate_rows, ld_gate, d, as),
                        extent(branch_weight, 1, d, d, ws),
                        extent(weight, 1, d, d, ws),
                        extent(branch_rstd, T, 1, 1, 4),
                        extent(rstd, T, 1, 1, 4),
                        extent(grad_normed, T, ld_grad_normed, d, as),
                        extent(grad_residual_out, T, ld_grad_residual_out, d, rs)};
  const Extent out[6] = {extent(grad_residual, T, ld_grad_residual, d, rs),
                         extent(grad_branch, T, ld_grad_branch, d, as),
                         gate_row ? extent(grad_gate, 1, d, d, 4)
                                  : extent(grad_gate, T, ld_grad_gate, d, as),
                         extent(grad_branch_weight, 1, d, d, 4), extent(grad_weight, 1, d, d, 4),
                         extent(sums ? workspace : nullptr, 1, 0,
                                static_cast<int64_t>(residual_norm_backward_workspace(T, d)), 1)};
  const bool in_place =
      grad_residual == grad_residual_out && ld_grad_residual == ld_grad_residual_out;
  for (int i = 0; i < 6; ++i) {
    for (int j = 0; j < 9; ++j)
      if (overlap(out[i], in[j]) && !(i == 0 && j == 8 && in_place)) return LP_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return LP_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(residual_out, rs) || !aligned(grad_residual_out, rs) ||
      !aligned(grad_residual, rs) || !aligned(branch, as) || !aligned(gate, as) ||
      !aligned(grad_normed, as) || !aligned(grad_branch, as) ||
      !aligned(grad_gate, gate_row ? 4 : as) || !aligned(branch_weight, ws) ||
      !aligned(weight, ws) || !aligned(branch_rstd, 4) || !aligned(rstd, 4) ||
      !aligned(grad_branch_weight, 4) || !aligned(grad_weight, 4) ||
      (sums && !aligned(workspace, 256)))
    return LP_ERR_MISALIGNED;
  if (sums && workspace_bytes < residual_norm_backward_workspace(T, d))
    return LP_ERR_WORKSPACE_TOO_SMALL;
  Device dev;
  const lp_status st = current_device(&dev);
  if (st != LP_OK) return st;
  NormGradArgs a{};
  a.residual_out = {const_cast<void*>(residual_out), ld_residual_out};
  a.branch = {const_cast<void*>(branch), ld_branch};
  a.gate = {const_cast<void*>(gate), ld_gate};
  a.branch_weight = branch_weight;
  a.weight = weight;
  a.residual_bf16 = rb;
  a.act_bf16 = ab;
  a.weight_bf16 = wb;
  a.T = T;
  a.d = d;
  a.residual_scale = residual_scale;
  a.branch_scale = branch_scale;
  a.branch_rstd = branch_rstd;
  a.rstd = rstd;
  a.grad_normed = {const_cast<void*>(grad_normed), ld_grad_normed};
  a.grad_residual_out = {const_cast<void*>(grad_residual_out), ld_grad_residual_out};
  a.grad_residual = {grad_residual, ld_grad_residual};
  a.grad_branch = {grad_branch, ld_grad_branch};
  a.grad_gate = {grad_gate, ld_grad_gate};
  a.grad_branch_weight = grad_branch_weight;
  a.grad_weight = grad_weight;
  a.partials = sums ? static_cast<float*>(workspace) : nullptr;
  return launch_residual_norm_backward(dev, a, static_cast<cudaStream_t>(stream));
}

size_t lp_policy_loss_workspace_size(int64_t T, int64_t n_sequences) {
  if (T < 0 || T > lp::kMaxRows || n_sequences < 0 || n_sequences > lp::kMaxRows) return 0;
  return lp::policy_loss_workspace(T, n_sequences);
}

lp_status lp_policy_loss(const float* logp, const float* old_logp, const float* ref_logp,
                         const float* entropy, const float* advantages,
                         int advantages_per_sequence, const uint8_t* mask,
                         const int64_t* cu_seqlens, int64_t T, int64_t n_sequences, int reduction,
                         double clip_low, double clip_high, double kl_coef,
                         double entropy_coef, float* stats, float* grad_logp, float* grad_entropy, void* workspace,
                         size_t workspace_bytes, void* stream) {
  using namespace lp;
  if (T < 0 || T > kMaxRows || n_sequences < 0 || n_sequences > kMaxRows)
    return LP_ERR_INVALID_ARGUMENT;
  if (reduction != LP_REDUCE_TOKEN && reduction != LP_REDUCE_SEQUENCE)
    return LP_ERR_INVALID_ARGUMENT;
  if (!(clip_low >= 0.0 && clip_low < 1.0) || !(clip_high >= 0.0) || !std::isfinite(clip_high) ||
      !std::isfinite(kl_coef) || !std::isfinite(entropy_coef))
    return LP_ERR_INVALID_ARGUMENT;
  const bool sequences = reduction == LP_REDUCE_SEQUENCE || advantages_per_sequence != 0;
  if (stats == nullptr || workspace == nullptr || (sequences && cu_seqlens == nullptr))
    return LP_ERR_INVALID_ARGUMENT;
  if (T > 0 && (logp == nullptr || old_logp == nullptr || grad_logp == nullptr ||
                mismatch(grad_entropy, entropy != nullptr)))
    return LP_ERR_INVALID_ARGUMENT;
  if (advantages == nullptr && (advantages_per_sequence != 0 ? n_sequences > 0 : T > 0))
    return LP_ERR_INVALID_ARGUMENT;
  const Extent in[7] = {extent(logp, T, 1, 1, 4),
                        extent(old_logp, T, 1, 1, 4),
                        extent(ref_logp, T, 1, 1, 4),
                        extent(entropy, T, 1, 1, 4),
                        extent(advantages, advantages_per_sequence != 0 ? n_sequences : T, 1, 1, 4),
                        extent(mask, T, 1, 1, 1),
                        extent(sequences ? cu_seqlens : nullptr, n_sequences + 1, 1, 1, 8)};
  const Extent out[4] = {
      extent(stats, 5, 1, 1, 4), extent(grad_logp, T, 1, 1, 4), extent(grad_entropy, T, 1, 1, 4),
      extent(workspace, 1, 0, static_cast<int64_t>(policy_loss_workspace(T, n_sequences)), 1)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 7; ++j)
      if (overlap(out[i], in[j])) return LP_ERR_INVALID_ARGUMENT;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return LP_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(logp, 4) || !aligned(old_logp, 4) || !aligned(ref_logp, 4) || !aligned(entropy, 4) ||
      !aligned(advantages, 4) || (sequences && !aligned(cu_seqlens, 8)) || !aligned(stats, 4) ||
      !aligned(grad_logp, 4) || !aligned(grad_entropy, 4) || !aligned(workspace, 256))
    return LP_ERR_MISALIGNED;
  if (workspace_bytes < policy_loss_workspace(T, n_sequences)) return LP_ERR_WORKSPACE_TOO_SMALL;
  Device dev;
  const lp_status st = current_device(&dev);
  if (st != LP_OK) return st;
  PolicyArgs a{};
  a.logp = logp;
  a.old_logp = old_logp;
  a.ref_logp = ref_logp;
  a.entropy = entropy;
  a.advantages = advantages;
  a.per_sequence = advantages_per_sequence != 0;
  a.by_sequence = reduction == LP_REDUCE_SEQUENCE;
  a.mask = mask;
  a.cu_seqlens = sequences ? cu_seqlens : nullptr;
  a.T = T;
  a.n_sequences = sequences ? n_sequences : 0;
  // the limits in float64, rounded to float32 once
  a.low = static_cast<float>(std::log1p(-clip_low));
  a.high = static_cast<float>(std::log1p(clip_high));
  a.ratio_low = static_cast<float>(1.0 - clip_low);
  a.ratio_high = static_cast<float>(1.0 + clip_high);
  a.kl_coef = ref_logp != nullptr ? static_cast<float>(kl_coef) : 0.0f;
  a.entropy_coef = entropy != nullptr ? static_cast<float>(entropy_coef) : 0.0f;
  a.stats = stats;
  a.grad_logp = grad_logp;
  a.grad_entropy = grad_entropy;
  a.workspace = workspace;
  return launch_policy_loss(a, static_cast<cudaStream_t>(stream));
}

int64_t lp_adamw_state_elements(const lp_adamw_tensor* tensors, int64_t n_tensors) {
  if (n_tensors < 0 || n_tensors > lp::kMaxRows || (tensors == nullptr && n_tensors > 0)) return -1;
  int64_t rows = 0;
  for (int64_t i = 0; i < n_tensors; ++i) {
    if (tensors[i].n < 0 || tensors[i].n > lp::kMaxStride) return -1;
    rows += (tensors[i].n + LP_ADAMW_ALIGN - 1) / LP_ADAMW_ALIGN;
    if (rows > lp::kMaxRows) return -1;
  }
  return rows * LP_ADAMW_ALIGN;
}

size_t lp_adamw_plan_size(const lp_adamw_tensor* tensors, int64_t n_tensors) {
  const int64_t elements = lp_adamw_state_elements(tensors, n_tensors);
  if (elements < 0) return 0;
  return lp::adamw_table_offset(n_tensors) +
         static_cast<size_t>(elements / LP_ADAMW_ALIGN) * sizeof(int32_t);
}

lp_status lp_adamw_plan(const lp_adamw_tensor* tensors, int64_t n_tensors, void* plan_host,
                        size_t plan_bytes) {
  using namespace lp;
  if (lp_adamw_state_elements(tensors, n_tensors) < 0 || (plan_host == nullptr && n_tensors > 0))
    return LP_ERR_INVALID_ARGUMENT;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const lp_adamw_tensor& t = tensors[i];
    if (!is_dtype(t.grad_dtype) || t.reserved != 0) return LP_ERR_INVALID_ARGUMENT;
    if (!(t.lr_scale >= 0.0f) || !std::isfinite(t.lr_scale) || !(t.weight_decay >= 0.0f) ||
        !std::isfinite(t.weight_decay))
      return LP_ERR_INVALID_ARGUMENT;
    if (t.n > 0 && (t.param == nullptr || t.grad == nullptr)) return LP_ERR_INVALID_ARGUMENT;
    const bool gb = t.grad_dtype == LP_BFLOAT16;
    const Extent p = extent(t.param, t.n, 1, 1, 4), c = extent(t.copy, t.n, 1, 1, 2),
                 g = extent(t.grad, t.n, 1, 1, size_of(gb));
    if (overlap(p, c) || overlap(p, g) || overlap(c, g)) return LP_ERR_INVALID_ARGUMENT;
  }
  for (int64_t i = 0; i < n_tensors; ++i) {
    const lp_adamw_tensor& t = tensors[i];
    if (!aligned(t.param, 4) || !aligned(t.copy, 2) ||
        !aligned(t.grad, size_of(t.grad_dtype == LP_BFLOAT16)))
      return LP_ERR_MISALIGNED;
  }
  if (plan_bytes < lp_adamw_plan_size(tensors, n_tensors)) return LP_ERR_WORKSPACE_TOO_SMALL;
  char* out = static_cast<char*>(plan_host);
  char* table = out + adamw_table_offset(n_tensors);
  int64_t row = 0;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const lp_adamw_tensor& t = tensors[i];
    AdamwRecord r{};
    r.param = t.param;
    r.copy = static_cast<__nv_bfloat16*>(t.copy);
    r.grad = t.grad;
    r.n = t.n;
    r.first_row = row;
    r.lr_scale = t.lr_scale;
    r.weight_decay = t.weight_decay;
    r.grad_bf16 = t.grad_dtype == LP_BFLOAT16;
    r.wide = aligned(t.param, 16) && aligned(t.copy, 8) && aligned(t.grad, r.grad_bf16 ? 8 : 16);
    std::memcpy(out + i * sizeof(r), &r, sizeof(r));
    const int32_t index = static_cast<int32_t>(i);
    for (int64_t k = (t.n + LP_ADAMW_ALIGN - 1) / LP_ADAMW_ALIGN; k > 0; --k, ++row)
      std::memcpy(table + row * sizeof(index), &index, sizeof(index));
  }
  return LP_OK;
}

namespace {
bool bad_plan(const void* plan, int64_t n_tensors, int64_t state_elements) {
  return n_tensors < 0 || n_tensors > lp::kMaxRows || state_elements < 0 ||
         state_elements % LP_ADAMW_ALIGN != 0 || state_elements / LP_ADAMW_ALIGN > lp::kMaxRows ||
         (n_tensors == 0 && state_elements > 0) || (plan == nullptr && state_elements > 0);
}
const lp::AdamwRecord* plan_records(const void* plan) {
  return static_cast<const lp::AdamwRecord*>(plan);
}
const int32_t* plan_table(const void* plan, int64_t n_tensors) {
  return reinterpret_cast<const int32_t*>(static_cast<const char*>(plan) +
                                          lp::adamw_table_offset(n_tensors));
}
}  // namespace

size_t lp_adamw_grad_norm_workspace_size(int64_t state_elements) {
  if (state_elements < 0 || state_elements % LP_ADAMW_ALIGN != 0 ||
      state_elements / LP_ADAMW_ALIGN > lp::kMaxRows)
    return 0;
  return lp::adamw_grad_norm_workspace(state_elements / LP_ADAMW_ALIGN);
}

lp_status lp_adamw_grad_norm(const void* plan, int64_t n_tensors, int64_t state_elements,
                             float max_norm, float* norm_out, void* workspace,
                             size_t workspace_bytes, void* stream) {
  using namespace lp;
  if (bad_plan(plan, n_tensors, state_elements) || !(max_norm > 0.0f) || norm_out == nullptr ||
      workspace == nullptr)
    return LP_ERR_INVALID_ARGUMENT;
  if (!aligned(plan, 256) || !aligned(norm_out, 4) || !aligned(workspace, 256))
    return LP_ERR_MISALIGNED;
  const int64_t rows = state_elements / LP_ADAMW_ALIGN;
  if (workspace_bytes < adamw_grad_norm_workspace(rows)) return LP_ERR_WORKSPACE_TOO_SMALL;
  Device dev;
  const lp_status st = current_device(&dev);
  if (st != LP_OK) return st;
  return launch_adamw_grad_norm(plan_records(plan), plan_table(plan, n_tensors), n_tensors, rows,
                                max_norm, norm_out, workspace, static_cast<cudaStream_t>(stream));
}

lp_status lp_adamw_step(const void* plan, int64_t n_tensors, int64_t state_elements,
                        int state_bits, void* exp_avg, void* exp_avg_sq, float* exp_avg_scale,
                        float* exp_avg_sq_scale, double lr, double beta1, double beta2, double eps,
                        int64_t step, uint64_t seed, const float* grad_scale, void* stream) {
  using namespace lp;
  if (bad_plan(plan, n_tensors, state_elements) || (state_bits != 32 && state_bits != 8))
    return LP_ERR_INVALID_ARGUMENT;
  if (!(lr >= 0.0) || !std::isfinite(lr) || !(beta1 >= 0.0 && beta1 < 1.0) ||
      !(beta2 >= 0.0 && beta2 < 1.0) || !std::isfinite(eps) || step < 1)
    return LP_ERR_INVALID_ARGUMENT;
  // where both moments are zero the step divides by eps, in float32 arithmetic that reads a
  // subnormal as zero
  if (!(static_cast<float>(eps) >= FLT_MIN)) return LP_ERR_INVALID_ARGUMENT;
  const bool small = state_bits == 8;
  if (state_elements > 0 && (exp_avg == nullptr || exp_avg_sq == nullptr ||
                             mismatch(exp_avg_scale, small) || mismatch(exp_avg_sq_scale, small)))
    return LP_ERR_INVALID_ARGUMENT;
  const int64_t size = small ? 1 : 4, blocks = state_elements / LP_ADAMW_BLOCK;
  const Extent e[4] = {extent(exp_avg, state_elements, 1, 1, size),
                       extent(exp_avg_sq, state_elements, 1, 1, size),
                       extent(exp_avg_scale, blocks, 1, 1, 4),
                       extent(exp_avg_sq_scale, blocks, 1, 1, 4)};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(e[i], e[j])) return LP_ERR_INVALID_ARGUMENT;
  if (!aligned(plan, 256) || !aligned(exp_avg, 16) || !aligned(exp_avg_sq, 16) ||
      !aligned(exp_avg_scale, 4) || !aligned(exp_avg_sq_scale, 4) || !aligned(grad_scale, 4))
    return LP_ERR_MISALIGNED;
  if (state_elements == 0) return LP_OK;
  Device dev;
  const lp_status st = current_device(&dev);
  if (st != LP_OK) return st;
  AdamwArgs a{};
  a.records = plan_records(plan);
  a.table = plan_table(plan, n_tensors);
  a.n_tensors = n_tensors;
  a.rows = state_elements / LP_ADAMW_ALIGN;
  a.exp_avg = exp_avg;
  a.exp_avg_sq = exp_avg_sq;
  a.exp_avg_scale = exp_avg_scale;
  a.exp_avg_sq_scale = exp_avg_sq_scale;
  // the factors of the step in float64, each rounded to float32 once
  const double t = static_cast<double>(step);
  a.lr = static_cast<float>(lr);
  a.step_size = static_cast<float>(lr / (1.0 - std::pow(beta1, t)));
  a.beta1 = static_cast<float>(beta1);
  a.beta2 = static_cast<float>(beta2);
  a.rest1 = static_cast<float>(1.0 - beta1);
  a.rest2 = static_cast<float>(1.0 - beta2);
  a.root_scale = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, t)));
  a.eps = static_cast<float>(eps);
  a.step = static_cast<uint64_t>(step);
  a.seed = seed;
  a.grad_scale = grad_scale;
  return launch_adamw_step(a, static_cast<cudaStream_t>(stream));
}

lp_status lp_adamw_state_values(const void* exp_avg, const void* exp_avg_sq,
                                const float* exp_avg_scale, const float* exp_avg_sq_scale,
                                int64_t state_elements, float* exp_avg_out, float* exp_avg_sq_out,
                                void* stream) {
  using namespace lp;
  if (state_elements < 0 || state_elements % LP_ADAMW_ALIGN != 0 ||
      state_elements / LP_ADAMW_ALIGN > kMaxRows)
    return LP_ERR_INVALID_ARGUMENT;
  if (state_elements == 0) return LP_OK;
  if (exp_avg == nullptr || exp_avg_sq == nullptr || exp_avg_scale == nullptr ||
      exp_avg_sq_scale == nullptr || exp_avg_out == nullptr || exp_avg_sq_out == nullptr)
    return LP_ERR_INVALID_ARGUMENT;
  const int64_t blocks = state_elements / LP_ADAMW_BLOCK;
  const Extent in[4] = {extent(exp_avg, state_elements, 1, 1, 1),
                        extent(exp_avg_sq, state_elements, 1, 1, 1),
                        extent(exp_avg_scale, blocks, 1, 1, 4),
                        extent(exp_avg_sq_scale, blocks, 1, 1, 4)};
  const Extent m = extent(exp_avg_out, state_elements, 1, 1, 4),
               v = extent(exp_avg_sq_out, state_elements, 1, 1, 4);
  if (overlap(m, v)) return LP_ERR_INVALID_ARGUMENT;
  for (const Extent& e : in)
    if (overlap(e, m) || overlap(e, v)) return LP_ERR_INVALID_ARGUMENT;
  if (!aligned(exp_avg, 16) || !aligned(exp_avg_sq, 16) || !aligned(exp_avg_scale, 4) ||
      !aligned(exp_avg_sq_scale, 4) || !aligned(exp_avg_out, 16) || !aligned(exp_avg_sq_out, 16))
    return LP_ERR_MISALIGNED;
  Device dev;
  const lp_status st = current_device(&dev);
  if (st != LP_OK) return st;
  return launch_adamw_state_values(exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale,
                                   state_elements / LP_ADAMW_ALIGN, exp_avg_out, exp_avg_sq_out,
                                   static_cast<cudaStream_t>(stream));
}

}  // extern "C"
