// lp_policy.cu: the clipped policy-gradient loss and its gradients (include/lp_train.h).
#include <cuda_runtime.h>

#include <algorithm>

#include "lp_check.cuh"
#include "lp_train_internal.h"

namespace lp {
namespace {

constexpr int kThreads = 1024;
constexpr int kStats = 4;  // w policy, w kl, w entropy, the clipped rows' w

// The sequence of row t: the number of sequences that end at or before it; B when
// there is none, also for the rows before the first.
__device__ __forceinline__ int64_t sequence_of(const int64_t* cu, int64_t B, int64_t t) {
  if (t < cu[0]) return B;
  int64_t lo = 0, hi = B;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (cu[mid + 1] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// One row's terms and gradients before the weight.
struct RowTerms {
  float policy, kl, entropy, clipped, grad;
};
__device__ __forceinline__ RowTerms row_terms(const PolicyArgs& a, int64_t t, float A) {
  RowTerms r{0.f, 0.f, 0.f, 0.f, 0.f};
  const float logp = a.logp[t];
  const float delta = logp - a.old_logp[t];
  const float ratio = expf(delta);
  const bool over = A > 0.f && delta > a.high, under = A < 0.f && delta < a.low;
  r.clipped = over || under ? 1.f : 0.f;
  r.policy = -A * (over ? a.ratio_high : under ? a.ratio_low : ratio);
  r.grad = over || under ? 0.f : -A * ratio;
  if (a.ref_logp != nullptr) {
    const float x = a.ref_logp[t] - logp;
    const float up = expm1f(x);
    r.kl = up - x;
    r.grad -= a.kl_coef * up;
  }
  if (a.entropy != nullptr) r.entropy = a.entropy[t];
  return r;
}

// One CTA: counts, then terms, then the sums in a fixed order.
__global__ void __launch_bounds__(kThreads) lp_policy_kernel(PolicyArgs a) {
  __shared__ unsigned total;
  __shared__ float slots[kThreads][kStats];
  unsigned* counts = static_cast<unsigned*>(a.workspace);
  const int64_t B = a.n_sequences;
  if (threadIdx.x == 0) total = 0;
  if (a.by_sequence)
    for (int64_t i = threadIdx.x; i < B; i += kThreads) counts[i] = 0;
  __syncthreads();
  for (int64_t t = threadIdx.x; t < a.T; t += kThreads) {
    if (a.mask != nullptr && a.mask[t] == 0) continue;
    const int64_t s = a.cu_seqlens != nullptr ? sequence_of(a.cu_seqlens, B, t) : 0;
    if (a.cu_seqlens != nullptr && s == B) continue;
    if (a.by_sequence)
      atomicAdd(&counts[s], 1u);
    else
      atomicAdd(&total, 1u);
  }
  __threadfence_block();
  __syncthreads();
  if (a.by_sequence) {
    unsigned some = 0;
    for (int64_t i = threadIdx.x; i < B; i += kThreads) some += __ldcg(&counts[i]) > 0 ? 1u : 0u;
    atomicAdd(&total, some);
    __syncthreads();
  }
  const float whole = static_cast<float>(max(total, 1u));
  float sum[kStats] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t t = threadIdx.x; t < a.T; t += kThreads) {
    float w = 0.f, A = 0.f;
    bool counted = a.mask == nullptr || a.mask[t] != 0;
    int64_t s = 0;
    if (counted && a.cu_seqlens != nullptr) {
      s = sequence_of(a.cu_seqlens, B, t);
      counted = s < B;
    }
    float grad = 0.f;
    if (counted) {
      w = a.by_sequence ? 1.f / (static_cast<float>(__ldcg(&counts[s])) * whole) : 1.f / whole;
      A = a.advantages[a.per_sequence ? s : t];
      const RowTerms r = row_terms(a, t, A);
      sum[0] += w * r.policy;
      sum[1] += w * r.kl;
      sum[2] += w * r.entropy;
      sum[3] += w * r.clipped;
      grad = w * r.grad;
    }
    a.grad_logp[t] = grad;
    if (a.grad_entropy != nullptr) a.grad_entropy[t] = -a.entropy_coef * w;
  }
  for (int k = 0; k < kStats; ++k) slots[threadIdx.x][k] = sum[k];
  for (int n = kThreads / 2; n > 0; n >>= 1) {
    __syncthreads();
    if (threadIdx.x < n)
      for (int k = 0; k < kStats; ++k) slots[threadIdx.x][k] += slots[threadIdx.x + n][k];
  }
  if (threadIdx.x == 0) {
    const float policy = slots[0][0], kl = slots[0][1], entropy = slots[0][2];
    a.stats[0] = policy + a.kl_coef * kl - a.entropy_coef * entropy;
    a.stats[1] = policy;
    a.stats[2] = kl;
    a.stats[3] = entropy;
    a.stats[4] = slots[0][3];
  }
}

}  // namespace

size_t policy_loss_workspace(int64_t, int64_t n_sequences) {
  return static_cast<size_t>(std::max<int64_t>(1, n_sequences)) * 4;
}

lp_status launch_policy_loss(const PolicyArgs& a, cudaStream_t stream) {
  lp_policy_kernel<<<1, kThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

cudaError_t take_check_word_policy(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
