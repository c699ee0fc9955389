// lp_norm.cu: the residual norm and its backward pass (include/lp_train.h).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "lp_check.cuh"
#include "lp_train_internal.h"

namespace lp {
namespace {

constexpr int kThreads = 256;
// The backward's row slots: one CTA per SM of a GB300.  Fixed, so that the order in
// which rows are summed does not depend on the device's partition.
constexpr int64_t kSlots = 152;

__device__ __forceinline__ float get(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float get(const __nv_bfloat16* p, int64_t i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ void put(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, int64_t i, float v) {
  p[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ float weight_at(const void* w, bool bf16, int64_t i) {
  return bf16 ? get(static_cast<const __nv_bfloat16*>(w), i) : get(static_cast<const float*>(w), i);
}
template <class T>
__device__ __forceinline__ T* row_of(const Rows& r, int64_t t) {
  return static_cast<T*>(r.p) + t * r.ld;
}

// Sum over the block's threads, the same for all of them; `slots` holds a float a warp.
__device__ __forceinline__ float block_sum(float v, float* slots) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) v += slots[w];
  return v;
}

template <class R, class A>
__global__ void __launch_bounds__(kThreads) lp_residual_norm_kernel(NormArgs a) {
  extern __shared__ float stream[];
  __shared__ float slots[kThreads / 32];
  const int64_t t = blockIdx.x;
  if (!LP_CHECK(t < a.T, kChkRowIndex)) return;
  const int64_t d = a.d;
  const R* r = row_of<const R>(a.residual, t);
  const A* y = a.branch.p ? row_of<const A>(a.branch, t) : nullptr;
  const A* g = a.gate.p ? row_of<const A>(a.gate, t) : nullptr;
  float root_y = 1.f;
  if (a.branch_weight != nullptr) {
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < d; c += kThreads) s += get(y, c) * get(y, c);
    root_y = 1.f / sqrtf(block_sum(s, slots) / static_cast<float>(d) + a.eps);
    if (a.branch_rstd != nullptr && threadIdx.x == 0) a.branch_rstd[t] = root_y;
  }
  float s = 0.f;
  for (int64_t c = threadIdx.x; c < d; c += kThreads) {
    float v = get(r, c);
    if (y != nullptr) {
      float n = get(y, c);
      if (a.branch_weight != nullptr) n = n * root_y * weight_at(a.branch_weight, a.weight_bf16, c);
      if (g != nullptr) n *= get(g, c);
      v = a.residual_scale * v + a.branch_scale * n;
      put(row_of<R>(a.residual_out, t), c, v);
    }
    stream[c] = v;
    s += v * v;
  }
  if (a.weight == nullptr) return;
  const float root = 1.f / sqrtf(block_sum(s, slots) / static_cast<float>(d) + a.eps);
  if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[t] = root;
  for (int64_t c = threadIdx.x; c < d; c += kThreads)
    put(row_of<A>(a.normed, t), c, stream[c] * root * weight_at(a.weight, a.weight_bf16, c));
}

// The sums of one CTA's rows in shared memory, [3][d]: grad_weight, grad_branch_weight
// and the gradient of a one-row gate.
template <class R, class A>
__global__ void __launch_bounds__(kThreads) lp_residual_norm_grad_kernel(NormGradArgs a) {
  extern __shared__ float sums[];
  __shared__ float slots[kThreads / 32];
  const int64_t d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  const bool post = a.branch_weight != nullptr;
  for (int64_t c = threadIdx.x; c < 3 * d; c += kThreads) sums[c] = 0.f;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const R* s = a.residual_out.p ? row_of<const R>(a.residual_out, t) : nullptr;
    const A* y = a.branch.p ? row_of<const A>(a.branch, t) : nullptr;
    const A* g = a.gate.p ? row_of<const A>(a.gate, t) : nullptr;
    const A* dh = a.grad_normed.p ? row_of<const A>(a.grad_normed, t) : nullptr;
    const R* dr = a.grad_residual_out.p ? row_of<const R>(a.grad_residual_out, t) : nullptr;
    const float root = dh != nullptr ? a.rstd[t] : 0.f;
    const float root_y = post ? a.branch_rstd[t] : 1.f;
    float s1 = 0.f, sa = 0.f, sb = 0.f;
    for (int64_t c = threadIdx.x; c < d; c += kThreads) {
      const float x = dh != nullptr ? get(s, c) * root : 0.f;
      const float dx = dh != nullptr ? get(dh, c) * weight_at(a.weight, a.weight_bf16, c) : 0.f;
      s1 += dx * x;
      if (post) {
        float e = a.branch_scale * weight_at(a.branch_weight, a.weight_bf16, c);
        if (g != nullptr) e *= get(g, c);
        e *= get(y, c) * root_y;
        sa += e * ((dr != nullptr ? get(dr, c) : 0.f) + root * dx);
        sb += e * (root * x);
      }
    }
    const float m1 = block_sum(s1, slots) * inv_d;
    const float m2 = post ? (block_sum(sa, slots) - m1 * block_sum(sb, slots)) * inv_d : 0.f;
    for (int64_t c = threadIdx.x; c < d; c += kThreads) {
      float D = dr != nullptr ? get(dr, c) : 0.f;
      if (dh != nullptr) {
        const float x = get(s, c) * root, h = get(dh, c);
        D += root * (h * weight_at(a.weight, a.weight_bf16, c) - x * m1);
        sums[c] += h * x;
      }
      put(row_of<R>(a.grad_residual, t), c, a.residual_scale * D);
      if (y == nullptr) continue;
      const float yh = get(y, c) * root_y;
      const float wb = post ? weight_at(a.branch_weight, a.weight_bf16, c) : 1.f;
      float dn = a.branch_scale * D;
      if (g != nullptr) {
        const float dg = dn * (yh * wb);
        if (a.grad_gate.p != nullptr) {
          if (a.gate.ld != 0)
            put(row_of<A>(a.grad_gate, t), c, dg);
          else
            sums[2 * d + c] += dg;
        }
        dn *= get(g, c);
      }
      if (post) {
        sums[d + c] += dn * yh;
        dn = root_y * (dn * wb - yh * m2);
      }
      put(row_of<A>(a.grad_branch, t), c, dn);
    }
  }
  if (a.partials == nullptr) return;
  __syncthreads();
  for (int64_t c = threadIdx.x; c < 3 * d; c += kThreads)
    a.partials[blockIdx.x * 3 * d + c] = sums[c];
}

// The CTAs' partial sums added in order, one thread a column.
__global__ void __launch_bounds__(kThreads)
    lp_norm_sum_kernel(const float* partials, int64_t parts, int64_t d, float* grad_weight,
                       float* grad_branch_weight, float* grad_gate) {
  float* const out = blockIdx.y == 0 ? grad_weight : blockIdx.y == 1 ? grad_branch_weight : grad_gate;
  const int64_t c = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (out == nullptr || c >= d) return;
  float s = 0.f;
  for (int64_t p = 0; p < parts; ++p) s += partials[(p * 3 + blockIdx.y) * d + c];
  out[c] = s;
}

// The types of the residual stream and of the activations, as template arguments.
template <class F>
lp_status with_types(bool residual_bf16, bool act_bf16, F&& f) {
  if (residual_bf16) {
    if (act_bf16) return f(__nv_bfloat16(), __nv_bfloat16());
    return f(__nv_bfloat16(), float());
  }
  if (act_bf16) return f(float(), __nv_bfloat16());
  return f(float(), float());
}

int64_t row_slots(int64_t T) { return std::min(T, kSlots); }

}  // namespace

lp_status launch_residual_norm(const Device& dev, const NormArgs& a, cudaStream_t stream) {
  return with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
    auto* kernel = lp_residual_norm_kernel<decltype(r), decltype(x)>;
    static PerContextOnce once;
    if (once.run(dev.ctx_id, [&] {
          return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      int(kNormMaxDim * 4));
        }) != cudaSuccess)
      return LP_ERR_CUDA;
    kernel<<<unsigned(a.T), kThreads, size_t(a.d) * 4, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
  });
}

size_t residual_norm_backward_workspace(int64_t T, int64_t d) {
  return static_cast<size_t>(std::max<int64_t>(1, row_slots(T)) * 3 * d * 4);
}

lp_status launch_residual_norm_backward(const Device& dev, const NormGradArgs& a,
                                        cudaStream_t stream) {
  const int64_t parts = row_slots(a.T);
  if (parts > 0) {
    const lp_status st = with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
      auto* kernel = lp_residual_norm_grad_kernel<decltype(r), decltype(x)>;
      static PerContextOnce once;
      if (once.run(dev.ctx_id, [&] {
            return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        int(kNormMaxDim * 12));
          }) != cudaSuccess)
        return LP_ERR_CUDA;
      kernel<<<unsigned(parts), kThreads, size_t(a.d) * 12, stream>>>(a);
      return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
    });
    if (st != LP_OK) return st;
  }
  float* gate_sum = a.gate.ld == 0 ? static_cast<float*>(a.grad_gate.p) : nullptr;
  if (a.grad_weight == nullptr && a.grad_branch_weight == nullptr && gate_sum == nullptr)
    return LP_OK;
  const dim3 grid(unsigned((a.d + kThreads - 1) / kThreads), 3);
  lp_norm_sum_kernel<<<grid, kThreads, 0, stream>>>(a.partials, parts, a.d, a.grad_weight,
                                                    a.grad_branch_weight, gate_sum);
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

cudaError_t take_check_word_norm(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
