// lp_adamw.cu: AdamW over many tensors, the norm of their gradients, and the values
// of 8-bit moments (include/lp_train.h).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "lp_check.cuh"
#include "lp_train_internal.h"

namespace lp {
namespace {

constexpr int kThreads = 256;
constexpr int kRow = LP_ADAMW_ALIGN;    // state elements of a CTA
constexpr int kBlock = LP_ADAMW_BLOCK;  // elements of a warp, with one scale
static_assert(kRow == kBlock * kThreads / 32, "one block of elements a warp");

// The magnitude codes of 8-bit moments: code c > 0 is the float of bits (c + kFirst) << kShift.
template <bool kSigned>
struct Code {
  static constexpr int kShift = kSigned ? 20 : 19;
  static constexpr int kFirst = kSigned ? 889 : 1777;
  // the lowest code's value over 2^kShift: what a random number below 2^kShift is scaled
  // by to round a magnitude below that value to it or to zero
  static constexpr float kLow = kSigned ? 0x1.4p-36f : 0x1.2p-35f;

  static __device__ __forceinline__ float decode(uint32_t byte, float scale) {
    const uint32_t c = kSigned ? byte & 127u : byte;
    float v = c > 0 ? __uint_as_float((c + kFirst) << kShift) : 0.f;
    if (kSigned && byte >= 128u) v = -v;
    return v * scale;
  }
  // x over the block's largest magnitude, as a byte; half: 16 random bits
  static __device__ __forceinline__ uint32_t encode(float x, float inverse, uint32_t half) {
    const float part = fminf(fabsf(x) * inverse, 1.f);
    const uint32_t bits = __float_as_uint(part), r = half << (kShift - 16);
    uint32_t c = ((bits + r) >> kShift) - kFirst;
    if (bits < uint32_t(kFirst + 1) << kShift) c = part > static_cast<float>(r) * kLow ? 1u : 0u;
    if (kSigned && x < 0.f && c > 0) c += 128u;
    return c;
  }
};

// Philox 4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers:
// as easy as 1, 2, 3", SC11) at counter (group, step) under `seed`.
__device__ __forceinline__ void random_words(uint64_t group, uint64_t step, uint64_t seed,
                                             uint32_t (&w)[4]) {
  uint32_t c0 = uint32_t(group), c1 = uint32_t(group >> 32), c2 = uint32_t(step),
           c3 = uint32_t(step >> 32), k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    c0 = uint32_t(b >> 32) ^ c1 ^ k0;
    c1 = uint32_t(b);
    c2 = uint32_t(a >> 32) ^ c3 ^ k1;
    c3 = uint32_t(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A block's scale from its largest magnitude: 0 below 2^-100, NaN when not finite.
__device__ __forceinline__ float scale_of(float largest, bool finite) {
  if (!finite) return __int_as_float(0x7fffffff);
  return largest < 0x1p-100f ? 0.f : largest;
}

__global__ void __launch_bounds__(kThreads) lp_adamw_kernel(AdamwArgs a) {
  const int64_t row = blockIdx.x;
  const int32_t index = a.table[row];
  if (!LP_CHECK(index >= 0 && index < a.n_tensors, kChkPlan)) return;
  const AdamwRecord rec = a.records[index];
  const float clip = a.grad_scale != nullptr ? *a.grad_scale : 1.f;
  if (clip != clip) return;
  const float lr = a.lr * rec.lr_scale;
  const float kept = 1.f - lr * rec.weight_decay, step_size = a.step_size * rec.lr_scale;
  const int lane = threadIdx.x & 31;
  const bool small = a.exp_avg_scale != nullptr;
  // this warp's block: its first element in the tensor and in the flat buffers
  const int64_t first = (row - rec.first_row) * kRow + (threadIdx.x >> 5) * kBlock;
  const int64_t flat = row * kRow + (threadIdx.x >> 5) * kBlock;
  if (first >= rec.n) return;
  const int64_t block = flat / kBlock;
  float m[8], u[8];
  float top_m = 0.f, top_u = 0.f;
  bool finite = true;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = (k >> 2) * 128 + lane * 4 + (k & 3);
    m[k] = u[k] = 0.f;
    if (first + e >= rec.n) continue;
    float g = rec.grad_bf16
                  ? __bfloat162float(static_cast<const __nv_bfloat16*>(rec.grad)[first + e])
                  : static_cast<const float*>(rec.grad)[first + e];
    if (a.grad_scale != nullptr) g *= clip;
    float m0, v0;
    if (small) {
      m0 = Code<true>::decode(static_cast<uint8_t*>(a.exp_avg)[flat + e], a.exp_avg_scale[block]);
      v0 = Code<false>::decode(static_cast<uint8_t*>(a.exp_avg_sq)[flat + e],
                               a.exp_avg_sq_scale[block]);
      v0 *= v0;
    } else {
      m0 = static_cast<float*>(a.exp_avg)[flat + e];
      v0 = static_cast<float*>(a.exp_avg_sq)[flat + e];
    }
    m[k] = a.beta1 * m0 + a.rest1 * g;
    const float v = a.beta2 * v0 + a.rest2 * (g * g);
    u[k] = sqrtf(v);
    const float change = m[k] / (u[k] * a.root_scale + a.eps);
    const float p = rec.param[first + e] * kept - step_size * change;
    rec.param[first + e] = p;
    if (rec.copy != nullptr) rec.copy[first + e] = __float2bfloat16_rn(p);
    if (!small) {
      static_cast<float*>(a.exp_avg)[flat + e] = m[k];
      static_cast<float*>(a.exp_avg_sq)[flat + e] = v;
    }
    top_m = fmaxf(top_m, fabsf(m[k]));
    top_u = fmaxf(top_u, u[k]);
    finite = finite && fabsf(m[k]) <= 0x1.fffffep127f && u[k] <= 0x1.fffffep127f;
  }
  if (!small) return;
  finite = __all_sync(0xffffffffu, finite);
  const float scale_m = scale_of(warp_max(top_m), finite);
  const float scale_u = scale_of(warp_max(top_u), finite);
  const float inv_m = scale_m > 0.f ? 1.f / scale_m : 0.f;
  const float inv_u = scale_u > 0.f ? 1.f / scale_u : 0.f;
  __syncwarp();  // every lane has read the old scales
  if (lane == 0) {
    a.exp_avg_scale[block] = scale_m;
    a.exp_avg_sq_scale[block] = scale_u;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[4];
    random_words(uint64_t(flat / 4 + h * 32 + lane), a.step, a.seed, w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = h * 128 + lane * 4 + j;
      static_cast<uint8_t*>(a.exp_avg)[flat + e] =
          uint8_t(Code<true>::encode(m[h * 4 + j], inv_m, w[j] & 0xffffu));
      static_cast<uint8_t*>(a.exp_avg_sq)[flat + e] =
          uint8_t(Code<false>::encode(u[h * 4 + j], inv_u, w[j] >> 16));
    }
  }
}

__global__ void __launch_bounds__(kThreads)
    lp_adamw_square_sum_kernel(const AdamwRecord* records, const int32_t* table, int64_t n_tensors,
                               float* sums) {
  __shared__ float slots[kThreads / 32];
  const int64_t row = blockIdx.x;
  const int32_t index = table[row];
  if (!LP_CHECK(index >= 0 && index < n_tensors, kChkPlan)) return;
  const AdamwRecord rec = records[index];
  const int64_t first = (row - rec.first_row) * kRow;
  float s = 0.f;
  for (int e = threadIdx.x; e < kRow && first + e < rec.n; e += kThreads) {
    const float g = rec.grad_bf16
                        ? __bfloat162float(static_cast<const __nv_bfloat16*>(rec.grad)[first + e])
                        : static_cast<const float*>(rec.grad)[first + e];
    s += g * g;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kThreads / 32; ++w) s += slots[w];
  sums[row] = s;
}

__global__ void __launch_bounds__(kThreads)
    lp_adamw_norm_kernel(const float* sums, int64_t rows, float max_norm, float* norm_out) {
  __shared__ double slots[kThreads];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < rows; i += kThreads) s += sums[i];
  slots[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < kThreads; ++i) s += slots[i];
  const float norm = static_cast<float>(sqrt(s));
  norm_out[0] = norm;
  norm_out[1] = norm <= 0x1.fffffep127f ? fminf(max_norm / (norm + 1e-6f), 1.f)
                                        : __int_as_float(0x7fffffff);
}

__global__ void __launch_bounds__(kThreads)
    lp_adamw_values_kernel(const uint8_t* m, const uint8_t* u, const float* m_scale,
                           const float* u_scale, float* m_out, float* v_out) {
  for (int e = threadIdx.x; e < kRow; e += kThreads) {
    const int64_t i = int64_t(blockIdx.x) * kRow + e;
    m_out[i] = Code<true>::decode(m[i], m_scale[i / kBlock]);
    const float root = Code<false>::decode(u[i], u_scale[i / kBlock]);
    v_out[i] = root * root;
  }
}

}  // namespace

lp_status launch_adamw_step(const AdamwArgs& a, cudaStream_t stream) {
  lp_adamw_kernel<<<unsigned(a.rows), kThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

size_t adamw_grad_norm_workspace(int64_t rows) {
  return static_cast<size_t>(rows > 0 ? rows : 1) * 4;
}

lp_status launch_adamw_grad_norm(const AdamwRecord* records, const int32_t* table,
                                 int64_t n_tensors, int64_t rows, float max_norm, float* norm_out,
                                 void* workspace, cudaStream_t stream) {
  float* sums = static_cast<float*>(workspace);
  if (rows > 0)
    lp_adamw_square_sum_kernel<<<unsigned(rows), kThreads, 0, stream>>>(records, table, n_tensors,
                                                                        sums);
  lp_adamw_norm_kernel<<<1, kThreads, 0, stream>>>(sums, rows, max_norm, norm_out);
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

lp_status launch_adamw_state_values(const void* exp_avg, const void* exp_avg_sq,
                                    const float* exp_avg_scale, const float* exp_avg_sq_scale,
                                    int64_t rows, float* m_out, float* v_out,
                                    cudaStream_t stream) {
  lp_adamw_values_kernel<<<unsigned(rows), kThreads, 0, stream>>>(
      static_cast<const uint8_t*>(exp_avg), static_cast<const uint8_t*>(exp_avg_sq), exp_avg_scale,
      exp_avg_sq_scale, m_out, v_out);
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

cudaError_t take_check_word_adamw(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
