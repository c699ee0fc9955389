// lp_layer_norm_backward.cu: the backward pass of the layer norm (include/lp_tune.h).
//
// A row takes one round of two sums, of dx and of dx x; a CTA takes rows in turn and keeps its share
// of the sums over rows (grad_weight, grad_bias) in registers, which a second kernel adds up in a
// fixed order.  lp_norm.cuh says how rows lie over threads and come on chip.
//
// 8192 x 4096 bfloat16 takes 53 us (0.74 of the measured copy rate), 16384 x 2048 under a float32 stream 92
// (0.86): one CTA an SM, since the sums over rows fill the registers, so that its warps wait together for a
// row's sums, and then the second kernel (4 us).  512 x 4096 takes 10 us, three or four rows a CTA and the second
// kernel; rows off 8 elements are bound by instructions: 1021 x 2047 float32 16 us for 5 of bytes.
#include <type_traits>

#include "lp_layer_norm.cuh"
#include "lp_tune_internal.h"

namespace lp {
namespace {

// Floats from one sum of a CTA to the next in the workspace: whole groups.
__host__ __device__ __forceinline__ int64_t pitch_of(int64_t d) { return (d + 7) / 8 * 8; }

// Where the registers and the ring allow, a team that has more than one row takes two a turn.
template <class R, class A, int G>
constexpr int kRowsATurn = G == 1 && sizeof(R) + sizeof(A) <= 6 ? 2 : 1;

// With one or two groups a thread a row's x and D stay in registers between the sums and the outputs
// (4096 x 8192 bfloat16 69 us, formed again 76); with four they are formed again from the ring, since the
// registers do not hold them beside the sums.
template <class R, class A, int G, int kRows, int kAlign>
__global__ void __launch_bounds__(kMaxTeam)
    lp_layer_norm_grad_kernel(const __grid_constant__ LayerNormGradArgs a, const Plan plan) {
  constexpr bool kHold = G <= 2, kKeep = G == 1;  // the row, the weight
  __shared__ __align__(16) float slots[2][kMaxWarps][padded(kRows * 2)];
  extern __shared__ __align__(32) unsigned char ring[];
  const Place p(a.T, a.d, plan.shape);
  const float inv_d = 1.f / static_cast<float>(a.d);
  const bool has_dr = a.grad_residual_out.p != nullptr;
  Pairs sum_w[G] = {}, sum_b[G] = {};
  const int64_t step = int64_t(gridDim.x) * plan.shape.teams;
  int64_t t = int64_t(blockIdx.x) * plan.shape.teams + p.in_cta;
  if (!LP_CHECK(a.d <= a.grad_residual.ld && t - p.in_cta < a.T, kChkRowIndex)) return;
  clear_ring<kAlign, G>(ring, plan.stages * plan.stage_bytes, p);
  // a stage: the rows of the stream, its gradient, the norm's gradient
  Stream<R, kAlign> s, dr;
  Stream<A, kAlign> dh;
  uint32_t offset = 0;
  const uint32_t stage0 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  s.template start<G>(stage0, &offset);
  if (has_dr) dr.template start<G>(stage0, &offset);
  dh.template start<G>(stage0, &offset);
  void* stretch = ring + plan.stages * plan.stage_bytes + p.warp * kStretch;
  const uint32_t accesses = plan.accesses;
  int64_t next = t;  // the row that is fetched next
  const auto fetch = [&](int stage) {
    const uint32_t at = stage * plan.stage_bytes;
    if (next < a.T) {
      s.template fetch<G>(a.residual_out, next, at, access_of(accesses, kOut), p);
      dh.template fetch<G>(a.grad_normed, next, at, access_of(accesses, kGradNormed), p);
      if (has_dr)
        dr.template fetch<G>(a.grad_residual_out, next, at, access_of(accesses, kGradOut), p);
    } else {
      s.template zero<G>(at), dh.template zero<G>(at);
      if (has_dr) dr.template zero<G>(at);
    }
    next += step;
    commit_copies();
  };
  for (int n = 0; n + kRows < plan.stages; ++n) fetch(n);
  const bool wide_w = access_of(accesses, kWeight) == kWide;
  Pairs kept_w;
  const auto weight_of = [&](int k, Pairs& w) {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = both(1.f);
    if (a.weight != nullptr) read_weight(a.weight, a.weight_bf16, k, wide_w, p, w);
  };
  if (kKeep) weight_of(0, kept_w);
  // the rows' means and roots, loaded a turn ahead
  float root[kRows], mean[kRows];
  const auto load_roots = [&](int64_t first) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const bool mine = first + j * step < a.T && LP_CHECK(p.has(first + j * step), kChkRowIndex);
      root[j] = mine ? a.rstd[first + j * step] : 0.f;
      mean[j] = mine ? a.mean[first + j * step] : 0.f;
    }
  };
  load_roots(t);
  int stage = 0, turn = 0;
  // every team runs as many turns as the CTA's first, so that all meet at the barriers
  for (; t - p.in_cta < a.T; t += kRows * step, turn ^= 1) {
    __syncwarp();  // the stages that are copied into have been read by the warp
    int to = stage - kRows;
    if (to < 0) to += plan.stages;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      fetch(to);
      if (++to == plan.stages) to = 0;
    }
    wait_copies(plan.stages - kRows);
    __syncwarp();
    uint32_t at[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      at[j] = stage * plan.stage_bytes;
      if (++stage == plan.stages) stage = 0;
    }
    Pairs x[kRows][kHold ? G : 1], D[kRows][kHold ? G : 1];
    // x and D before the sums' part of group k of the turn's row j; h: grad_normed
    const auto form = [&](int j, int k, const Pairs& w, Pairs& xk, Pairs& Dk, Pairs& h) {
      s.get(a.residual_out, t + j * step, at[j], k, xk);
      dh.get(a.grad_normed, t + j * step, at[j], k, h);
      if (has_dr) {
        dr.get(a.grad_residual_out, t + j * step, at[j], k, Dk);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) Dk[e] = both(0.f);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xk[e] = mul(add(xk[e], both(-mean[j])), both(root[j]));
        Dk[e] = fma(both(root[j]), mul(h[e], w[e]), Dk[e]);
      }
    };
    float m[kRows * 2];
    float2 sums[kRows][2];
#pragma unroll
    for (int j = 0; j < kRows; ++j) sums[j][0] = sums[j][1] = both(0.f);
#pragma unroll
    for (int k = 0; k < G; ++k) {
      Pairs w;
      if (!kKeep) weight_of(k, w);
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        Pairs h, x1, D1;
        Pairs& xk = kHold ? x[j][kHold ? k : 0] : x1;
        form(j, k, kKeep ? kept_w : w, xk, kHold ? D[j][kHold ? k : 0] : D1, h);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // columns past the row have a gradient of 0
          const float2 dx = mul(h[e], kKeep ? kept_w[e] : w[e]);
          sums[j][0] = add(sums[j][0], dx);
          sums[j][1] = fma(dx, xk[e], sums[j][1]);
          sum_w[k][e] = fma(h[e], xk[e], sum_w[k][e]);
          sum_b[k][e] = add(sum_b[k][e], h[e]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) m[j * 2 + q] = sums[j][q].x + sums[j][q].y;
    team_sum(m, slots[turn], p);
#pragma unroll
    for (int k = 0; k < G; ++k) {
      Pairs w;
      if (!kHold) weight_of(k, w);
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const bool mine = t + j * step < a.T;
        Pairs h, x1, D1;
        if (!kHold) form(j, k, w, x1, D1, h);
        Pairs& xk = kHold ? x[j][kHold ? k : 0] : x1;
        Pairs& Dk = kHold ? D[j][kHold ? k : 0] : D1;
        // rstd mean(dx) and rstd mean(dx x)
        const float m0 = root[j] * (m[2 * j] * inv_d), m1 = root[j] * (m[2 * j + 1] * inv_d);
#pragma unroll
        for (int e = 0; e < 4; ++e) Dk[e] = fma(both(-m1), xk[e], add(Dk[e], both(-m0)));
        put<R, kAlign>(a.grad_residual, t + j * step, k, mine, access_of(accesses, kGradResidual), p,
                       stretch, Dk);
        if (a.grad_branch.p != nullptr)
          put<A, kAlign>(a.grad_branch, t + j * step, k, mine, access_of(accesses, kGradBranch), p,
                         stretch, Dk);
      }
    }
    load_roots(t + kRows * step);
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.partials == nullptr) return;
  // the teams' sums in order, then the CTA's: two rows of whole groups in the workspace, or of a
  // lone CTA the sums themselves
  float2* shared = reinterpret_cast<float2*>(ring);  // all copies have been waited for
  float* part = a.partials + int64_t(blockIdx.x) * 2 * pitch_of(a.d);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    Pairs(&sum)[G] = q == 0 ? sum_w : sum_b;
    float* const out = q == 0 ? a.grad_weight : a.grad_bias;
    if (out == nullptr) continue;
    for (int from = 1; from < plan.shape.teams; ++from) {
      __syncthreads();
      if (p.in_cta == from)
#pragma unroll
        for (int k = 0; k < G; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) shared[(k * p.team + p.i) * 4 + e] = sum[k][e];
      __syncthreads();
      if (p.in_cta == 0)
#pragma unroll
        for (int k = 0; k < G; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[k][e] = add(sum[k][e], shared[(k * p.team + p.i) * 4 + e]);
    }
    if (p.in_cta == 0)
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const int c = 8 * (p.i + k * p.team);
        if (gridDim.x > 1) {
          if (c < p.d && LP_CHECK(c >= 0 && c + 8 <= pitch_of(a.d), kChkSplitIndex))
            store_group(part + q * pitch_of(a.d) + c, pack(sum[k], float()));
          continue;
        }
        if (!LP_CHECK(c >= 0, kChkCopyIndex)) continue;
        if (c + 8 <= p.d && reinterpret_cast<uintptr_t>(out) % 32 == 0) {
          store_group(out + c, pack(sum[k], float()));
          continue;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < p.d) out[c + e] = e & 1 ? sum[k][e / 2].y : sum[k][e / 2].x;
      }
  }
}

// The CTAs' partial sums: 16 threads a column take every sixteenth part in order, and their
// sums are added in order.
constexpr int kSumLanes = 16;
__global__ void __launch_bounds__(32 * kSumLanes)
    lp_layer_norm_sum_kernel(const float* partials, int64_t parts, int64_t d, float* grad_weight,
                             float* grad_bias) {
  __shared__ float slots[kSumLanes][32];
  float* const out = blockIdx.y == 0 ? grad_weight : grad_bias;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, from = threadIdx.x / 32;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane, pitch = pitch_of(d);
  // launched as a programmatic dependent of the row kernel: wait for its partial sums
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.f;
  if (c < d) {
    const float* p = partials + (int64_t(from) * 2 + blockIdx.y) * pitch + c;
#pragma unroll 4
    for (int64_t k = from; k < parts; k += kSumLanes, p += 2 * kSumLanes * pitch)
      if (LP_CHECK(p >= partials && p < partials + parts * 2 * pitch, kChkSplitIndex)) s += __ldcg(p);
  }
  slots[from][lane] = s;
  __syncthreads();
  if (from != 0 || c >= d) return;
#pragma unroll
  for (int k = 1; k < kSumLanes; ++k) s += slots[k][lane];
  out[c] = s;
}

// Groups of a thread, the CTAs of an SM (two where a row takes no more than half of its threads)
// and how many CTAs there are.
int groups_of(int64_t d) { return d <= kMaxTeam * 8 ? 1 : d <= kMaxTeam * 16 ? 2 : 4; }
int ctas_of_sm(int threads) { return threads <= kMaxTeam / 2 ? 2 : 1; }
int64_t backward_blocks(int64_t T, int64_t d) {
  const Shape s = shape_of(d, groups_of(d), T);
  return std::min((T + s.teams - 1) / s.teams, kSlots * ctas_of_sm(s.team * s.teams));
}

template <int G>
lp_status launch_backward(const Device& dev, const LayerNormGradArgs& a, uint32_t accesses,
                          Align align, int64_t blocks, cudaStream_t stream) {
  return with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
    using R = decltype(r);
    using A = decltype(x);
    constexpr int kMost = kRowsATurn<R, A, G>;
    Plan plan{shape_of(a.d, G, a.T), accesses, 1, 0};
    const int64_t at_once = blocks * plan.shape.teams, rows = (a.T + at_once - 1) / at_once;
    const auto launch = [&](auto* kernel, int least, PerContextOnce* once) {
      if (!allow_ring(kernel, dev, once)) return LP_ERR_CUDA;
      const int columns = int(sizeof(R) + sizeof(A)) + (a.grad_residual_out.p ? int(sizeof(R)) : 0);
      int smem = plan_ring(&plan, columns, G, align != kAligned, rows, least,
                           kRingBytes / ctas_of_sm(plan.shape.team * plan.shape.teams));
      if (plan.shape.teams > 1) smem = std::max(smem, plan.shape.team * G * 8 * int(sizeof(float)));
      kernel<<<unsigned(blocks), plan.shape.team * plan.shape.teams, smem, stream>>>(a, plan);
      return launched();
    };
    static PerContextOnce once[4];
    constexpr Align kLeast = sizeof(R) + sizeof(A) < 8 ? kShifted : kByWords;
    if (align == kByWords)
      return launch(lp_layer_norm_grad_kernel<R, A, G, 1, kByWords>, 1, once);
    if (align == kShifted) return launch(lp_layer_norm_grad_kernel<R, A, G, 1, kLeast>, 1, once + 1);
    if constexpr (kMost > 1)
      if (rows == 1) return launch(lp_layer_norm_grad_kernel<R, A, G, 1, kAligned>, 1, once + 2);
    return launch(lp_layer_norm_grad_kernel<R, A, G, kMost, kAligned>, kMost, once + 3);
  });
}

}  // namespace

size_t layer_norm_backward_workspace(int64_t T, int64_t d) {
  return static_cast<size_t>(backward_blocks(std::max<int64_t>(T, 1), d) * 2 * pitch_of(d) * 4);
}

lp_status launch_layer_norm_backward(const Device& dev, const LayerNormGradArgs& a,
                                     cudaStream_t stream) {
  const int64_t blocks = a.T > 0 ? backward_blocks(a.T, a.d) : 0;
  if (blocks > 0) {
    const uint32_t accesses = access_bits(kOut, a.residual_out, a.residual_bf16) |
                              access_bits(kWeight, a.weight, 0, a.weight_bf16) |
                              access_bits(kGradNormed, a.grad_normed, a.act_bf16) |
                              access_bits(kGradOut, a.grad_residual_out, a.residual_bf16) |
                              access_bits(kGradResidual, a.grad_residual, a.residual_bf16) |
                              access_bits(kGradBranch, a.grad_branch, a.act_bf16);
    const auto operands = {int(kOut), int(kGradNormed), int(kGradOut), int(kGradResidual), int(kGradBranch)};
    const bool fast = all_wide(accesses, operands, a.d) && near(a.residual_out) &&
                      near(a.grad_normed) && near(a.grad_residual_out) && near(a.grad_residual) &&
                      near(a.grad_branch);
    const Align align = fast ? kAligned : any_halves(accesses, operands) ? kShifted : kByWords;
    const int groups = groups_of(a.d);
    const lp_status st = groups == 1   ? launch_backward<1>(dev, a, accesses, align, blocks, stream)
                         : groups == 2 ? launch_backward<2>(dev, a, accesses, align, blocks, stream)
                                       : launch_backward<4>(dev, a, accesses, align, blocks, stream);
    if (st != LP_OK) return st;
  }
  if (a.grad_weight == nullptr && a.grad_bias == nullptr) return LP_OK;
  if (blocks == 1) return LP_OK;  // the CTA wrote them
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.d + 31) / 32), 2);
  cfg.blockDim = dim3(32 * kSumLanes);
  cfg.stream = stream;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl;
  cfg.numAttrs = blocks > 0 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, lp_layer_norm_sum_kernel, static_cast<const float*>(a.partials),
                         blocks, a.d, a.grad_weight, a.grad_bias) != cudaSuccess)
    return LP_ERR_CUDA;
  return launched();
}

cudaError_t take_check_word_layer_norm_backward(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
