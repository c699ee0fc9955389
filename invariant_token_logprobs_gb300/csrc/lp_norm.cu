// lp_norm.cu: the residual norm (include/lp_train.h).  Bound by HBM: 8 bytes a column
// in bfloat16.  lp_norm.cuh says how rows lie over threads and come on chip.
#include "lp_norm.cuh"

namespace lp {
namespace {

template <class R, class A, int G, bool kPost, bool kFast>
__global__ void __launch_bounds__(kMaxTeam)
    lp_residual_norm_kernel(const __grid_constant__ NormArgs a, const Plan plan) {
  __shared__ float slots[2][2][kMaxWarps][1];
  extern __shared__ __align__(32) unsigned char ring[];
  const Place p(a.d, plan.shape);
  const float inv_d = 1.f / static_cast<float>(a.d);
  const bool branch = a.branch.p != nullptr, gate = a.gate.p != nullptr;
  const int64_t step = int64_t(gridDim.x) * plan.shape.teams;
  int64_t t = int64_t(blockIdx.x) * plan.shape.teams + p.in_cta;
  if (!LP_CHECK(a.d <= a.residual.ld && t - p.in_cta < a.T, kChkRowIndex)) return;
  // a stage: the residual's rows, the branch's, the gate's
  Stream<R> residual;
  Stream<A> y, g;
  int offset = 0;
  residual.template start<kFast, G>(a.residual, t, step, p, ring, &offset);
  if (branch) y.template start<kFast, G>(a.branch, t, step, p, ring, &offset);
  if (gate) g.template start<kFast, G>(a.gate, t, step, p, ring, &offset);
  void* stretch = ring + plan.stages * plan.stage_bytes + p.warp * kStretch;
  const uint32_t accesses = plan.accesses;
  int64_t next = t;  // the row that is fetched next
  const auto fetch = [&](int stage) {
    if (next - p.in_cta < a.T) {  // the CTA has a turn for it
      const uint32_t at = stage * plan.stage_bytes;
      const bool mine = next < a.T;
      residual.template fetch<kFast, G>(at, mine, access_of(accesses, kResidual), p, a.residual.p);
      if (branch) y.template fetch<kFast, G>(at, mine, access_of(accesses, kBranch), p, a.branch.p);
      if (gate) g.template fetch<kFast, G>(at, mine, access_of(accesses, kGate), p, a.gate.p);
    }
    next += step;
    commit_copies();
  };
  for (int s = 0; s + 1 < plan.stages; ++s) fetch(s);
  int stage = 0, turn = 0;
  // every team runs as many turns as the CTA's first, so that all meet at the barriers
  for (; t - p.in_cta < a.T; t += step, turn ^= 1) {
    const int ahead = plan.stages - 1;
    __syncwarp();  // the stage that is copied into has been read by the warp
    fetch(stage == 0 ? ahead : stage - 1);
    wait_copies(ahead);
    __syncwarp();
    const bool mine = t < a.T;
    const uint32_t at = stage * plan.stage_bytes;
    float v[G][8], root_y[1] = {0.f}, root[1] = {0.f};
    if (kPost) {
#pragma unroll
      for (int k = 0; k < G; ++k) {
        float n[8];
        y.get(at, k, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) root_y[0] = __fmaf_rn(n[e], n[e], root_y[0]);
      }
      team_sum(root_y, slots[turn][0], p);
      root_y[0] = 1.f / sqrtf(__fmaf_rn(root_y[0], inv_d, a.eps));
      if (a.branch_rstd != nullptr && p.i == 0 && mine) a.branch_rstd[t] = root_y[0];
    }
#pragma unroll
    for (int k = 0; k < G; ++k) {
      residual.get(at, k, v[k]);
      if (branch) {
        float n[8];
        y.get(at, k, n);
        if (kPost) {
          float w[8];
          read_weight(a.branch_weight, a.weight_bf16, k, access_of(accesses, kBranchWeight) == kWide, p, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) n[e] = n[e] * root_y[0] * w[e];
        }
        if (gate) {
          float f[8];
          g.get(at, k, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) n[e] *= f[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[k][e] = __fmaf_rn(a.branch_scale, n[e], a.residual_scale * v[k][e]);
        write_group<kFast, R>(a.residual_out, t, k, mine, access_of(accesses, kOut), p, stretch, v[k]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) root[0] = __fmaf_rn(v[k][e], v[k][e], root[0]);
    }
    if (a.weight != nullptr) {
      team_sum(root, slots[turn][1], p);
      root[0] = 1.f / sqrtf(__fmaf_rn(root[0], inv_d, a.eps));
      if (a.rstd != nullptr && p.i == 0 && mine) a.rstd[t] = root[0];
#pragma unroll
      for (int k = 0; k < G; ++k) {
        float w[8];
        read_weight(a.weight, a.weight_bf16, k, access_of(accesses, kWeight) == kWide, p, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = v[k][e] * root[0] * w[e];
        write_group<kFast, A>(a.normed, t, k, mine, access_of(accesses, kNormed), p, stretch, w);
      }
    }
    stage = stage + 1 == plan.stages ? 0 : stage + 1;
  }
}

// Several CTAs share an SM, each with rows in flight of its own.
constexpr int kForwardBudget = 48 << 10;  // of a CTA of 256 threads

template <int G>
lp_status launch_forward(const Device& dev, const NormArgs& a, uint32_t accesses, bool fast,
                         cudaStream_t stream) {
  return with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
    using R = decltype(r);
    using A = decltype(x);
    const auto launch = [&](auto* kernel, PerContextOnce* once) {
      if (!allow_ring(kernel, dev, once)) return LP_ERR_CUDA;
      Plan plan{shape_of(a.d, G, a.T), accesses, 1, 0};
      const int threads = plan.shape.team * plan.shape.teams;
      const int64_t all = (a.T + plan.shape.teams - 1) / plan.shape.teams;
      const int64_t blocks = std::min<int64_t>(all, kSlots * (1024 / threads));
      const int columns = int(sizeof(R)) + (a.branch.p ? int(sizeof(A)) : 0) + (a.gate.p ? int(sizeof(A)) : 0);
      const int smem = plan_ring(&plan, columns, G, !fast, (all + blocks - 1) / blocks, 1,
                                 std::max(kForwardBudget * threads / 256, threads * G * 8 * columns));
      kernel<<<unsigned(blocks), threads, smem, stream>>>(a, plan);
      return launched();
    };
    static PerContextOnce once[4];
    if (a.branch_weight != nullptr)
      return fast ? launch(lp_residual_norm_kernel<R, A, G, true, true>, &once[0])
                  : launch(lp_residual_norm_kernel<R, A, G, true, false>, &once[1]);
    return fast ? launch(lp_residual_norm_kernel<R, A, G, false, true>, &once[2])
                : launch(lp_residual_norm_kernel<R, A, G, false, false>, &once[3]);
  });
}

}  // namespace

lp_status launch_residual_norm(const Device& dev, const NormArgs& a, cudaStream_t stream) {
  const uint32_t accesses = access_bits(kResidual, a.residual, a.residual_bf16) |
                            access_bits(kBranch, a.branch, a.act_bf16) |
                            access_bits(kGate, a.gate, a.act_bf16) |
                            access_bits(kBranchWeight, a.branch_weight, 0, a.weight_bf16) |
                            access_bits(kWeight, a.weight, 0, a.weight_bf16) |
                            access_bits(kOut, a.residual_out, a.residual_bf16) |
                            access_bits(kNormed, a.normed, a.act_bf16);
  const bool fast = all_wide(accesses, {kResidual, kBranch, kGate, kOut, kNormed}, a.d);
  // a thread's groups: one while that leaves a CTA of 256 threads or fewer, so that several
  // CTAs fit an SM; more only for rows that 512 threads do not cover
  if (a.d <= kMaxTeam / 2 * 8) return launch_forward<1>(dev, a, accesses, fast, stream);
  if (a.d <= kMaxTeam * 16) return launch_forward<2>(dev, a, accesses, fast, stream);
  return launch_forward<4>(dev, a, accesses, fast, stream);
}

cudaError_t take_check_word_norm(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
