// lp_norm.cu: the residual norm (include/lp_train.h).
//
// Two sums a row, of the branch's squares and of the new stream's: the second needs the first, so
// a row passes three times over its columns, which stay in registers and in the ring.  Bound by
// HBM (8 bytes a column in bfloat16): 16384 x 2048 with a float32 stream and a normed bfloat16
// branch takes 65 us, 6.2 TB/s; one CTA a row that reads its operands three times took 123, a row
// in registers with a CTA each 88, with the ring 75, with two rows a turn 65.  512 x 4096 takes
// 5.0 us, of which its 16.8 MB are 2.5: the rest is the launch and the chain of loads, two sums
// and stores.  Wider rows, bfloat16: 4096 x 7168 takes 40 us of 35 at the copy rate and 53 with a normed
// branch, 4096 x 12288 68 and 105 of 59; from 8193 columns on a thread holds four groups, which its 64
// registers do not (8 to 96 bytes spill).  Rows that are not aligned cost up to twice that, in
// instructions (4864 x 2047 bfloat16 26 us, 4864 x 2048 13).  lp_norm.cuh says how rows lie over threads
// and come on chip.
#include <type_traits>

#include "lp_norm.cuh"

namespace lp {
namespace {

// With one group a thread a team takes two rows a turn: their waits for the team are one, the
// weights are read once, and the work of one hides the latencies of the other.
template <int G>
constexpr int kRowsATurn = G == 1 ? 2 : 1;

template <class R, class A, int G, bool kPost, int kAlign>
__global__ void __launch_bounds__(kMaxTeam, 2)
    lp_residual_norm_kernel(const __grid_constant__ NormArgs a, const Plan plan) {
  constexpr int kRows = kRowsATurn<G>;
  __shared__ __align__(16) float slots[2][2][kMaxWarps][padded(kRows)];
  extern __shared__ __align__(32) unsigned char ring[];
  const Place p(a.T, a.d, plan.shape);
  const float inv_d = 1.f / static_cast<float>(a.d);
  const bool branch = a.branch.p != nullptr, gate = a.gate.p != nullptr, norm = a.weight != nullptr;
  const int64_t step = int64_t(gridDim.x) * plan.shape.teams;
  int64_t t = int64_t(blockIdx.x) * plan.shape.teams + p.in_cta;
  if (!LP_CHECK(a.d <= a.residual.ld && t - p.in_cta < a.T, kChkRowIndex)) return;
  clear_ring<kAlign, G>(ring, plan.stages * plan.stage_bytes, p);
  // a stage: the residual's rows, the branch's, the gate's
  Stream<R, kAlign> residual;
  Stream<A, kAlign> y, g;
  uint32_t offset = 0;
  const uint32_t stage0 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  residual.template start<G>(stage0, &offset);
  if (branch) y.template start<G>(stage0, &offset);
  if (gate) g.template start<G>(stage0, &offset);
  void* stretch = ring + plan.stages * plan.stage_bytes + p.warp * kStretch;
  const uint32_t accesses = plan.accesses;
  int64_t next = t;  // the row that is fetched next
  const auto fetch = [&](int stage) {
    if (next < a.T) {
      const uint32_t at = stage * plan.stage_bytes;
      residual.template fetch<G>(a.residual, next, at, access_of(accesses, kResidual), p);
      if (branch) y.template fetch<G>(a.branch, next, at, access_of(accesses, kBranch), p);
      if (gate) g.template fetch<G>(a.gate, next, at, access_of(accesses, kGate), p);
    }
    next += step;
    commit_copies();
  };
  for (int s = 0; s + kRows < plan.stages; ++s) fetch(s);
  const bool wide_w = access_of(accesses, kWeight) == kWide;
  const bool wide_b = access_of(accesses, kBranchWeight) == kWide;
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
    // a row that the team does not have is computed like the others, of what the ring holds, and
    // not written
    Pairs v[kRows][G];
    float root_y[kRows] = {}, root[kRows] = {};
    if (kPost) {
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        float2 s = both(0.f);
#pragma unroll
        for (int k = 0; k < G; ++k) {
          Pairs n;
          y.get(a.branch, t + j * step, at[j], k, n);
#pragma unroll
          for (int e = 0; e < 4; ++e) s = fma(n[e], n[e], s);
        }
        root_y[j] = s.x + s.y;
      }
      team_sum(root_y, slots[turn][0], p);
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        root_y[j] = 1.f / sqrtf(__fmaf_rn(root_y[j], inv_d, a.eps));
        if (a.branch_rstd != nullptr && p.i == 0 && t + j * step < a.T &&
            LP_CHECK(p.has(t + j * step), kChkRowIndex))
          a.branch_rstd[t + j * step] = root_y[j];
      }
    }
#pragma unroll
    for (int k = 0; k < G; ++k) {
      Pairs wb;
      if (kPost) read_weight(a.branch_weight, a.weight_bf16, k, wide_b, p, wb);
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        Pairs& vk = v[j][k];
        residual.get(a.residual, t + j * step, at[j], k, vk);
        if (!branch) continue;
        Pairs n;
        y.get(a.branch, t + j * step, at[j], k, n);
        if (kPost)
#pragma unroll
          for (int e = 0; e < 4; ++e) n[e] = mul(mul(n[e], both(root_y[j])), wb[e]);
        if (gate) {
          Pairs f;
          g.get(a.gate, t + j * step, at[j], k, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) n[e] = mul(n[e], f[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vk[e] = fma(both(a.branch_scale), n[e], mul(both(a.residual_scale), vk[e]));
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      float2 s = both(0.f);
#pragma unroll
      for (int k = 0; k < G; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fma(v[j][k][e], v[j][k][e], s);
      root[j] = s.x + s.y;
      if (branch)
#pragma unroll
        for (int k = 0; k < G; ++k)
          put<R, kAlign>(a.residual_out, t + j * step, k, t + j * step < a.T,
                        access_of(accesses, kOut), p, stretch, v[j][k]);
    }
    if (!norm) continue;
    team_sum(root, slots[turn][1], p);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      root[j] = 1.f / sqrtf(__fmaf_rn(root[j], inv_d, a.eps));
      if (a.rstd != nullptr && p.i == 0 && t + j * step < a.T &&
          LP_CHECK(p.has(t + j * step), kChkRowIndex))
        a.rstd[t + j * step] = root[j];
    }
#pragma unroll
    for (int k = 0; k < G; ++k) {
      Pairs w;
      read_weight(a.weight, a.weight_bf16, k, wide_w, p, w);
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][k][e] = mul(mul(v[j][k][e], both(root[j])), w[e]);
        put<A, kAlign>(a.normed, t + j * step, k, t + j * step < a.T, access_of(accesses, kNormed),
                      p, stretch, v[j][k]);
      }
    }
  }
}

// The CTAs of an SM have up to 1024 threads between them, each CTA with rows in flight of its own,
// and this much shared memory for them.
constexpr int kForwardBytes = 216 << 10;

template <int G>
lp_status launch_forward(const Device& dev, const NormArgs& a, uint32_t accesses, Align align,
                         cudaStream_t stream) {
  return with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
    using R = decltype(r);
    using A = decltype(x);
    const auto launch = [&](auto* kernel, PerContextOnce* once) {
      if (!allow_ring(kernel, dev, once)) return LP_ERR_CUDA;
      Plan plan{shape_of(a.d, G, a.T), accesses, 1, 0};
      const int threads = plan.shape.team * plan.shape.teams;
      const int columns = int(sizeof(R)) + (a.branch.p ? int(sizeof(A)) : 0) + (a.gate.p ? int(sizeof(A)) : 0);
      // as many CTAs as leave each the rows that it works on: 4864 x 2048 in float32 with a gate
      // takes 34.8 us so, and 38 with one row more ahead and half of the CTAs
      const int least = stage_bytes_of(threads, G, columns, align != kAligned) * kRowsATurn<G> +
                        (align == kAligned ? 0 : threads / 32 * kStretch);
      const int ctas = std::max(1, std::min(1024 / threads, kForwardBytes / least));
      const int64_t all = (a.T + plan.shape.teams - 1) / plan.shape.teams;
      const int64_t blocks = std::min<int64_t>(all, kSlots * ctas);
      const int smem = plan_ring(&plan, columns, G, align != kAligned, (all + blocks - 1) / blocks,
                                 kRowsATurn<G>, kForwardBytes / ctas);
      kernel<<<unsigned(blocks), threads, smem, stream>>>(a, plan);
      return launched();
    };
    static PerContextOnce once[6];
    const auto with_post = [&](auto post, PerContextOnce* once) {
      constexpr bool kPost = decltype(post)::value;
      constexpr Align kLeast = sizeof(R) + sizeof(A) < 8 ? kByElements : kByWords;
      return align == kAligned   ? launch(lp_residual_norm_kernel<R, A, G, kPost, kAligned>, once)
             : align == kByWords ? launch(lp_residual_norm_kernel<R, A, G, kPost, kByWords>, once + 1)
                                 : launch(lp_residual_norm_kernel<R, A, G, kPost, kLeast>, once + 2);
    };
    return a.branch_weight != nullptr ? with_post(std::true_type(), once)
                                      : with_post(std::false_type(), once + 3);
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
  const bool fast = all_wide(accesses, {kResidual, kBranch, kGate, kOut, kNormed}, a.d) &&
                    near(a.residual) && near(a.branch) && near(a.gate) && near(a.residual_out) &&
                    near(a.normed);
  const Align align = fast ? kAligned
                      : any_halves(accesses, {kResidual, kBranch, kGate, kOut, kNormed}) ? kByElements
                                                                                         : kByWords;
  // as few groups a thread as its team's 512 threads allow
  if (a.d <= kMaxTeam * 8) return launch_forward<1>(dev, a, accesses, align, stream);
  if (a.d <= kMaxTeam * 16) return launch_forward<2>(dev, a, accesses, align, stream);
  return launch_forward<4>(dev, a, accesses, align, stream);
}

cudaError_t take_check_word_norm(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
