// lp_layer_norm.cu: the layer norm (include/lp_tune.h).
//
// The squares are of the deviations from the row's mean, so a row takes two rounds of sums; it
// stays in registers between them.  (Taking the mean of the squares less the square of the mean
// would need one, and lose what a row's mean is above its spread.)  lp_norm.cuh says how rows lie
// over threads and come on chip.
//
// Bound by HBM where rows are whole groups: 16384 x 2048, float32 stream under bfloat16, 67 us (0.89 of the
// measured copy rate), 8192 x 4096 bfloat16 47 (0.85), without a branch 29 (0.68).  Rows off 8 elements are
// bound by instructions (4-byte copies, outputs through shared memory): 16384 x 2047 bfloat16 98 to 102 us, 0.40.
// One token is bound by the call: 7 us, of which the kernel is 4.
#include <type_traits>

#include "lp_layer_norm.cuh"
#include "lp_tune_internal.h"

namespace lp {
namespace {

// With one group a thread a team takes two rows a turn: their waits for the team are one, and the
// weights are read once (16384 x 1024 float32 under bfloat16 takes 36.8 us so, with one row 38.9; rows off 8
// elements, 16384 x 2047 bfloat16, 102 and 124).  Where both operands are float32 the rows are long enough to
// hide the waits, and one row a turn leaves more CTAs theirs: 8192 x 4096 85 us, with two 92.
template <class R, class A, int G>
constexpr int kRowsATurn = G == 1 && sizeof(R) + sizeof(A) < 8 ? 2 : 1;
// Which rows the wide kernel takes where they are aligned: those of few bytes a column, which are bound by
// instructions and by the waits for the sums, and fit eight warps.  Under a branch a float32 stream's rows gain
// more from the ring's deeper copies (16384 x 2048 with a bfloat16 branch 67 us, by the wide kernel 71; 8192 x 4096
// float32 85 and 93).
bool few_bytes(bool branch, bool residual_bf16, bool act_bf16, int64_t d) {
  return d % 8 == 0 && d <= 8192 && (!branch || (residual_bf16 && act_bf16));
}
// Groups of a thread.  Of the wide kernel's rows two from 257 columns on and four from 4097 (8192 x 4096 bfloat16
// without a branch takes 29 us with two, 27 with four, but a single row 4.6 and 6.3); rows that are not aligned
// have as many, and so the same sums.  Otherwise as few as 512 threads allow, but two from 1024 columns on under a
// stream of the other type (16384 x 2048 float32 under bfloat16 67 us, with one group 75).
int groups_of(bool branch, bool residual_bf16, bool act_bf16, int64_t d) {
  if (few_bytes(branch, residual_bf16, act_bf16, d)) return d <= 256 ? 1 : d <= 4096 ? 2 : 4;
  const int64_t one = residual_bf16 != act_bf16 ? 1024 : kMaxTeam * 8;
  return d <= one ? 1 : d <= kMaxTeam * 16 ? 2 : 4;
}

template <class R, class A, int G, int kAlign>
__global__ void __launch_bounds__(kMaxTeam, 2)
    lp_layer_norm_kernel(const __grid_constant__ LayerNormArgs a, const Plan plan) {
  constexpr int kRows = kRowsATurn<R, A, G>;
  __shared__ __align__(16) float slots[2][2][kMaxWarps][padded(kRows)];
  extern __shared__ __align__(32) unsigned char ring[];
  const Place p(a.T, a.d, plan.shape);
  const float inv_d = 1.f / static_cast<float>(a.d);
  const bool branch = a.branch.p != nullptr;
  const int64_t step = int64_t(gridDim.x) * plan.shape.teams;
  int64_t t = int64_t(blockIdx.x) * plan.shape.teams + p.in_cta;
  if (!LP_CHECK(a.d <= a.residual.ld && t - p.in_cta < a.T, kChkRowIndex)) return;
  clear_ring<kAlign, G>(ring, plan.stages * plan.stage_bytes, p);
  // a stage: the residual's rows, the branch's
  Stream<R, kAlign> residual;
  Stream<A, kAlign> y;
  uint32_t offset = 0;
  const uint32_t stage0 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  residual.template start<G>(stage0, &offset);
  if (branch) y.template start<G>(stage0, &offset);
  void* stretch = ring + plan.stages * plan.stage_bytes + p.warp * kStretch;
  const uint32_t accesses = plan.accesses;
  int64_t next = t;  // the row that is fetched next
  const auto fetch = [&](int stage) {
    if (next < a.T) {
      const uint32_t at = stage * plan.stage_bytes;
      residual.template fetch<G>(a.residual, next, at, access_of(accesses, kResidual), p);
      if (branch) y.template fetch<G>(a.branch, next, at, access_of(accesses, kBranch), p);
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
    // a row that the team does not have is computed like the others, of what the ring holds, and
    // not written
    Pairs v[kRows][G];
    float mean[kRows], root[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const uint32_t at = stage * plan.stage_bytes;
      if (++stage == plan.stages) stage = 0;
      float2 s = both(0.f);
#pragma unroll
      for (int k = 0; k < G; ++k) {
        Pairs& vk = v[j][k];
        residual.get(a.residual, t + j * step, at, k, vk);
        if (branch) {
          Pairs n;
          y.get(a.branch, t + j * step, at, k, n);
#pragma unroll
          for (int e = 0; e < 4; ++e) vk[e] = add(vk[e], n[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s = add(s, vk[e]);
      }
      mean[j] = s.x + s.y;
    }
    team_sum(mean, slots[turn][0], p);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      mean[j] *= inv_d;
      float2 s = both(0.f);
#pragma unroll
      for (int k = 0; k < G; ++k) {
        if (branch)
          put<R, kAlign>(a.residual_out, t + j * step, k, t + j * step < a.T,
                         access_of(accesses, kOut), p, stretch, v[j][k]);
        // columns past the row are no part of its spread
        const int left = p.d - 8 * (p.i + k * p.team);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2& x = v[j][k][e];
          x = add(x, both(-mean[j]));
          if (kAlign == kAligned ? left <= 0 : left <= 2 * e) x.x = 0.f;
          if (kAlign == kAligned ? left <= 0 : left <= 2 * e + 1) x.y = 0.f;
          s = fma(x, x, s);
        }
      }
      root[j] = s.x + s.y;
    }
    team_sum(root, slots[turn][1], p);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      root[j] = 1.f / sqrtf(__fmaf_rn(root[j], inv_d, a.eps));
      if (p.i == 0 && t + j * step < a.T && LP_CHECK(p.has(t + j * step), kChkRowIndex)) {
        if (a.mean != nullptr) a.mean[t + j * step] = mean[j];
        if (a.rstd != nullptr) a.rstd[t + j * step] = root[j];
      }
    }
#pragma unroll
    for (int k = 0; k < G; ++k) {
      Pairs w, b;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = both(1.f), b[e] = both(0.f);
      if (a.weight != nullptr) read_weight(a.weight, a.weight_bf16, k, wide_w, p, w);
      if (a.bias != nullptr) read_weight(a.bias, a.weight_bf16, k, wide_b, p, b);
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][k][e] = fma(mul(v[j][k][e], both(root[j])), w[e], b[e]);
        put<A, kAlign>(a.normed, t + j * step, k, t + j * step < a.T, access_of(accesses, kNormed),
                       p, stretch, v[j][k]);
      }
    }
  }
}

// ---- few bytes a column, aligned
//
// A thread has two or four groups of its row, fetched into registers a turn ahead, so that what a row costs beside
// its columns (sums, addresses) is spread over 16 or 32 of them; a team has a barrier of its own, so that rows wait for
// themselves alone; and one CTA an SM keeps weight and bias in shared memory, as float32 in the order of the
// reads.  (Read from L1 by every row, in 16-byte loads 32 bytes apart, they took 12 us of 8192 x 4096's 37.)

template <class T>
__device__ __forceinline__ void load_group(const T* p, Group<T>& g) {
  if constexpr (sizeof(T) == 2)
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(g.w[0]), "=r"(g.w[1]), "=r"(g.w[2]), "=r"(g.w[3])
                 : "l"(p));
  else
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(g.w[0]), "=r"(g.w[1]), "=r"(g.w[2]), "=r"(g.w[3]), "=r"(g.w[4]), "=r"(g.w[5]), "=r"(g.w[6]),
                   "=r"(g.w[7])
                 : "l"(p));
}
template <class T, int G>
struct Ahead {
  Group<T> g[G] = {};
  __device__ __forceinline__ void fetch(const Rows& r, int64_t t, const Place& p) {
    if (t >= p.rows) return;
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const int c = 8 * (p.i + k * p.team);
      if (c < p.d && LP_CHECK(p.has(t, c, 8), kChkCopyIndex)) load_group(row_at<const T, kAligned>(r, t, c), g[k]);
    }
  }
};

// A sum over a team of at most eight warps, as team_sum takes it and in its order, with a barrier of the team's own.
// slots: eight of the team, zeros where it has no warp; written again only after another barrier.
__device__ __forceinline__ float own_sum(float v, float (*slots)[8], const Place& p) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (p.team == 32) return v;
  if (p.lane == 0) (*slots)[p.warp - p.first_warp] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(p.in_cta + 1), "r"(p.team) : "memory");
  const float4 x = *reinterpret_cast<const float4*>(&(*slots)[0]), y = *reinterpret_cast<const float4*>(&(*slots)[4]);
  return ((x.x + y.x) + (x.z + y.z)) + ((x.y + y.y) + (x.w + y.w));
}

// 80 registers a thread, with four groups 128.
template <int G>
constexpr int kWideThreads = G <= 2 ? 768 : 512;
constexpr int kWideTeams = 15;  // named barriers

template <class R, class A, int G, bool kBranch>
__global__ void __launch_bounds__(kWideThreads<G>, 1)
    lp_layer_norm_wide_kernel(const __grid_constant__ LayerNormArgs a, const Plan plan) {
  __shared__ __align__(16) float slots[kWideTeams][2][2][8];
  extern __shared__ __align__(32) unsigned char ring[];
  const Place p(a.T, a.d, plan.shape);
  const float inv_d = 1.f / static_cast<float>(a.d);
  const int64_t step = int64_t(gridDim.x) * plan.shape.teams;
  int64_t t = int64_t(blockIdx.x) * plan.shape.teams + p.in_cta;
  if (!LP_CHECK(a.d <= a.residual.ld && t - p.in_cta < a.T, kChkRowIndex)) return;
  Ahead<R, G> residual;
  Ahead<A, kBranch ? G : 1> y;
  residual.fetch(a.residual, t, p);
  if constexpr (kBranch) y.fetch(a.branch, t, p);
  // weight and bias as a thread reads them: the first four columns of each group's weight, the others, the
  // bias's, so that a warp's accesses are of neighbours
  float4* const affine = reinterpret_cast<float4*>(ring);
  const int groups = G * p.team;
  for (int n = threadIdx.x; n < groups; n += blockDim.x) {
    Place q = p;
    q.i = n;
    Pairs w, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = both(1.f), b[e] = both(0.f);
    if (a.weight != nullptr) read_weight(a.weight, a.weight_bf16, 0, access_of(plan.accesses, kWeight) == kWide, q, w);
    if (a.bias != nullptr) read_weight(a.bias, a.weight_bf16, 0, access_of(plan.accesses, kBranchWeight) == kWide, q, b);
    affine[n] = make_float4(w[0].x, w[0].y, w[1].x, w[1].y);
    affine[n + groups] = make_float4(w[2].x, w[2].y, w[3].x, w[3].y);
    affine[n + 2 * groups] = make_float4(b[0].x, b[0].y, b[1].x, b[1].y);
    affine[n + 3 * groups] = make_float4(b[2].x, b[2].y, b[3].x, b[3].y);
  }
  if (p.team > 32)
    for (int n = threadIdx.x; n < int(sizeof(slots) / sizeof(float)); n += blockDim.x) (&slots[0][0][0][0])[n] = 0.f;
  __syncthreads();
  const int own = p.team > 32 ? p.in_cta : 0;
  for (int turn = 0; t < a.T; t += step, turn ^= 1) {
    Pairs v[G];
    float2 s = both(0.f);
#pragma unroll
    for (int k = 0; k < G; ++k) {
      unpack(residual.g[k], v[k]);
      if constexpr (kBranch) {
        Pairs n;
        unpack(y.g[k], n);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = add(v[k][e], n[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) s = add(s, v[k][e]);
    }
    residual.fetch(a.residual, t + step, p);
    if constexpr (kBranch) y.fetch(a.branch, t + step, p);
    const float mean = own_sum(s.x + s.y, &slots[own][turn][0], p) * inv_d;
    s = both(0.f);
#pragma unroll
    for (int k = 0; k < G; ++k) {
      if constexpr (kBranch)
        put<R, kAligned>(a.residual_out, t, k, true, access_of(plan.accesses, kOut), p, nullptr, v[k]);
      if (8 * (p.i + k * p.team) < p.d)  // columns past the row are no part of its spread
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[k][e] = add(v[k][e], both(-mean));
          s = fma(v[k][e], v[k][e], s);
        }
    }
    const float root = 1.f / sqrtf(__fmaf_rn(own_sum(s.x + s.y, &slots[own][turn][1], p), inv_d, a.eps));
    if (p.i == 0 && LP_CHECK(p.has(t), kChkRowIndex)) {
      if (a.mean != nullptr) a.mean[t] = mean;
      if (a.rstd != nullptr) a.rstd[t] = root;
    }
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const float4* at = affine + p.i + k * p.team;
      const float4 w0 = at[0], w1 = at[groups], b0 = at[2 * groups], b1 = at[3 * groups];
      const Pairs w = {{w0.x, w0.y}, {w0.z, w0.w}, {w1.x, w1.y}, {w1.z, w1.w}};
      const Pairs b = {{b0.x, b0.y}, {b0.z, b0.w}, {b1.x, b1.y}, {b1.z, b1.w}};
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k][e] = fma(mul(v[k][e], both(root)), w[e], b[e]);
      put<A, kAligned>(a.normed, t, k, true, access_of(plan.accesses, kNormed), p, nullptr, v[k]);
    }
  }
}

// One CTA an SM, of as many teams as take its rows in the fewest turns.
template <class R, class A, int G, bool kBranch>
lp_status launch_wide(const Device& dev, const LayerNormArgs& a, uint32_t accesses, cudaStream_t stream) {
  static PerContextOnce once;
  void (*const kernel)(LayerNormArgs, Plan) = lp_layer_norm_wide_kernel<R, A, G, kBranch>;
  if (!allow_ring(kernel, dev, &once)) return LP_ERR_CUDA;
  Plan plan{shape_of(a.d, G, a.T), accesses, 0, 0};
  const int team = plan.shape.team, fit = kWideThreads<G> / team;
  const int64_t most = team > 32 ? std::min(fit, kWideTeams) : fit, rows = (a.T + kSlots - 1) / kSlots;
  const int64_t turns = (rows + most - 1) / most;
  plan.shape.teams = int((rows + turns - 1) / turns);
  const int64_t all = (a.T + plan.shape.teams - 1) / plan.shape.teams;
  kernel<<<unsigned(std::min<int64_t>(all, kSlots)), team * plan.shape.teams, G * team * 64, stream>>>(a, plan);
  return launched();
}

// The CTAs of an SM have up to 1024 threads between them, each CTA with rows in flight of its own,
// and this much shared memory for them.
constexpr int kForwardBytes = 216 << 10;

template <int G>
lp_status launch_forward(const Device& dev, const LayerNormArgs& a, uint32_t accesses, Align align,
                         cudaStream_t stream) {
  return with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
    using R = decltype(r);
    using A = decltype(x);
    const auto launch = [&](auto* kernel, PerContextOnce* once) {
      if (!allow_ring(kernel, dev, once)) return LP_ERR_CUDA;
      Plan plan{shape_of(a.d, G, a.T), accesses, 1, 0};
      const int threads = plan.shape.team * plan.shape.teams;
      const int columns = int(sizeof(R)) + (a.branch.p ? int(sizeof(A)) : 0);
      const int least = stage_bytes_of(threads, G, columns, align != kAligned) * kRowsATurn<R, A, G> +
                        (align == kAligned ? 0 : threads / 32 * kStretch);
      const int ctas = std::max(1, std::min(1024 / threads, kForwardBytes / least));
      const int64_t all = (a.T + plan.shape.teams - 1) / plan.shape.teams;
      const int64_t blocks = std::min<int64_t>(all, kSlots * ctas);
      const int smem = plan_ring(&plan, columns, G, align != kAligned, (all + blocks - 1) / blocks,
                                 kRowsATurn<R, A, G>, kForwardBytes / ctas);
      kernel<<<unsigned(blocks), threads, smem, stream>>>(a, plan);
      return launched();
    };
    static PerContextOnce once[3];
    constexpr Align kLeast = sizeof(R) + sizeof(A) < 8 ? kByElements : kByWords;
    // aligned rows of bfloat16 of one or two groups are the wide kernel's
    if constexpr (sizeof(R) + sizeof(A) > 4 || G > 2)
      if (align == kAligned) return launch(lp_layer_norm_kernel<R, A, G, kAligned>, once);
    return align == kByWords ? launch(lp_layer_norm_kernel<R, A, G, kByWords>, once + 1)
                             : launch(lp_layer_norm_kernel<R, A, G, kLeast>, once + 2);
  });
}

template <int G>
lp_status launch_few_bytes(const Device& dev, const LayerNormArgs& a, uint32_t accesses, cudaStream_t stream) {
  if (a.branch.p != nullptr) return launch_wide<__nv_bfloat16, __nv_bfloat16, G, true>(dev, a, accesses, stream);
  return with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
    return launch_wide<decltype(r), decltype(x), G, false>(dev, a, accesses, stream);
  });
}

}  // namespace

lp_status launch_layer_norm(const Device& dev, const LayerNormArgs& a, cudaStream_t stream) {
  const uint32_t accesses = access_bits(kResidual, a.residual, a.residual_bf16) |
                            access_bits(kBranch, a.branch, a.act_bf16) |
                            access_bits(kWeight, a.weight, 0, a.weight_bf16) |
                            access_bits(kBranchWeight, a.bias, 0, a.weight_bf16) |
                            access_bits(kOut, a.residual_out, a.residual_bf16) |
                            access_bits(kNormed, a.normed, a.act_bf16);
  const bool fast = all_wide(accesses, {kResidual, kBranch, kOut, kNormed}, a.d) &&
                    near(a.residual) && near(a.branch) && near(a.residual_out) && near(a.normed);
  const Align align = fast                                                            ? kAligned
                      : any_halves(accesses, {kResidual, kBranch, kOut, kNormed}) ? kByElements
                                                                                      : kByWords;
  const int groups = groups_of(a.branch.p != nullptr, a.residual_bf16, a.act_bf16, a.d);
  if (fast && few_bytes(a.branch.p != nullptr, a.residual_bf16, a.act_bf16, a.d))
    return groups == 1   ? launch_few_bytes<1>(dev, a, accesses, stream)
           : groups == 2 ? launch_few_bytes<2>(dev, a, accesses, stream)
                         : launch_few_bytes<4>(dev, a, accesses, stream);
  return groups == 1   ? launch_forward<1>(dev, a, accesses, align, stream)
         : groups == 2 ? launch_forward<2>(dev, a, accesses, align, stream)
                       : launch_forward<4>(dev, a, accesses, align, stream);
}

cudaError_t take_check_word_layer_norm(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
