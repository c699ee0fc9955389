// lp_norm_backward.cu: the backward pass of the residual norm (include/lp_train.h).
//
// Bound by HBM (12 bytes a column in bfloat16) where a row has one sum: 8192 x 4096 takes 66 us,
// 6.1 TB/s.  With a normed branch (three sums) 4864 x 4096 takes 65 us of 35 at the copy rate and
// 8192 x 4096 101 of 59: a team of 16 warps owns a row, the sums over rows hold 24 of each thread's
// registers, so one team fits an SM, and all of it waits for the row's sums (the two-row kernels also
// spill 36 to 44 bytes a thread at 128 registers).  In float32 that is 45 us of 35 for 4864 x 2048.
// The sums over rows cost some 3 us a call, for the CTAs' partial sums and the second kernel: 512 x 4096
// takes 13 us of 4.  Two groups a thread spill 92 to 156 bytes with a normed branch: 4096 x 7168 takes
// 77 us of 52 without one, 127 with it.  From 8193 columns on the row is read twice, a column a thread at
// a time: 4096 x 12288 takes 514 us of 89.  History at 8192 x 4096: sums in shared memory 1083 us, rows
// and sums in registers 158, with the ring and kept addresses 100, two rows a turn 69, two columns an
// instruction 66.  A row's second pass beside the next row's first one gained only with a normed branch
// of 4096 (59 us) and lost elsewhere (4864 x 2400: 58 us instead of 50).  lp_norm.cuh says how rows lie
// over threads and come on chip.
#include <type_traits>

#include "lp_norm.cuh"

namespace lp {
namespace {

// Floats from one sum of a CTA to the next in the workspace: whole groups.
__host__ __device__ __forceinline__ int64_t pitch_of(int64_t d) { return (d + 7) / 8 * 8; }

// d up to kTeamDim: a CTA takes rows in turn and keeps its share of the sums over rows
// (grad_weight, grad_branch_weight, a one-row gate's gradient) in registers.
//
// One round of sums a row: with e = b g w_b yh the second mean is linear in the first,
//   mean(e D) = mean(e (dr' + rstd dx)) - mean(dx x) mean(e rstd x),
// so the three sums are taken together.
//
// Where the registers and the ring allow, a team that has more than one row takes two a turn: their
// waits for the team are one, and the work of one hides the latencies of the other.  A team's only
// row is taken alone, 1.1 us less for one row of 4096 with a normed branch, and 1216 of 512 in 7.7 us
// instead of 8.5.
template <class R, class A, int G>
constexpr int kRowsATurn = G == 1 && sizeof(R) + sizeof(A) <= 6 ? 2 : 1;

// kSolo: the CTA is one team, so that a turn's first row is there without asking.
template <class R, class A, int G, int kRows, bool kPost, int kAlign, bool kSolo>
__global__ void __launch_bounds__(kMaxTeam)
    lp_residual_norm_grad_kernel(const __grid_constant__ NormGradArgs a, const Plan plan) {
  constexpr int kSums = kPost ? 3 : 1;
  __shared__ __align__(16) float slots[2][kMaxWarps][padded(kRows * kSums)];
  extern __shared__ __align__(32) unsigned char ring[];
  const Place p(a.T, a.d, plan.shape);
  const float inv_d = 1.f / static_cast<float>(a.d);
  const bool norm = a.weight != nullptr, branch = a.branch.p != nullptr, gate = a.gate.p != nullptr;
  const bool has_dr = a.grad_residual_out.p != nullptr;
  const bool gate_sum = gate && a.gate.ld == 0 && a.grad_gate.p != nullptr;
  Pairs sum_w[G] = {}, sum_b[G] = {}, sum_g[G] = {};
  const int64_t step = int64_t(gridDim.x) * plan.shape.teams;
  int64_t t = int64_t(blockIdx.x) * plan.shape.teams + p.in_cta;
  if (!LP_CHECK(a.d <= a.grad_residual.ld && t - p.in_cta < a.T, kChkRowIndex)) return;
  clear_ring<kAlign, G>(ring, plan.stages * plan.stage_bytes, p);
  // a stage: the rows of the stream, its gradient, the norm's gradient, the branch, the gate
  Stream<R, kAlign> s, dr;
  Stream<A, kAlign> dh, y, g;
  uint32_t offset = 0;
  const uint32_t stage0 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  if (norm) s.template start<G>(stage0, &offset);
  if (has_dr) dr.template start<G>(stage0, &offset);
  if (norm) dh.template start<G>(stage0, &offset);
  if (branch) y.template start<G>(stage0, &offset);
  if (gate) g.template start<G>(stage0, &offset);
  const bool write_gate = gate && a.gate.ld != 0 && a.grad_gate.p != nullptr;
  void* stretch = ring + plan.stages * plan.stage_bytes + p.warp * kStretch;
  const uint32_t accesses = plan.accesses;
  int64_t next = t;  // the row that is fetched next
  const auto fetch = [&](int stage) {
    const uint32_t at = stage * plan.stage_bytes;
    if (next < a.T) {
      if (norm) {
        s.template fetch<G>(a.residual_out, next, at, access_of(accesses, kOut), p);
        dh.template fetch<G>(a.grad_normed, next, at, access_of(accesses, kGradNormed), p);
      }
      if (has_dr)
        dr.template fetch<G>(a.grad_residual_out, next, at, access_of(accesses, kGradOut), p);
      if (branch) y.template fetch<G>(a.branch, next, at, access_of(accesses, kBranch), p);
      if (gate) g.template fetch<G>(a.gate, next, at, access_of(accesses, kGate), p);
    } else {
      if (norm) s.template zero<G>(at), dh.template zero<G>(at);
      if (has_dr) dr.template zero<G>(at);
      if (branch) y.template zero<G>(at);
      if (gate) g.template zero<G>(at);
    }
    next += step;
    commit_copies();
  };
  for (int n = 0; n + kRows < plan.stages; ++n) fetch(n);
  const bool wide_w = access_of(accesses, kWeight) == kWide;
  const bool wide_b = access_of(accesses, kBranchWeight) == kWide;
  // the weights stay in registers where these allow: without a norm of the branch, or with one row
  // a turn
  constexpr bool kKeep = G == 1 && (!kPost || kRows == 1);
  Pairs kept_w, kept_b;
  if (kKeep && norm) read_weight(a.weight, a.weight_bf16, 0, wide_w, p, kept_w);
  if (kKeep && kPost) read_weight(a.branch_weight, a.weight_bf16, 0, wide_b, p, kept_b);
  // the rows' roots, loaded a turn ahead
  float root[kRows], root_y[kRows];
  const auto load_roots = [&](int64_t first) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const bool mine = first + j * step < a.T && LP_CHECK(p.has(first + j * step), kChkRowIndex);
      root[j] = norm && mine ? a.rstd[first + j * step] : 0.f;
      root_y[j] = kPost && mine ? a.branch_rstd[first + j * step] : 1.f;
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
    Pairs x[kRows][G], D[kRows][G];
    float m[kRows * kSums];
    float2 sums[kRows][kSums];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int q = 0; q < kSums; ++q) sums[j][q] = both(0.f);
#pragma unroll
    for (int k = 0; k < G; ++k) {
      Pairs w, wb;
      if (norm && !kKeep) read_weight(a.weight, a.weight_bf16, k, wide_w, p, w);
      if (kPost) {
        if (!kKeep) read_weight(a.branch_weight, a.weight_bf16, k, wide_b, p, wb);
#pragma unroll
        for (int e = 0; e < 4; ++e) wb[e] = mul(both(a.branch_scale), kKeep ? kept_b[e] : wb[e]);
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        Pairs& xk = x[j][k];
        Pairs& Dk = D[j][k];
        if (has_dr) {
          dr.get(a.grad_residual_out, t + j * step, at[j], k, Dk);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) Dk[e] = both(0.f);
        }
        if (norm) {
          Pairs h;
          s.get(a.residual_out, t + j * step, at[j], k, xk);
          dh.get(a.grad_normed, t + j * step, at[j], k, h);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 dx = mul(h[e], kKeep ? kept_w[e] : w[e]);
            xk[e] = mul(xk[e], both(root[j]));
            sums[j][0] = fma(dx, xk[e], sums[j][0]);
            sum_w[k][e] = fma(h[e], xk[e], sum_w[k][e]);
            Dk[e] = fma(both(root[j]), dx, Dk[e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) xk[e] = both(0.f);
        }
        if (kPost) {
          Pairs f;
          y.get(a.branch, t + j * step, at[j], k, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = mul(mul(f[e], both(root_y[j])), wb[e]);
          if (gate) {
            Pairs by;
            g.get(a.gate, t + j * step, at[j], k, by);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = mul(f[e], by[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sums[j][1 % kSums] = fma(f[e], Dk[e], sums[j][1 % kSums]);
            sums[j][2 % kSums] = fma(f[e], xk[e], sums[j][2 % kSums]);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int q = 0; q < kSums; ++q) m[j * kSums + q] = sums[j][q].x + sums[j][q].y;
    if (norm || kPost) team_sum(m, slots[turn], p);
    float m1[kRows], m2[kRows], scale_y[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      m1[j] = root[j] * (m[j * kSums] * inv_d);  // rstd mean(dx x)
      // mean(e D)
      m2[j] = kPost ? __fmaf_rn(-m1[j], m[j * kSums + 2 % kSums], m[j * kSums + 1 % kSums]) * inv_d : 0.f;
      scale_y[j] = root_y[j];
    }
    load_roots(t + kRows * step);
#pragma unroll
    for (int k = 0; k < G; ++k) {
      Pairs wb;
      if (kPost && !kKeep) read_weight(a.branch_weight, a.weight_bf16, k, wide_b, p, wb);
      if (kPost && kKeep)
#pragma unroll
        for (int e = 0; e < 4; ++e) wb[e] = kept_b[e];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const bool mine = (kSolo && j == 0) || t + j * step < a.T;
        Pairs& Dk = D[j][k];
        Pairs out;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          Dk[e] = fma(both(-m1[j]), x[j][k][e], Dk[e]);
          out[e] = mul(both(a.residual_scale), Dk[e]);
        }
        put<R, kAlign>(a.grad_residual, t + j * step, k, mine, access_of(accesses, kGradResidual), p,
                      stretch, out);
        if (!branch) continue;
        Pairs yh;
        if (kPost || gate) {
          y.get(a.branch, t + j * step, at[j], k, yh);
          if (kPost)
#pragma unroll
            for (int e = 0; e < 4; ++e) yh[e] = mul(yh[e], both(scale_y[j]));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = mul(both(a.branch_scale), Dk[e]);
        if (gate) {
          Pairs f, dg;
          g.get(a.gate, t + j * step, at[j], k, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dg[e] = kPost ? mul(yh[e], wb[e]) : yh[e];
            if (gate_sum) sum_g[k][e] = fma(out[e], dg[e], sum_g[k][e]);
            dg[e] = mul(out[e], dg[e]);
            out[e] = mul(out[e], f[e]);
          }
          if (write_gate)
            put<A, kAlign>(a.grad_gate, t + j * step, k, mine, access_of(accesses, kGradGate), p,
                          stretch, dg);
        }
        if (kPost) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sum_b[k][e] = fma(out[e], yh[e], sum_b[k][e]);
            out[e] = mul(both(scale_y[j]), fma(out[e], wb[e], mul(yh[e], both(-m2[j]))));
          }
        }
        put<A, kAlign>(a.grad_branch, t + j * step, k, mine, access_of(accesses, kGradBranch), p,
                      stretch, out);
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.partials == nullptr) return;
  // the teams' sums in order, then the CTA's: three rows of whole groups in the workspace, or of a
  // lone CTA the sums themselves
  float2* shared = reinterpret_cast<float2*>(ring);  // all copies have been waited for
  float* part = a.partials + int64_t(blockIdx.x) * 3 * pitch_of(a.d);
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    Pairs(&sum)[G] = q == 0 ? sum_w : q == 1 ? sum_b : sum_g;
    if (q == 0 ? a.grad_weight == nullptr : q == 1 ? a.grad_branch_weight == nullptr : !gate_sum)
      continue;
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
          for (int e = 0; e < 4; ++e) {
            const float2 other = shared[(k * p.team + p.i) * 4 + e];
            sum[k][e] = make_float2(sum[k][e].x + other.x, sum[k][e].y + other.y);
          }
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
        float* out = q == 0   ? a.grad_weight
                     : q == 1 ? a.grad_branch_weight
                              : static_cast<float*>(a.grad_gate.p);
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

// Backward of rows wider than that: the row is read twice (the second time from L2) and the
// sums over rows lie in shared memory, where each column has one owner.  4096 x 12288 bfloat16 takes
// 514 us, 647 with a normed branch, of 89 at the copy rate: loads of 2 and 4 bytes, weights from L2 at
// every row, one CTA an SM (issue slots 30%, DRAM 13% busy).
constexpr int kWideThreads = 1024;

template <class T>
__device__ __forceinline__ T* row_of(const Rows& r, int64_t t) {
  return static_cast<T*>(r.p) + t * r.ld;
}
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

// Three sums over the CTA, the same bits for all threads.
__device__ __forceinline__ void wide_sum(float (&v)[3], float (*slots)[3]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < 3; ++k) slots[threadIdx.x / 32][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) v[k] = slots[threadIdx.x & 31][k];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}

template <class R, class A>
__global__ void __launch_bounds__(kWideThreads)
    lp_residual_norm_grad_wide_kernel(const __grid_constant__ NormGradArgs a) {
  extern __shared__ float sums[];
  __shared__ float slots[2][kWideThreads / 32][3];
  const int64_t d = a.d;
  const float inv_d = 1.f / static_cast<float>(d);
  const bool post = a.branch_weight != nullptr, norm = a.weight != nullptr;
  for (int64_t c = threadIdx.x; c < d; c += kWideThreads)
    sums[c] = sums[d + c] = sums[2 * d + c] = 0.f;
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    // every operand's row has d columns (a one-row gate's pitch is 0)
    if (!LP_CHECK(t >= 0 && d <= kNormMaxDim && d <= a.grad_residual.ld && (!norm || d <= a.residual_out.ld) &&
                      (a.branch.p == nullptr || (d <= a.branch.ld && d <= a.grad_branch.ld)),
                  kChkRowIndex))
      break;
    const R* s = norm ? row_of<const R>(a.residual_out, t) : nullptr;
    const A* y = a.branch.p ? row_of<const A>(a.branch, t) : nullptr;
    const A* g = a.gate.p ? row_of<const A>(a.gate, t) : nullptr;
    const A* dh = norm ? row_of<const A>(a.grad_normed, t) : nullptr;
    const R* dr = a.grad_residual_out.p ? row_of<const R>(a.grad_residual_out, t) : nullptr;
    const float root = norm ? a.rstd[t] : 0.f, root_y = post ? a.branch_rstd[t] : 1.f;
    float m[3] = {0.f, 0.f, 0.f};
    for (int64_t c = threadIdx.x; c < d; c += kWideThreads) {
      const float x = norm ? get(s, c) * root : 0.f;
      const float dx = norm ? get(dh, c) * weight_at(a.weight, a.weight_bf16, c) : 0.f;
      m[0] += dx * x;
      if (post) {
        float f = a.branch_scale * weight_at(a.branch_weight, a.weight_bf16, c);
        if (g != nullptr) f *= get(g, c);
        f *= get(y, c) * root_y;
        m[1] += f * ((dr != nullptr ? get(dr, c) : 0.f) + root * dx);
        m[2] += f * (root * x);
      }
    }
    if (norm || post) wide_sum(m, slots[turn]);
    const float m1 = m[0] * inv_d, m2 = (m[1] - m1 * m[2]) * inv_d;
    for (int64_t c = threadIdx.x; c < d; c += kWideThreads) {
      float D = dr != nullptr ? get(dr, c) : 0.f;
      if (norm) {
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
        if (a.gate.ld == 0)
          sums[2 * d + c] += dg;
        else if (a.grad_gate.p != nullptr)
          put(row_of<A>(a.grad_gate, t), c, dg);
        dn *= get(g, c);
      }
      if (post) {
        sums[d + c] += dn * yh;
        dn = root_y * (dn * wb - yh * m2);
      }
      put(row_of<A>(a.grad_branch, t), c, dn);
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.partials == nullptr) return;
  float* part = a.partials + int64_t(blockIdx.x) * 3 * pitch_of(d);
  for (int64_t c = threadIdx.x; c < d; c += kWideThreads)
#pragma unroll
    for (int q = 0; q < 3; ++q)
      if (LP_CHECK(c < pitch_of(d), kChkSplitIndex)) part[q * pitch_of(d) + c] = sums[q * d + c];
}

// The CTAs' partial sums: 16 threads a column take every sixteenth part in order, and their
// sums are added in order.
constexpr int kSumLanes = 16;
__global__ void __launch_bounds__(32 * kSumLanes)
    lp_norm_sum_kernel(const float* partials, int64_t parts, int64_t d, float* grad_weight,
                       float* grad_branch_weight, float* grad_gate) {
  __shared__ float slots[kSumLanes][32];
  float* const out = blockIdx.y == 0 ? grad_weight : blockIdx.y == 1 ? grad_branch_weight : grad_gate;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, from = threadIdx.x / 32;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane, pitch = pitch_of(d);
  // launched as a programmatic dependent of the row kernel: wait for its partial sums
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.f;
  if (c < d) {
    const float* p = partials + (int64_t(from) * 3 + blockIdx.y) * pitch + c;
#pragma unroll 4
    for (int64_t k = from; k < parts; k += kSumLanes, p += 3 * kSumLanes * pitch)
      if (LP_CHECK(p >= partials && p < partials + parts * 3 * pitch, kChkSplitIndex)) s += __ldcg(p);
  }
  slots[from][lane] = s;
  __syncthreads();
  if (from != 0 || c >= d) return;
#pragma unroll
  for (int k = 1; k < kSumLanes; ++k) s += slots[k][lane];
  out[c] = s;
}

// The rows that the CTAs take at once, and how many CTAs there are.
constexpr int64_t kTeamDim = kMaxTeam * 8 * 2;  // the widest row of the team kernel
int groups_of(int64_t d) { return d <= kTeamDim / 2 ? 1 : 2; }
// CTAs of an SM: two where a row takes no more than half of its threads.
int ctas_of_sm(int threads) { return threads <= kMaxTeam / 2 ? 2 : 1; }
int64_t backward_blocks(int64_t T, int64_t d) {
  if (d > kTeamDim) return std::min(T, kSlots);
  const Shape s = shape_of(d, groups_of(d), T);
  return std::min((T + s.teams - 1) / s.teams, kSlots * ctas_of_sm(s.team * s.teams));
}

template <int G>
lp_status launch_backward(const Device& dev, const NormGradArgs& a, uint32_t accesses, Align align,
                          int64_t blocks, cudaStream_t stream) {
  return with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
    using R = decltype(r);
    using A = decltype(x);
    constexpr int kMost = kRowsATurn<R, A, G>;
    Plan plan{shape_of(a.d, G, a.T), accesses, 1, 0};
    const int64_t at_once = blocks * plan.shape.teams, rows = (a.T + at_once - 1) / at_once;
    const auto launch = [&](auto* kernel, int least, PerContextOnce* once) {
      if (!allow_ring(kernel, dev, once)) return LP_ERR_CUDA;
      const int columns = (a.weight ? int(sizeof(R) + sizeof(A)) : 0) +
                          (a.grad_residual_out.p ? int(sizeof(R)) : 0) +
                          (a.branch.p ? int(sizeof(A)) : 0) + (a.gate.p ? int(sizeof(A)) : 0);
      int smem = plan_ring(&plan, columns, G, align != kAligned, rows, least,
                           kRingBytes / ctas_of_sm(plan.shape.team * plan.shape.teams));
      if (plan.shape.teams > 1) smem = std::max(smem, plan.shape.team * G * 8 * int(sizeof(float)));
      kernel<<<unsigned(blocks), plan.shape.team * plan.shape.teams, smem, stream>>>(a, plan);
      return launched();
    };
    static PerContextOnce once[10];
    const bool solo = plan.shape.teams == 1;
    const auto with_post = [&](auto post_, PerContextOnce* once) {
      constexpr bool kPost = decltype(post_)::value;
      constexpr Align kLeast = sizeof(R) + sizeof(A) < 8 ? kShifted : kByWords;
      if (align == kByWords)
        return launch(lp_residual_norm_grad_kernel<R, A, G, 1, kPost, kByWords, false>, 1, once);
      if (align == kShifted)
        return launch(lp_residual_norm_grad_kernel<R, A, G, 1, kPost, kLeast, false>, 1, once + 1);
      if constexpr (kMost > 1)
        if (rows == 1)
          return launch(lp_residual_norm_grad_kernel<R, A, G, 1, kPost, kAligned, false>, 1, once + 2);
      return solo
                 ? launch(lp_residual_norm_grad_kernel<R, A, G, kMost, kPost, kAligned, true>, kMost, once + 3)
                 : launch(lp_residual_norm_grad_kernel<R, A, G, kMost, kPost, kAligned, false>, kMost,
                          once + 4);
    };
    return a.branch_weight != nullptr ? with_post(std::true_type(), once)
                                      : with_post(std::false_type(), once + 5);
  });
}

lp_status launch_backward_wide(const Device& dev, const NormGradArgs& a, int64_t blocks,
                               cudaStream_t stream) {
  return with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
    auto* kernel = lp_residual_norm_grad_wide_kernel<decltype(r), decltype(x)>;
    static PerContextOnce once;
    if (once.run(dev.ctx_id, [&] {
          return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      int(kNormMaxDim * 12));
        }) != cudaSuccess)
      return LP_ERR_CUDA;
    kernel<<<unsigned(blocks), kWideThreads, size_t(a.d) * 12, stream>>>(a);
    return launched();
  });
}

}  // namespace

size_t residual_norm_backward_workspace(int64_t T, int64_t d) {
  return static_cast<size_t>(std::max<int64_t>(1, backward_blocks(std::max<int64_t>(T, 1), d)) * 3 *
                             pitch_of(d) * 4);
}

lp_status launch_residual_norm_backward(const Device& dev, const NormGradArgs& a,
                                        cudaStream_t stream) {
  const int64_t blocks = a.T > 0 ? backward_blocks(a.T, a.d) : 0;
  if (blocks > 0) {
    const uint32_t accesses = access_bits(kOut, a.residual_out, a.residual_bf16) |
                              access_bits(kBranch, a.branch, a.act_bf16) |
                              access_bits(kGate, a.gate, a.act_bf16) |
                              access_bits(kBranchWeight, a.branch_weight, 0, a.weight_bf16) |
                              access_bits(kWeight, a.weight, 0, a.weight_bf16) |
                              access_bits(kGradNormed, a.grad_normed, a.act_bf16) |
                              access_bits(kGradOut, a.grad_residual_out, a.residual_bf16) |
                              access_bits(kGradResidual, a.grad_residual, a.residual_bf16) |
                              access_bits(kGradBranch, a.grad_branch, a.act_bf16) |
                              access_bits(kGradGate, a.grad_gate, a.act_bf16);
    const bool fast = all_wide(accesses,
                               {kOut, kBranch, kGate, kGradNormed, kGradOut, kGradResidual, kGradBranch,
                                kGradGate},
                               a.d) &&
                      near(a.residual_out) && near(a.branch) && near(a.gate) && near(a.grad_normed) &&
                      near(a.grad_residual_out) && near(a.grad_residual) && near(a.grad_branch) &&
                      near(a.grad_gate);
    const Align align =
        fast ? kAligned
        : any_halves(accesses, {kOut, kBranch, kGate, kGradNormed, kGradOut, kGradResidual, kGradBranch, kGradGate})
            ? kShifted
            : kByWords;
    const lp_status st = a.d > kTeamDim        ? launch_backward_wide(dev, a, blocks, stream)
                         : groups_of(a.d) == 1 ? launch_backward<1>(dev, a, accesses, align, blocks, stream)
                                               : launch_backward<2>(dev, a, accesses, align, blocks, stream);
    if (st != LP_OK) return st;
  }
  float* gate_sum = a.gate.ld == 0 ? static_cast<float*>(a.grad_gate.p) : nullptr;
  if (a.grad_weight == nullptr && a.grad_branch_weight == nullptr && gate_sum == nullptr)
    return LP_OK;
  if (blocks == 1 && a.d <= kTeamDim) return LP_OK;  // the CTA wrote them
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.d + 31) / 32), 3);
  cfg.blockDim = dim3(32 * kSumLanes);
  cfg.stream = stream;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl;
  cfg.numAttrs = blocks > 0 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, lp_norm_sum_kernel, static_cast<const float*>(a.partials), blocks, a.d,
                         a.grad_weight, a.grad_branch_weight, gate_sum) != cudaSuccess)
    return LP_ERR_CUDA;
  return launched();
}

cudaError_t take_check_word_norm_backward(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
