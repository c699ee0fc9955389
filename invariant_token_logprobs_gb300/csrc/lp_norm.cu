// lp_norm.cu: the residual norm and its backward pass (include/lp_train.h).
//
// Both are bound by the bytes of their row operands, so a row is read once and held
// in registers.  A row belongs to a team of whole warps; thread i of a team of n owns
// the groups of 8 columns i, i + n, i + 2n, ... of the row, which is 16 bytes of
// bfloat16 or 32 of float32 an access.  The team's size and the groups a thread holds
// depend on d alone, so a row's sums are taken in the same order whatever the batch.
// Rows that are not aligned for such accesses go through a warp's stretch of shared
// memory, 32 neighbouring elements an access: same owners, same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "lp_check.cuh"
#include "lp_train_internal.h"

namespace lp {
namespace {

constexpr int kMaxTeam = 512;  // threads of a row, and of a CTA
constexpr int kMaxWarps = kMaxTeam / 32;
// The backward's row slots: one CTA per SM of a GB300.  Fixed, so that the order in
// which rows are summed does not depend on the device's partition.
constexpr int64_t kSlots = 152;

// 8 columns as they lie in memory.
template <class T>
struct __align__(8 * sizeof(T)) Group {
  uint32_t w[2 * sizeof(T)];
};
using Group16 = Group<__nv_bfloat16>;
using Group32 = Group<float>;

__device__ __forceinline__ Group16 load_group(const __nv_bfloat16* p) {
  Group16 g;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(g.w[0]), "=r"(g.w[1]), "=r"(g.w[2]), "=r"(g.w[3])
               : "l"(p)
               : "memory");
  return g;
}
__device__ __forceinline__ Group32 load_group(const float* p) {
  Group32 g;
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(g.w[0]), "=r"(g.w[1]), "=r"(g.w[2]), "=r"(g.w[3]), "=r"(g.w[4]), "=r"(g.w[5]),
                 "=r"(g.w[6]), "=r"(g.w[7])
               : "l"(p)
               : "memory");
  return g;
}
__device__ __forceinline__ void store_group(__nv_bfloat16* p, const Group16& g) {
  asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(g.w[0]), "r"(g.w[1]),
               "r"(g.w[2]), "r"(g.w[3])
               : "memory");
}
__device__ __forceinline__ void store_group(float* p, const Group32& g) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(g.w[0]),
               "r"(g.w[1]), "r"(g.w[2]), "r"(g.w[3]), "r"(g.w[4]), "r"(g.w[5]), "r"(g.w[6]),
               "r"(g.w[7])
               : "memory");
}

__device__ __forceinline__ float element(const Group32& g, int i) { return __uint_as_float(g.w[i]); }
__device__ __forceinline__ float element(const Group16& g, int i) {
  return __uint_as_float(i & 1 ? g.w[i / 2] & 0xffff0000u : g.w[i / 2] << 16);
}
__device__ __forceinline__ Group32 pack(const float (&v)[8], float) {
  Group32 g;
#pragma unroll
  for (int i = 0; i < 8; ++i) g.w[i] = __float_as_uint(v[i]);
  return g;
}
__device__ __forceinline__ Group16 pack(const float (&v)[8], __nv_bfloat16) {
  Group16 g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    g.w[i] = *reinterpret_cast<const uint32_t*>(&two);
  }
  return g;
}

// A thread's place in its row: its first column, and its warp's shared stretch of 256
// elements for rows that are not aligned.
struct Place {
  int64_t d;  // the row's columns; 0 for a team without a row
  int lane;
  void* stretch;
};

// Group `index` of a row; columns past the row are zero.  All threads of a warp call this
// together, with consecutive indexes.
template <class T>
__device__ __forceinline__ Group<T> read_group(const T* row, int64_t index, bool wide,
                                               const Place& p) {
  Group<T> g{};
  const int64_t c = 8 * index;
  if (wide) {
    if (c + 8 <= p.d) return load_group(row + c);
    T* e = reinterpret_cast<T*>(&g);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < p.d) e[i] = row[c + i];
    return g;
  }
  T* s = static_cast<T*>(p.stretch);
  const int64_t first = c - 8 * p.lane;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t k = first + 32 * i + p.lane;
    s[32 * i + p.lane] = k < p.d ? row[k] : T(0.f);
  }
  __syncwarp();
  return reinterpret_cast<const Group<T>*>(s)[p.lane];
}
template <class T>
__device__ __forceinline__ void write_group(T* row, int64_t index, bool wide, const Place& p,
                                            const Group<T>& g) {
  const int64_t c = 8 * index;
  if (wide) {
    if (c + 8 <= p.d) return store_group(row + c, g);
    const T* e = reinterpret_cast<const T*>(&g);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < p.d) row[c + i] = e[i];
    return;
  }
  T* s = static_cast<T*>(p.stretch);
  const int64_t first = c - 8 * p.lane;
  __syncwarp();
  reinterpret_cast<Group<T>*>(s)[p.lane] = g;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t k = first + 32 * i + p.lane;
    if (k < p.d) row[k] = s[32 * i + p.lane];
  }
}
// The same for a weight vector, of a type known at run time.  It is read again by every
// row, so it may stay in L1.
__device__ __forceinline__ void read_weight(const void* w, bool bf16, int64_t index, bool wide,
                                            const Place& p, float (&v)[8]) {
  if (wide && 8 * index + 8 <= p.d) {
    if (bf16) {
      const uint4 x = __ldg(static_cast<const uint4*>(w) + index);
      const Group16 g{{x.x, x.y, x.z, x.w}};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = element(g, i);
    } else {
      const float4 a = __ldg(static_cast<const float4*>(w) + 2 * index);
      const float4 b = __ldg(static_cast<const float4*>(w) + 2 * index + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t c = 8 * index + i;
    v[i] = c >= p.d ? 0.f
           : bf16   ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c])
                    : static_cast<const float*>(w)[c];
  }
}

template <class T>
__device__ __forceinline__ T* row_of(const Rows& r, int64_t t) {
  return static_cast<T*>(r.p) + t * r.ld;
}

// Bits of the operands whose rows are aligned for whole groups.
enum : uint32_t {
  kWideResidual = 1u, kWideBranch = 2u, kWideGate = 4u, kWideBranchWeight = 8u, kWideWeight = 16u,
  kWideOut = 32u, kWideNormed = 64u, kWideGradNormed = 128u, kWideGradOut = 256u,
  kWideGradResidual = 512u, kWideGradBranch = 1024u, kWideGradGate = 2048u,
};
uint32_t wide(uint32_t bit, const void* p, int64_t ld, bool bf16) {
  const uintptr_t size = bf16 ? 2 : 4, group = 8 * size;
  return reinterpret_cast<uintptr_t>(p) % group == 0 &&
                 (static_cast<uintptr_t>(ld) * size) % group == 0
             ? bit
             : 0u;
}

// How rows of d columns are laid over threads.
struct Shape {
  int team;   // threads of a row
  int teams;  // rows of a CTA at once
};
Shape shape_of(int64_t d, int groups_per_thread, int64_t T) {
  const int64_t groups = (d + 7) / 8;
  Shape s;
  s.team = int((groups + 32 * groups_per_thread - 1) / (32 * groups_per_thread)) * 32;
  s.teams = int(std::max<int64_t>(1, std::min<int64_t>(256 / s.team, T)));
  return s;
}

// N sums over a team at once, the same bits for all its threads: shuffles, then the warps'
// sums in order.  `slots` is used by one call between two barriers.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*slots)[N], int team, int warp,
                                         int first_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (team == 32) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) slots[warp][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
  for (int w = 0; w < team / 32; ++w)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += slots[first_warp + w][k];
}

// Forward: one row a team, G groups a thread.
template <class R, class A, int G>
__global__ void __launch_bounds__(kMaxTeam)
    lp_residual_norm_kernel(const __grid_constant__ NormArgs a, Shape shape, uint32_t aligned) {
  __shared__ float slots[2][kMaxWarps][1];
  extern __shared__ __align__(32) unsigned char stretches[];
  const int warp = threadIdx.x / 32, in_cta = threadIdx.x / shape.team;
  const int i = threadIdx.x - in_cta * shape.team, first_warp = in_cta * (shape.team / 32);
  int64_t t = int64_t(blockIdx.x) * shape.teams + in_cta;
  Place p{t < a.T ? a.d : 0, int(threadIdx.x & 31), stretches + warp * 256 * sizeof(float)};
  if (t >= a.T) t = 0;
  const float inv_d = 1.f / static_cast<float>(a.d);
  Group<R> r[G];
  Group<A> y[G], g[G];
#pragma unroll
  for (int k = 0; k < G; ++k) {
    const int64_t index = i + k * shape.team;
    r[k] = read_group(row_of<const R>(a.residual, t), index, aligned & kWideResidual, p);
    if (a.branch.p) y[k] = read_group(row_of<const A>(a.branch, t), index, aligned & kWideBranch, p);
    if (a.gate.p) g[k] = read_group(row_of<const A>(a.gate, t), index, aligned & kWideGate, p);
  }
  float root_y[1] = {0.f};
  if (a.branch_weight != nullptr) {
#pragma unroll
    for (int k = 0; k < G; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) root_y[0] += element(y[k], e) * element(y[k], e);
    team_sum(root_y, slots[0], shape.team, warp, first_warp);
    root_y[0] = 1.f / sqrtf(root_y[0] * inv_d + a.eps);
    if (a.branch_rstd != nullptr && i == 0 && p.d > 0) a.branch_rstd[t] = root_y[0];
  }
  float v[G][8], root[1] = {0.f};
#pragma unroll
  for (int k = 0; k < G; ++k) {
    const int64_t index = i + k * shape.team;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[k][e] = element(r[k], e);
    if (a.branch.p) {
      float n[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = element(y[k], e);
      if (a.branch_weight != nullptr) {
        float w[8];
        read_weight(a.branch_weight, a.weight_bf16, index, aligned & kWideBranchWeight, p, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = n[e] * root_y[0] * w[e];
      }
      if (a.gate.p)
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] *= element(g[k], e);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = a.residual_scale * v[k][e] + a.branch_scale * n[e];
      write_group(row_of<R>(a.residual_out, t), index, aligned & kWideOut, p, pack(v[k], R()));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) root[0] += v[k][e] * v[k][e];
  }
  if (a.weight == nullptr) return;
  team_sum(root, slots[1], shape.team, warp, first_warp);
  root[0] = 1.f / sqrtf(root[0] * inv_d + a.eps);
  if (a.rstd != nullptr && i == 0 && p.d > 0) a.rstd[t] = root[0];
#pragma unroll
  for (int k = 0; k < G; ++k) {
    const int64_t index = i + k * shape.team;
    float w[8];
    read_weight(a.weight, a.weight_bf16, index, aligned & kWideWeight, p, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = v[k][e] * root[0] * w[e];
    write_group(row_of<A>(a.normed, t), index, aligned & kWideNormed, p, pack(w, A()));
  }
}

// Backward, d up to kMaxTeam * 8 * 2: a CTA takes rows in turn and keeps its share of the
// sums over rows (grad_weight, grad_branch_weight, a one-row gate's gradient) in registers.
//
// One round of sums a row: with e = b g w_b yh the second mean is linear in the first,
//   mean(e D) = mean(e (dr' + rstd dx)) - mean(dx x) mean(e rstd x),
// so the three sums are taken together.
template <class R, class A, int G>
__global__ void __launch_bounds__(kMaxTeam)
    lp_residual_norm_grad_kernel(const __grid_constant__ NormGradArgs a, Shape shape,
                                 uint32_t aligned) {
  __shared__ float slots[2][kMaxWarps][3];
  extern __shared__ __align__(32) unsigned char stretches[];
  const int warp = threadIdx.x / 32, in_cta = threadIdx.x / shape.team;
  const int i = threadIdx.x - in_cta * shape.team, first_warp = in_cta * (shape.team / 32);
  const float inv_d = 1.f / static_cast<float>(a.d);
  const bool post = a.branch_weight != nullptr, norm = a.weight != nullptr;
  const bool has_gate = a.gate.p != nullptr, has_dr = a.grad_residual_out.p != nullptr;
  const bool gate_sum = has_gate && a.gate.ld == 0;
  float sum_w[G][8] = {}, sum_b[G][8] = {}, sum_g[G][8] = {};
  const int64_t step = int64_t(gridDim.x) * shape.teams;
  int turn = 0;
  // every team runs as many turns as the CTA's first, so that all meet at the barriers
  for (int64_t t0 = int64_t(blockIdx.x) * shape.teams; t0 < a.T; t0 += step, turn ^= 1) {
    int64_t t = t0 + in_cta;
    Place p{t < a.T ? a.d : 0, int(threadIdx.x & 31), stretches + warp * 256 * sizeof(float)};
    if (t >= a.T) t = 0;
    Group<R> s[G], dr[G];
    Group<A> y[G], g[G], dh[G];
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const int64_t index = i + k * shape.team;
      if (norm) {
        s[k] = read_group(row_of<const R>(a.residual_out, t), index, aligned & kWideOut, p);
        dh[k] = read_group(row_of<const A>(a.grad_normed, t), index, aligned & kWideGradNormed, p);
      }
      if (has_dr)
        dr[k] = read_group(row_of<const R>(a.grad_residual_out, t), index, aligned & kWideGradOut, p);
      if (a.branch.p)
        y[k] = read_group(row_of<const A>(a.branch, t), index, aligned & kWideBranch, p);
      if (has_gate) g[k] = read_group(row_of<const A>(a.gate, t), index, aligned & kWideGate, p);
    }
    const float root = norm ? a.rstd[t] : 0.f, root_y = post ? a.branch_rstd[t] : 1.f;
    float m[3] = {0.f, 0.f, 0.f};
    if (norm) {
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const int64_t index = i + k * shape.team;
        float w[8];
        read_weight(a.weight, a.weight_bf16, index, aligned & kWideWeight, p, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) m[0] += element(dh[k], e) * w[e] * (element(s[k], e) * root);
      }
    }
    if (post) {
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const int64_t index = i + k * shape.team;
        float w[8], wb[8];
        if (norm) read_weight(a.weight, a.weight_bf16, index, aligned & kWideWeight, p, w);
        read_weight(a.branch_weight, a.weight_bf16, index, aligned & kWideBranchWeight, p, wb);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float f = a.branch_scale * wb[e];
          if (has_gate) f *= element(g[k], e);
          f *= element(y[k], e) * root_y;
          float D = has_dr ? element(dr[k], e) : 0.f;
          if (norm) {
            D += root * (element(dh[k], e) * w[e]);
            m[2] += f * (root * (element(s[k], e) * root));
          }
          m[1] += f * D;
        }
      }
    }
    if (norm || post) team_sum(m, slots[turn], shape.team, warp, first_warp);
    const float m1 = m[0] * inv_d, m2 = (m[1] - m1 * m[2]) * inv_d;
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const int64_t index = i + k * shape.team;
      float D[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) D[e] = has_dr ? element(dr[k], e) : 0.f;
      if (norm) {
        float w[8];
        read_weight(a.weight, a.weight_bf16, index, aligned & kWideWeight, p, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = element(s[k], e) * root, h = element(dh[k], e);
          D[e] += root * (h * w[e] - x * m1);
          sum_w[k][e] += h * x;
        }
      }
      float out[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) out[e] = a.residual_scale * D[e];
      write_group(row_of<R>(a.grad_residual, t), index, aligned & kWideGradResidual, p,
                  pack(out, R()));
      if (a.branch.p == nullptr) continue;
      float wb[8];
      if (post) read_weight(a.branch_weight, a.weight_bf16, index, aligned & kWideBranchWeight, p, wb);
      float dg[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float yh = element(y[k], e) * root_y;
        float dn = a.branch_scale * D[e];
        if (has_gate) {
          dg[e] = dn * (post ? yh * wb[e] : yh);
          if (gate_sum) sum_g[k][e] += dg[e];
          dn *= element(g[k], e);
        }
        if (post) {
          sum_b[k][e] += dn * yh;
          dn = root_y * (dn * wb[e] - yh * m2);
        }
        out[e] = dn;
      }
      if (has_gate && !gate_sum && a.grad_gate.p != nullptr)
        write_group(row_of<A>(a.grad_gate, t), index, aligned & kWideGradGate, p, pack(dg, A()));
      write_group(row_of<A>(a.grad_branch, t), index, aligned & kWideGradBranch, p, pack(out, A()));
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (a.partials == nullptr) return;
  // the teams' sums in order, then the CTA's [3][d]
  float* shared = reinterpret_cast<float*>(stretches);
  float* part = a.partials + int64_t(blockIdx.x) * 3 * a.d;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    float(&sum)[G][8] = q == 0 ? sum_w : q == 1 ? sum_b : sum_g;
    if (q == 0 ? a.grad_weight == nullptr : q == 1 ? a.grad_branch_weight == nullptr : !gate_sum)
      continue;
    for (int from = 1; from < shape.teams; ++from) {
      __syncthreads();
      if (in_cta == from)
#pragma unroll
        for (int k = 0; k < G; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) shared[(k * shape.team + i) * 8 + e] = sum[k][e];
      __syncthreads();
      if (in_cta == 0)
#pragma unroll
        for (int k = 0; k < G; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[k][e] += shared[(k * shape.team + i) * 8 + e];
    }
    if (in_cta == 0)
#pragma unroll
      for (int k = 0; k < G; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t c = 8 * int64_t(i + k * shape.team) + e;
          if (c < a.d) part[q * a.d + c] = sum[k][e];
        }
  }
}

// Backward of rows wider than that: the row is read twice (the second time from L2) and the
// sums over rows lie in shared memory, where each column has one owner.
constexpr int kWideThreads = 1024;

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
    if (norm || post) team_sum(m, slots[turn], kWideThreads, threadIdx.x / 32, 0);
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
  float* part = a.partials + int64_t(blockIdx.x) * 3 * d;
  for (int64_t c = threadIdx.x; c < d; c += kWideThreads)
#pragma unroll
    for (int q = 0; q < 3; ++q) part[q * d + c] = sums[q * d + c];
}

// The CTAs' partial sums: 8 threads a column take every eighth part in order, and their
// sums are added in order.
constexpr int kSumLanes = 8;
__global__ void __launch_bounds__(32 * kSumLanes)
    lp_norm_sum_kernel(const float* partials, int64_t parts, int64_t d, float* grad_weight,
                       float* grad_branch_weight, float* grad_gate) {
  __shared__ float slots[kSumLanes][32];
  float* const out = blockIdx.y == 0 ? grad_weight : blockIdx.y == 1 ? grad_branch_weight : grad_gate;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, from = threadIdx.x / 32;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  // launched as a programmatic dependent of the row kernel: wait for its partial sums
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.f;
  if (c < d)
    for (int64_t p = from; p < parts; p += kSumLanes) s += partials[(p * 3 + blockIdx.y) * d + c];
  slots[from][lane] = s;
  __syncthreads();
  if (from != 0 || c >= d) return;
  for (int k = 1; k < kSumLanes; ++k) s += slots[k][lane];
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

lp_status launched() { return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA; }

// Shared bytes of the warps' stretches; none when every operand is aligned.
size_t stretch_bytes(uint32_t aligned, uint32_t all, const Shape& s) {
  return (aligned & all) == all ? 0 : size_t(s.team) * s.teams / 32 * 256 * sizeof(float);
}

template <int G>
lp_status launch_forward(const NormArgs& a, uint32_t aligned, cudaStream_t stream) {
  return with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
    const Shape s = shape_of(a.d, G, a.T);
    const int64_t blocks = (a.T + s.teams - 1) / s.teams;
    constexpr uint32_t all = kWideResidual | kWideBranch | kWideGate | kWideOut | kWideNormed;
    lp_residual_norm_kernel<decltype(r), decltype(x), G>
        <<<unsigned(blocks), s.team * s.teams, stretch_bytes(aligned, all, s), stream>>>(a, s,
                                                                                       aligned);
    return launched();
  });
}

// The rows that the backward's CTAs take at once, and how many CTAs there are.
constexpr int64_t kTeamDim = kMaxTeam * 8 * 2;  // the widest row of the team kernel
int groups_of(int64_t d) { return d <= kTeamDim / 2 ? 1 : 2; }
int64_t backward_blocks(int64_t T, int64_t d) {
  const int64_t at_once = d <= kTeamDim ? shape_of(d, groups_of(d), T).teams : 1;
  return std::min((T + at_once - 1) / at_once, kSlots);
}

template <int G>
lp_status launch_backward(const NormGradArgs& a, uint32_t aligned, int64_t blocks,
                          cudaStream_t stream) {
  return with_types(a.residual_bf16, a.act_bf16, [&](auto r, auto x) {
    const Shape s = shape_of(a.d, G, a.T);
    constexpr uint32_t all = kWideOut | kWideBranch | kWideGate | kWideGradNormed | kWideGradOut |
                             kWideGradResidual | kWideGradBranch | kWideGradGate;
    size_t smem = stretch_bytes(aligned, all, s);
    if (s.teams > 1) smem = std::max(smem, size_t(s.team) * G * 8 * sizeof(float));
    lp_residual_norm_grad_kernel<decltype(r), decltype(x), G>
        <<<unsigned(blocks), s.team * s.teams, smem, stream>>>(a, s, aligned);
    return launched();
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

lp_status launch_residual_norm(const Device&, const NormArgs& a, cudaStream_t stream) {
  const uint32_t aligned =
      wide(kWideResidual, a.residual.p, a.residual.ld, a.residual_bf16) |
      wide(kWideBranch, a.branch.p, a.branch.p ? a.branch.ld : 0, a.act_bf16) |
      wide(kWideGate, a.gate.p, a.gate.p ? a.gate.ld : 0, a.act_bf16) |
      wide(kWideBranchWeight, a.branch_weight, 0, a.weight_bf16) |
      wide(kWideWeight, a.weight, 0, a.weight_bf16) |
      wide(kWideOut, a.residual_out.p, a.residual_out.p ? a.residual_out.ld : 0, a.residual_bf16) |
      wide(kWideNormed, a.normed.p, a.normed.p ? a.normed.ld : 0, a.act_bf16);
  if (a.d <= kMaxTeam / 2 * 8) return launch_forward<1>(a, aligned, stream);
  if (a.d <= kMaxTeam * 16) return launch_forward<2>(a, aligned, stream);
  return launch_forward<4>(a, aligned, stream);
}

size_t residual_norm_backward_workspace(int64_t T, int64_t d) {
  return static_cast<size_t>(std::max<int64_t>(1, backward_blocks(std::max<int64_t>(T, 1), d)) * 3 *
                             d * 4);
}

lp_status launch_residual_norm_backward(const Device& dev, const NormGradArgs& a,
                                        cudaStream_t stream) {
  const int64_t blocks = a.T > 0 ? backward_blocks(a.T, a.d) : 0;
  if (blocks > 0) {
    const auto rows = [](uint32_t bit, const Rows& r, bool bf16) {
      return wide(bit, r.p, r.p ? r.ld : 0, bf16);
    };
    const uint32_t aligned = rows(kWideOut, a.residual_out, a.residual_bf16) |
                             rows(kWideBranch, a.branch, a.act_bf16) |
                             rows(kWideGate, a.gate, a.act_bf16) |
                             wide(kWideBranchWeight, a.branch_weight, 0, a.weight_bf16) |
                             wide(kWideWeight, a.weight, 0, a.weight_bf16) |
                             rows(kWideGradNormed, a.grad_normed, a.act_bf16) |
                             rows(kWideGradOut, a.grad_residual_out, a.residual_bf16) |
                             rows(kWideGradResidual, a.grad_residual, a.residual_bf16) |
                             rows(kWideGradBranch, a.grad_branch, a.act_bf16) |
                             rows(kWideGradGate, a.grad_gate, a.act_bf16);
    const lp_status st = a.d > kTeamDim         ? launch_backward_wide(dev, a, blocks, stream)
                         : groups_of(a.d) == 1 ? launch_backward<1>(a, aligned, blocks, stream)
                                               : launch_backward<2>(a, aligned, blocks, stream);
    if (st != LP_OK) return st;
  }
  float* gate_sum = a.gate.ld == 0 ? static_cast<float*>(a.grad_gate.p) : nullptr;
  if (a.grad_weight == nullptr && a.grad_branch_weight == nullptr && gate_sum == nullptr)
    return LP_OK;
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

cudaError_t take_check_word_norm(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
