// lp_norm.cuh: what the residual norm's forward and backward kernels share.
//
// Both are bound by the bytes of their row operands, so a row is read once and held
// on chip.  A row belongs to a team of whole warps; thread i of a team of n owns the
// groups of 8 columns i, i + n, i + 2n, ... of the row, which is 16 bytes of bfloat16
// or 32 of float32.  The team's size and the groups a thread holds depend on d alone,
// so a row's sums are taken in the same order whatever the batch.
//
// A CTA takes rows in turn.  The operands of the next rows are on their way into a ring
// of shared memory (cp.async) while the current one is computed, so that the two
// sums of a row, each a wait for all its threads, do not leave the memory idle.  A thread
// copies its own groups where every row is aligned for it; else its warp copies its stretch of
// the row, 32 neighbouring words an access.  Where bfloat16 rows begin in the middle of a word,
// the forward, whose two CTAs an SM hide the wait, loads elements; the backward copies the words that
// hold the stretch and shifts the group out of them.  (4864 x 2397: 30 and 65 us.  The forward with
// shifts takes 33, the backward with elements 116.)  The arithmetic and its order are the same.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "lp_check.cuh"
#include "lp_train_internal.h"

namespace lp {
namespace {

constexpr int kMaxTeam = 512;  // threads of a row, and of a CTA
constexpr int kMaxWarps = kMaxTeam / 32;
// Row slots: one for each SM of a GB300.  Fixed, so that the order in which the backward
// sums rows does not depend on the device's partition.
constexpr int64_t kSlots = 152;

// 8 columns as they lie in memory.
template <class T>
struct __align__(8 * sizeof(T)) Group {
  uint32_t w[2 * sizeof(T)];
};
using Group16 = Group<__nv_bfloat16>;
using Group32 = Group<float>;

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

// The columns as four pairs, and back: the arithmetic is on pairs, two columns an instruction.
using Pairs = float2[4];
__device__ __forceinline__ void unpack(const Group32& g, Pairs& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = make_float2(__uint_as_float(g.w[2 * i]), __uint_as_float(g.w[2 * i + 1]));
}
__device__ __forceinline__ void unpack(const Group16& g, Pairs& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = make_float2(__uint_as_float(g.w[i] << 16), __uint_as_float(g.w[i] & 0xffff0000u));
}
__device__ __forceinline__ Group32 pack(const Pairs& v, float) {
  Group32 g;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    g.w[2 * i] = __float_as_uint(v[i].x), g.w[2 * i + 1] = __float_as_uint(v[i].y);
  return g;
}
__device__ __forceinline__ Group16 pack(const Pairs& v, __nv_bfloat16) {
  Group16 g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(v[i].x, v[i].y);
    g.w[i] = *reinterpret_cast<const uint32_t*>(&two);
  }
  return g;
}
// Element i as it is stored.
__device__ __forceinline__ float item(const Group32& g, int i) { return __uint_as_float(g.w[i]); }
__device__ __forceinline__ __nv_bfloat16 item(const Group16& g, int i) {
  return __ushort_as_bfloat16(
      static_cast<unsigned short>(i & 1 ? g.w[i / 2] >> 16 : g.w[i / 2] & 0xffffu));
}

__device__ __forceinline__ uint64_t as_bits(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 as_pair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_bits(a)), "l"(as_bits(b)));
  return as_pair(r);
}
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_bits(a)), "l"(as_bits(b)), "l"(as_bits(c)));
  return as_pair(r);
}

// How an operand's rows can be reached: by whole groups, by words, or by words that some rows begin
// in the middle of (bfloat16).  2 bits an operand.
enum Access : uint32_t { kHalves = 0, kWords = 1, kWide = 2 };
// What a kernel is built for: row operands of whole groups (d a multiple of 8, rows less than 2^32
// bytes apart), none in the middle of a word, any by elements, any by words and shifts.
enum Align : int { kAligned, kByWords, kByElements, kShifted };
enum Operand : int {
  kResidual, kBranch, kGate, kOut, kNormed, kGradNormed, kGradOut, kGradResidual, kGradBranch,
  kGradGate, kBranchWeight, kWeight,
};
__host__ __device__ __forceinline__ uint32_t access_of(uint32_t accesses, int operand) {
  return accesses >> 2 * operand & 3u;
}

// How rows of d columns are laid over threads.
struct Shape {
  int team;   // threads of a row
  int teams;  // rows of a CTA at once
};

// What the kernels need to know besides the operands.
struct Plan {
  Shape shape;
  uint32_t accesses;
  int stages;       // of the ring
  int stage_bytes;
};

// A thread's place in its CTA, and the call's rows.
struct Place {
  int64_t rows;
  int d;           // the row's columns
  int i, team;     // which thread of its team
  int lane, warp;
  int in_cta;      // which team of the CTA
  int first_warp;  // of the team
  __device__ __forceinline__ Place(int64_t rows, int64_t columns, const Shape& s)
      : rows(rows),
        d(int(columns)),
        i(int(threadIdx.x)),
        team(s.team),
        lane(int(threadIdx.x & 31)),
        warp(int(threadIdx.x / 32)),
        in_cta(0),
        first_warp(0) {
    if (s.teams > 1) {
      in_cta = int(threadIdx.x) / s.team;
      i -= in_cta * s.team;
      first_warp = in_cta * (s.team / 32);
    }
  }
  // What the checked build tests: that the operands have row t, and in it `n` columns from `from` on.
  __device__ __forceinline__ bool has(int64_t t) const { return t >= 0 && t < rows; }
  __device__ __forceinline__ bool has(int64_t t, int from, int n) const {
    return has(t) && from >= 0 && from + n <= d;
  }
};

// Where row t of an operand begins, `column` elements on.  With kAligned rows are less than 2^32 bytes
// apart, and the address is one multiplication.
template <class T, int kAlign>
__device__ __forceinline__ T* row_at(const Rows& r, int64_t t, int column) {
  if (kAlign == kAligned) {
    const uint64_t first = reinterpret_cast<uint64_t>(r.p) + uint32_t(column) * uint32_t(sizeof(T));
    return reinterpret_cast<T*>(first + uint64_t(uint32_t(t)) * uint32_t(r.ld * int64_t(sizeof(T))));
  }
  return static_cast<T*>(r.p) + t * r.ld + column;
}

// Whether row t of bfloat16 begins in the middle of a word.
__device__ __forceinline__ bool mid_word(const Rows& r, int64_t t) {
  return ((reinterpret_cast<uintptr_t>(r.p) >> 1) + uint32_t(t) * uint32_t(r.ld)) & 1u;
}

// A row operand on its way through the ring.
template <class T, int kAlign>
struct Stream {
  // rows that may begin in the middle of a word: a warp's stretch of such a row is copied from that
  // word on, so that it takes a word more
  static constexpr bool kMayShift = kAlign == kShifted && sizeof(T) == 2;
  static constexpr uint32_t kWarp = 256 * uint32_t(sizeof(T)) + (kMayShift ? 16 : 0);
  uint32_t first;  // the shared address of the thread's first group in stage 0

  // `offset` is the operand's first byte in a stage, moved past it.
  template <int G>
  __device__ __forceinline__ void start(uint32_t stage0, uint32_t* offset) {
    first = stage0 + *offset + threadIdx.x / 32 * kWarp + (threadIdx.x & 31) * 8 * uint32_t(sizeof(T));
    *offset += blockDim.x / 32 * G * kWarp;
  }
  __device__ __forceinline__ uint32_t slot(uint32_t at, int k) const {
    return first + at + k * (blockDim.x / 32) * kWarp;
  }
  // Starts the copy of row t's groups into the stage `at` bytes on.  Columns past the row become
  // zero (with kAligned they are never written: the ring starts as zeros).
  template <int G>
  __device__ __forceinline__ void fetch(const Rows& r, int64_t t, uint32_t at, uint32_t access,
                                        const Place& p) const {
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const uint32_t to = slot(at, k);
      const int c = 8 * (p.i + k * p.team);
      if (kAlign == kAligned) {
        const T* from = row_at<const T, kAligned>(r, t, c);
        if (c < p.d && LP_CHECK(p.has(t, c, 8), kChkCopyIndex))
#pragma unroll
          for (int q = 0; q < int(sizeof(T)) / 2; ++q)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16 * q),
                         "l"(from + q * (16 / int(sizeof(T))))
                         : "memory");
        continue;
      }
      const T* row = row_at<const T, kAlign>(r, t, 0);
      // an address for copies of no bytes
      const T* none = reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(r.p) & ~uintptr_t(3));
      if (access == kWide) {  // aligned rows whose last group is not whole
#pragma unroll
        for (int q = 0; q < int(sizeof(T)) / 2; ++q) {
          constexpr int kOf16 = 16 / int(sizeof(T));
          const int bytes = min(max((p.d - c - q * kOf16) * int(sizeof(T)), 0), 16);
          if (!LP_CHECK(bytes == 0 || p.has(t, c + q * kOf16, bytes / int(sizeof(T))), kChkCopyIndex)) continue;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + 16 * q),
                       "l"(bytes ? row + c + q * kOf16 : none), "r"(bytes)
                       : "memory");
        }
        continue;
      }
      // the warp's stretch, 32 neighbours an access
      const int first_column = 8 * (p.i - p.lane + k * p.team);
      const bool whole = first_column + 256 <= p.d;
      if (kAlign == kByElements && sizeof(T) == 2 && access == kHalves) {
        T* to_first = shared_pointer(to) - 7 * p.lane;
        const T* from = row + first_column + p.lane;
        T v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          v[q] = (whole || first_column + 32 * q + p.lane < p.d) &&
                         LP_CHECK(p.has(t, first_column + 32 * q + p.lane, 1), kChkCopyIndex)
                     ? from[32 * q]
                     : T(0.f);
#pragma unroll
        for (int q = 0; q < 8; ++q) to_first[32 * q] = v[q];
        continue;
      }
      constexpr int kOf4 = 4 / sizeof(T);
      const int shift = kMayShift && mid_word(r, t) ? 1 : 0;
      const uint32_t stretch = to - 8 * p.lane * uint32_t(sizeof(T)) + 4 * p.lane;
      const T* from = row + first_column + p.lane * kOf4 - shift;
      const T* begin = static_cast<const T*>(r.p);
      // whether word q's elements, the first `n` of them, are the row's; a shifted row's first word
      // begins with the element in front of it, which is the operand's unless the row is its first
      const auto inside = [&](int q, int n) {
        const int first = first_column + (32 * q + p.lane) * kOf4 - shift;
        const int front = first < 0 && from + 32 * q * kOf4 >= begin ? 1 : 0;
        return p.has(t, first + front, n - front);
      };
      const auto copy = [&](int q) {
        const int left = p.d - first_column + shift - (32 * q + p.lane) * kOf4;
        const uint32_t bytes = left >= kOf4 ? 4u : left > 0 ? uint32_t(sizeof(T)) : 0u;
        if (!LP_CHECK(bytes == 0u || inside(q, int(bytes / sizeof(T))), kChkCopyIndex)) return;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(stretch + 128 * q),
                     "l"(bytes ? from + 32 * q * kOf4 : none), "r"(bytes)
                     : "memory");
      };
      const bool before = kMayShift && from < begin;  // nothing before the operand is read
      if (kMayShift && shift != 0 && p.lane == 0) copy(2 * int(sizeof(T)));  // the word more
      if (whole && !before) {
#pragma unroll
        for (int q = 0; q < 2 * int(sizeof(T)); ++q)
          if (LP_CHECK(inside(q, kOf4), kChkCopyIndex))
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(stretch + 128 * q),
                         "l"(from + 32 * q * kOf4)
                         : "memory");
        continue;
      }
      if (before) {
        shared_pointer(stretch)[0] = T(0.f);
        if (LP_CHECK(p.has(t, 0, 1), kChkCopyIndex)) shared_pointer(stretch)[1] = *begin;
      } else {
        copy(0);
      }
#pragma unroll
      for (int q = 1; q < 2 * int(sizeof(T)); ++q) copy(q);
    }
  }
  // Zeros instead of a row that the team does not have: it then adds nothing to any sum.
  template <int G>
  __device__ __forceinline__ void zero(uint32_t at) const {
#pragma unroll
    for (int k = 0; k < G; ++k)
#pragma unroll
      for (int q = 0; q < int(sizeof(T)) / 2 + (kMayShift ? 1 : 0); ++q)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(slot(at, k) + 16 * q), "r"(0)
                     : "memory");
  }
  // The thread's group k of row t in the stage `at` bytes on.
  __device__ __forceinline__ void get(const Rows& r, int64_t t, uint32_t at, int k, Pairs& v) const {
    const uint32_t from = slot(at, k);
    Group<T> g;
#pragma unroll
    for (int q = 0; q < int(sizeof(T)) / 2; ++q)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(g.w[4 * q]), "=r"(g.w[4 * q + 1]), "=r"(g.w[4 * q + 2]), "=r"(g.w[4 * q + 3])
                   : "r"(from + 16 * q)
                   : "memory");
    if constexpr (kMayShift) {
      if (mid_word(r, t)) {
        uint32_t after;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(after) : "r"(from + 16) : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) g.w[i] = __funnelshift_r(g.w[i], i < 3 ? g.w[i + 1] : after, 16);
      }
    }
    unpack(g, v);
  }
  static __device__ __forceinline__ T* shared_pointer(uint32_t address) {
    return static_cast<T*>(__cvta_shared_to_generic(address));
  }
};

// Zeros in the ring, for the threads of kAligned whose groups lie past the row's columns.  (Elsewhere
// every group is written, or copied as zeros.)
template <int kAlign, int G>
__device__ __forceinline__ void clear_ring(unsigned char* ring, int bytes, const Place& p) {
  if constexpr (kAlign == kAligned) {
    if (8 * G * p.team == p.d) return;
    for (int i = threadIdx.x; i < bytes / 16; i += blockDim.x)
      reinterpret_cast<uint4*>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  }
}

// Rows of a team in the ring.  Eight, for deeper copies, made the backward of 4864 x 4096 69 us
// instead of 63, and no case faster.
constexpr int kMaxStages = 4;
// Waits for all but the newest `ahead` commits of this thread's copies; ahead < kMaxStages.
__device__ __forceinline__ void wait_copies(int ahead) {
  switch (ahead) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}
__device__ __forceinline__ void commit_copies() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Writes the thread's group k of row t, through a warp's stretch of 256 elements where rows are not
// aligned, if the team has the row.  All threads of a warp call it together.
template <class T, int kAlign>
__device__ __forceinline__ void put(const Rows& r, int64_t t, int k, bool mine, uint32_t access,
                                    const Place& p, void* stretch, const Pairs& v) {
  if (!mine) return;
  const Group<T> g = pack(v, T());
  const int c = 8 * (p.i + k * p.team);
  if (kAlign == kAligned) {
    T* to = row_at<T, kAligned>(r, t, c);
    if (c < p.d && LP_CHECK(p.has(t, c, 8), kChkRowIndex)) store_group(to, g);
    return;
  }
  T* row = row_at<T, kAlign>(r, t, 0);
  if (access == kWide) {
    if (!LP_CHECK(p.has(t), kChkRowIndex)) return;
    if (c + 8 <= p.d) return store_group(row + c, g);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < p.d) row[c + e] = item(g, e);
    return;
  }
  T* s = static_cast<T*>(stretch);
  const int first = c - 8 * p.lane;
  __syncwarp();
  reinterpret_cast<Group<T>*>(s)[p.lane] = g;
  __syncwarp();
  // 32 neighbours an access: words, or elements where rows may begin in the middle of a word (to shift
  // a group over the warp instead cost 2 us of the forward's 33 for 4864 x 2397)
  T* to = row + first + p.lane;
  const T* from = s + p.lane;
  if (!LP_CHECK(p.has(t) && first >= 0, kChkRowIndex)) return;
  if (first + 256 > p.d) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (first + 32 * q + p.lane < p.d) to[32 * q] = from[32 * q];
  } else if (kAlign == kByWords && sizeof(T) == 2) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      reinterpret_cast<uint32_t*>(row + first)[32 * q + p.lane] =
          reinterpret_cast<const uint32_t*>(s)[32 * q + p.lane];
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) to[32 * q] = from[32 * q];
  }
}

// Group k of a weight vector, of a type known at run time.  It is read again by every row, so it
// may stay in L1.
__device__ __forceinline__ void read_weight(const void* w, bool bf16, int k, bool wide,
                                            const Place& p, Pairs& v) {
  const int index = p.i + k * p.team, c = 8 * index;
  if (!LP_CHECK(index >= 0, kChkCopyIndex)) return;
  if (wide && c + 8 <= p.d) {
    if (bf16) {
      const uint4 x = __ldg(static_cast<const uint4*>(w) + index);
      unpack(Group16{{x.x, x.y, x.z, x.w}}, v);
    } else {
      const float4 a = __ldg(static_cast<const float4*>(w) + 2 * index);
      const float4 b = __ldg(static_cast<const float4*>(w) + 2 * index + 1);
      v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w);
      v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = c + e >= p.d ? 0.f
                    : bf16       ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c + e])
                                 : static_cast<const float*>(w)[c + e];
    if (e & 1)
      v[e / 2].y = x;
    else
      v[e / 2].x = x;
  }
}

// Sums over lanes of kCount values at once: in each step a lane hands half of its values to the
// lane `distance` away and takes that one's share of the other half, until it has one; its index is
// in the lane's bits from the first distance down.  Then the rest of the distances down to kLast.
template <int kCount>
__device__ __forceinline__ float exchange_sum(float (&v)[kCount], int lane, int last) {
  int distance = 16;
#pragma unroll
  for (int half = kCount / 2; half > 0; half /= 2, distance /= 2) {
    const bool upper = (lane & distance) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float give = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, distance);
    }
  }
  float s = v[0];
#pragma unroll
  for (; distance >= last; distance /= 2) s += __shfl_xor_sync(0xffffffffu, s, distance);
  return s;
}
// N sums over a team at once, the same bits for all its threads: over the warps' lanes, then over
// the warps, of which there are at most 16.  `slots` is written again only after another barrier.
__host__ __device__ constexpr int padded(int n) { return n <= 2 ? n : n <= 4 ? 4 : 8; }
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*slots)[padded(N)], const Place& p) {
  constexpr int kCount = padded(N), kLanes = 32 / kCount;
  float all[kCount];
#pragma unroll
  for (int i = 0; i < kCount; ++i) all[i] = i < N ? v[i] : 0.f;
  const float mine = exchange_sum(all, p.lane, 1);  // of value lane / kLanes
  if (p.team == 32) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, mine, i * kLanes);
    return;
  }
  if (p.lane % kLanes == 0) slots[p.warp][p.lane / kLanes] = mine;
  __syncthreads();
  if (kCount == 1) {
    const int w = p.lane & (kMaxWarps - 1);
    float s = 32 * w < p.team ? slots[p.first_warp + w][0] : 0.f;
#pragma unroll
    for (int o = kMaxWarps / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    v[0] = s;
    return;
  }
  // lane 2 w + h: half h of warp w's values
  constexpr int kHalf = kCount > 1 ? kCount / 2 : 1;
  const int w = p.lane / 2, h = p.lane & 1;
  float part[kHalf];
#pragma unroll
  for (int i = 0; i < kHalf; ++i)
    part[i] = 32 * w < p.team ? slots[p.first_warp + w][h * kHalf + i] : 0.f;
  const float sum = exchange_sum(part, p.lane, 2);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // value i: half i / kHalf, and the bits of i % kHalf are the lane's from 16 down
    const int in_half = i % kHalf;
    const int from = i / kHalf + (kHalf == 4   ? (in_half >> 1) * 16 + (in_half & 1) * 8
                                  : kHalf == 2 ? in_half * 16
                                               : 0);
    v[i] = __shfl_sync(0xffffffffu, sum, from);
  }
}

// ------------------------------------------------------------------------- host

Shape shape_of(int64_t d, int groups_per_thread, int64_t T) {
  const int64_t groups = (d + 7) / 8;
  Shape s;
  s.team = int((groups + 32 * groups_per_thread - 1) / (32 * groups_per_thread)) * 32;
  s.teams = int(std::max<int64_t>(1, std::min<int64_t>(256 / s.team, T)));
  return s;
}

// The access that a row operand allows, in its place among the others'.
uint32_t access_bits(int operand, const void* p, int64_t ld, bool bf16) {
  const uintptr_t size = bf16 ? 2 : 4;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld) * size;
  return (at % (8 * size) == 0 ? kWide : at % 4 == 0 ? kWords : kHalves) << 2 * operand;
}
uint32_t access_bits(int operand, const Rows& r, bool bf16) {
  return access_bits(operand, r.p, r.p != nullptr ? r.ld : 0, bf16);
}
// Whether every operand allows whole groups and rows are made of them (an absent operand does).
bool all_wide(uint32_t accesses, std::initializer_list<int> operands, int64_t d) {
  for (int o : operands)
    if (access_of(accesses, o) != kWide) return false;
  return d % 8 == 0;
}
bool any_halves(uint32_t accesses, std::initializer_list<int> operands) {
  for (int o : operands)
    if (access_of(accesses, o) == kHalves) return true;
  return false;
}
// Whether rows are near enough for 32-bit pitches in bytes.
bool near(const Rows& r) { return r.p == nullptr || r.ld < (int64_t(1) << 30); }

// The ring and, where an output is not aligned, the warps' stretches.
constexpr int kRingBytes = 200 << 10;
constexpr int kStretch = 256 * int(sizeof(float));
// A stage: a row a team; where rows are not aligned 16 bytes more for each stretch of up to five operands.
int stage_bytes_of(int threads, int groups, int column_bytes, bool stretches) {
  return threads * groups * 8 * column_bytes + (stretches ? threads / 32 * groups * 6 * 16 : 0);
}
// Sets the stages, of one row a team, that fit `budget` bytes, at least `least`, and returns the
// dynamic shared bytes.  `rows`: that a team takes in all.
int plan_ring(Plan* plan, int column_bytes, int groups, bool stretches, int64_t rows, int least,
              int budget) {
  const int threads = plan->shape.team * plan->shape.teams;
  plan->stage_bytes = stage_bytes_of(threads, groups, column_bytes, stretches);
  const int extra = stretches ? threads / 32 * kStretch : 0;
  plan->stages = std::max(least, std::min({kMaxStages, (budget - extra) / plan->stage_bytes,
                                           int(std::min<int64_t>(rows, kMaxStages))}));
  return plan->stages * plan->stage_bytes + extra;
}

template <class K>
bool allow_ring(K* kernel, const Device& dev, PerContextOnce* once) {
  return once->run(dev.ctx_id, [&] {
           return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kRingBytes + (20 << 10));
         }) == cudaSuccess;
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

}  // namespace
}  // namespace lp
