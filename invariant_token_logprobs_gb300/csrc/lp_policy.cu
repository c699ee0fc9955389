// lp_policy.cu: the clipped policy-gradient loss and its gradients (include/lp_train.h).
//
// A row's weight needs the number of counted rows of its sequence, or of all, before any
// gradient can be written, so the call has two passes: over the masks (a byte a row) and over
// the rest.  Up to kSmallRows rows one CTA does both from registers in one launch; beyond
// that they are two grids over chunks of rows, launched as programmatic dependents.
//
// 512 rows take 3.0 us, next to nothing of it bytes: a launch, the loads, two barriers.  4.2 M rows
// of 1024 ragged sequences take 34 us where their 103 MB are 15: a turn of rows on all SMs takes
// 2.7 us, 5.7 TB/s, and there are 7, but 15 us pass outside them.  The first pass reads 4 MB in some
// 7 us, most of it the search for a CTA's sequences and the atomics' way; the second has its own
// search before its first turn, and 3 us for the last CTA's sum.  Copies two turns ahead (34 us),
// three or five CTAs an SM (34, 41) and a first pass of a quarter of the CTAs, to leave room for the
// second's start (36), gained nothing.  One CTA for everything took 11.6 ms; a chunk of 4096 rows a
// CTA 51 us, with 64-bit searches for each row.  Without a mask the counts are differences of the
// offsets, but the first pass runs all the same (36 us a call).
//
// Counts are integers added by atomics, whose order does not show.  The loss's sums are
// taken in a fixed order: a thread's rows, the CTA's tree, then the CTAs' sums by whichever
// CTA finishes last.
#include <cuda_runtime.h>

#include <algorithm>

#include "lp_check.cuh"
#include "lp_train_internal.h"

namespace lp {
namespace {

constexpr int kStats = 4;  // w policy, w kl, w entropy, the clipped rows' w

// ---- one CTA
constexpr int kSmallThreads = 1024;
constexpr int kSmallRounds = 2;  // groups of 4 rows a thread
constexpr int64_t kSmallRows = int64_t(kSmallThreads) * 4 * kSmallRounds;
constexpr int64_t kSmallSequences = 2048;

// ---- two grids
constexpr int kThreads = 256;
constexpr int kTurn = kThreads * 4;              // rows of a CTA at once in the second pass
constexpr int64_t kMostChunks = 152 * 4;         // its CTAs: four to an SM of a GB300
constexpr int kCountRun = 16;                    // neighbouring rows a thread of the first
constexpr int kCountChunk = kThreads * kCountRun;
constexpr int kStaged = 1024;                    // sequences of a chunk held in shared memory
// Rows of a CTA of the second pass: whole turns, as many as it takes.
int64_t chunk_of(int64_t T) {
  const int64_t turns = (T + kTurn - 1) / kTurn;
  return (turns + kMostChunks - 1) / kMostChunks * kTurn;
}

struct Header {
  unsigned counted;    // rows that count, in all
  unsigned sequences;  // sequences with a row that counts
  unsigned finished;   // CTAs of the second pass that have written their sums
};
constexpr size_t kHeaderBytes = 256;
size_t counts_bytes(int64_t n_sequences) {
  return static_cast<size_t>((n_sequences * 4 + 255) / 256 * 256);
}

// The first of n ascending offsets that is above t, in [0, n].
template <class Int>
__device__ __forceinline__ int64_t upper_bound(const Int* offsets, int64_t n, int64_t t) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (offsets[mid] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}
// The same by a whole warp, 32 probes a step: for offsets in global memory.
__device__ __forceinline__ int64_t warp_upper_bound(const int64_t* offsets, int64_t n, int64_t t) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = n;  // the answer is in [lo, hi]
  while (lo < hi) {
    const int64_t stride = (hi - lo + 31) / 32;
    const int64_t at = lo + lane * stride;
    const bool below = at < hi && offsets[at] <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, below));  // the probes below t come first
    if (k == 0) return lo;
    hi = min(hi, lo + k * stride);
    lo += (k - 1) * stride + 1;
  }
  return lo;
}

// Four values of an operand; rows from T on read as zero.
__device__ __forceinline__ void load4(const float* p, int64_t t, int64_t T, bool wide,
                                      float (&v)[4]) {
  if (wide && t + 4 <= T) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p + t));
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = t + j < T ? p[t + j] : 0.f;
}
__device__ __forceinline__ void store4(float* p, int64_t t, int64_t T, bool wide,
                                       const float (&v)[4]) {
  if (wide && t + 4 <= T) {
    *reinterpret_cast<float4*>(p + t) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (t + j < T) p[t + j] = v[j];
}
// Bit j: row t + j counts by the mask.
__device__ __forceinline__ unsigned load_mask4(const uint8_t* mask, int64_t t, int64_t T, bool wide) {
  const unsigned inside = t + 4 <= T ? 0xfu : t < T ? (1u << (T - t)) - 1u : 0u;
  if (mask == nullptr) return inside;
  unsigned kept = 0;
  if (wide && inside == 0xfu) {
    const uchar4 m = __ldg(reinterpret_cast<const uchar4*>(mask + t));
    kept = (m.x ? 1u : 0u) | (m.y ? 2u : 0u) | (m.z ? 4u : 0u) | (m.w ? 8u : 0u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (inside >> j & 1u) kept |= mask[t + j] != 0 ? 1u << j : 0u;
  }
  return kept;
}

// Four rows in registers.
struct Four {
  float logp[4], old[4], ref[4], entropy[4], advantage[4];
};
__device__ __forceinline__ void load_rows(const PolicyArgs& a, int64_t t, int64_t T, Four& f) {
  if (!LP_CHECK(t >= 0 && T <= a.T, kChkRowIndex)) return;
  load4(a.logp, t, T, a.wide, f.logp);
  load4(a.old_logp, t, T, a.wide, f.old);
  if (a.ref_logp != nullptr) load4(a.ref_logp, t, T, a.wide, f.ref);
  if (a.entropy != nullptr) load4(a.entropy, t, T, a.wide, f.entropy);
  if (!a.per_sequence) load4(a.advantages, t, T, a.wide, f.advantage);
}
// Their gradients, and their terms added to `sum`.  kept: the rows that count; w: weights.
__device__ __forceinline__ void finish_rows(const PolicyArgs& a, int64_t t, int64_t T,
                                            const Four& f, unsigned kept, const float (&w)[4],
                                            float (&sum)[kStats]) {
  float grad[4] = {0.f, 0.f, 0.f, 0.f}, grad_entropy[4] = {0.f, 0.f, 0.f, 0.f};
  // A row that does not count, whatever it holds, is one of zeros: without branches the four rows'
  // chains run side by side (512 rows: 0.4 us less).
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (kept == 0) break;
    const bool counts = kept >> j & 1u;
    const float weight = counts ? w[j] : 0.f, A = counts ? f.advantage[j] : 0.f;
    const float delta = counts ? f.logp[j] - f.old[j] : 0.f;
    const float ratio = expf(delta);
    // a finite difference whose exponential passes float32 gains nothing where there is no advantage
    const float gain = A != 0.f || !(fabsf(delta) <= 0x1.fffffep127f) ? A * ratio : 0.f;
    const bool over = A > 0.f && delta > a.high, under = A < 0.f && delta < a.low;
    const bool clipped = over || under;
    float g = clipped ? 0.f : -gain;
    sum[0] -= weight * (over ? A * a.ratio_high : under ? A * a.ratio_low : gain);
    if (a.ref_logp != nullptr) {
      const float r = counts ? f.ref[j] - f.logp[j] : 0.f, up = expm1f(r);
      sum[1] += weight * (up - r);
      if (a.kl_coef != 0.f) g -= a.kl_coef * up;
    }
    if (a.entropy != nullptr) sum[2] += weight * (counts ? f.entropy[j] : 0.f);
    sum[3] += clipped ? weight : 0.f;
    grad[j] = counts ? weight * g : 0.f;
    grad_entropy[j] = counts ? -a.entropy_coef * weight : 0.f;
  }
  if (!LP_CHECK(t >= 0 && T <= a.T, kChkRowIndex)) return;
  store4(a.grad_logp, t, T, a.wide, grad);
  if (a.grad_entropy != nullptr) store4(a.grad_entropy, t, T, a.wide, grad_entropy);
}

// The sums of a CTA's threads, in thread 0: shuffles, then the warps' sums in order.
template <int kCtaThreads>
__device__ __forceinline__ void cta_sum(float (&sum)[kStats], float (*slots)[kStats]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < kStats; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < kStats; ++k) slots[threadIdx.x / 32][k] = sum[k];
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int warp = 1; warp < int(blockDim.x) / 32; ++warp)
#pragma unroll
    for (int k = 0; k < kStats; ++k) sum[k] += slots[warp][k];
}

__device__ __forceinline__ void write_stats(const PolicyArgs& a, const float (&sum)[kStats]) {
  // a term with a coefficient of 0 is watched only: what it sums to may be no float32 number
  a.stats[0] = sum[0] + (a.kl_coef != 0.f ? a.kl_coef * sum[1] : 0.f) -
               (a.entropy_coef != 0.f ? a.entropy_coef * sum[2] : 0.f);
#pragma unroll
  for (int k = 0; k < kStats; ++k) a.stats[k + 1] = sum[k];
}

__device__ __forceinline__ float weight_of(bool by_sequence, unsigned in_sequence, unsigned whole) {
  return by_sequence
             ? 1.f / (static_cast<float>(max(in_sequence, 1u)) * static_cast<float>(max(whole, 1u)))
             : 1.f / static_cast<float>(max(whole, 1u));
}

__global__ void __launch_bounds__(kSmallThreads) lp_policy_small_kernel(const __grid_constant__ PolicyArgs a) {
  __shared__ int offsets[kSmallSequences + 1];
  __shared__ unsigned counts[kSmallSequences];
  __shared__ unsigned whole;
  __shared__ float slots[kSmallThreads / 32][kStats];
  const int B = int(a.n_sequences), threads = int(blockDim.x);
  const bool sequences = a.cu_seqlens != nullptr;
  if (threadIdx.x == 0) whole = 0;
  if (sequences)
    for (int i = threadIdx.x; i <= B; i += threads) {
      if (!LP_CHECK(i <= a.n_sequences && i <= kSmallSequences, kChkRowIndex)) continue;
      const int64_t c = a.cu_seqlens[i];
      offsets[i] = int(min(max(c, int64_t(0)), a.T));
      if (i < B) counts[i] = 0;
    }
  // all rows are on their way before the counts are needed
  Four rows[kSmallRounds];
  unsigned kept[kSmallRounds];
#pragma unroll
  for (int k = 0; k < kSmallRounds; ++k) {
    const int64_t t = 4 * (int64_t(threadIdx.x) + k * threads);
    kept[k] = load_mask4(a.mask, t, a.T, a.wide);
    load_rows(a, t, a.T, rows[k]);
  }
  __syncthreads();
  int sequence[kSmallRounds][4];
  unsigned mine = 0;
#pragma unroll
  for (int k = 0; k < kSmallRounds; ++k) {
    const int64_t t = 4 * (int64_t(threadIdx.x) + k * threads);
    if (sequences) {
      int s = t < a.T ? int(upper_bound(offsets + 1, B, t)) : B;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // the next sequence is mostly the next row's; past empty ones it is searched for
        if ((kept[k] >> j & 1u) && s < B && offsets[s + 1] <= t + j) {
          ++s;
          s += int(upper_bound(offsets + 1 + s, B - s, t + j));
        }
        sequence[k][j] = s;
        if (s == B || t + j < offsets[0]) kept[k] &= ~(1u << j);
        if (a.by_sequence && kept[k] >> j & 1u) mine += atomicAdd(&counts[s], 1u) == 0 ? 1u : 0u;
      }
    }
    if (!a.by_sequence) mine += __popc(kept[k]);
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if ((threadIdx.x & 31) == 0 && mine > 0) atomicAdd(&whole, mine);
  __syncthreads();
  float sum[kStats] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kSmallRounds; ++k) {
    const int64_t t = 4 * (int64_t(threadIdx.x) + k * threads);
    float w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!(kept[k] >> j & 1u)) continue;
      w[j] = weight_of(a.by_sequence, a.by_sequence ? counts[sequence[k][j]] : 0u, whole);
      if (a.per_sequence && LP_CHECK(sequence[k][j] >= 0 && sequence[k][j] < B, kChkRowIndex))
        rows[k].advantage[j] = a.advantages[sequence[k][j]];
    }
    finish_rows(a, t, a.T, rows[k], kept[k], w, sum);
  }
  cta_sum<kSmallThreads>(sum, slots);
  if (threadIdx.x == 0) write_stats(a, sum);
}

// The sequences that a chunk of rows [t0, t1) touches, with offsets counted from t0.
struct Span {
  int64_t first;  // of row t0
  int sequences;  // that the chunk's rows may lie in, from `first` on; 0: the rows lie in none
  int begin;      // where the first sequence of all begins
  bool staged;    // their ends are in shared memory
};
// Whether sequence i of the span is one of the call's.
__device__ __forceinline__ bool in_call(const PolicyArgs& a, const Span& span, int64_t i) {
  return i >= 0 && span.first >= 0 && span.first + i < a.n_sequences;
}
__device__ __forceinline__ int from_chunk(int64_t offset, int64_t t0) {
  return int(min(max(offset - t0, int64_t(0)), int64_t(1) << 30));
}
__device__ __forceinline__ Span find_span(const PolicyArgs& a, int64_t t0, int64_t t1, int* ends,
                                          int64_t* found) {
  const int warp = threadIdx.x / 32;
  if (warp < 2) {
    const int64_t s = warp_upper_bound(a.cu_seqlens + 1, a.n_sequences, warp == 0 ? t0 : t1 - 1);
    if ((threadIdx.x & 31) == 0) found[warp] = s;
  }
  Span span{};
  span.begin = from_chunk(__ldg(a.cu_seqlens), t0);
  __syncthreads();
  span.first = found[0];
  const int64_t sequences = max(min(found[1] + 1, a.n_sequences) - span.first, int64_t(0));
  span.staged = sequences <= kStaged;
  span.sequences = int(min(sequences, a.n_sequences));
  if (span.staged) {
    for (int i = threadIdx.x; i < span.sequences; i += kThreads)
      if (LP_CHECK(in_call(a, span, i), kChkRowIndex)) ends[i] = from_chunk(a.cu_seqlens[span.first + 1 + i], t0);
    __syncthreads();
  }
  return span;
}
// Where the span's sequence i ends.
__device__ __forceinline__ int local_end(const PolicyArgs& a, const Span& span, const int* ends,
                                         int64_t t0, int i) {
  if (span.staged) return ends[i];
  if (!LP_CHECK(in_call(a, span, i), kChkRowIndex)) return 0;
  return from_chunk(a.cu_seqlens[span.first + 1 + i], t0);
}
// Which of the span's sequences the chunk's row `r` lies in; span.sequences: in none.
// It is `lo` or a later one.
__device__ __forceinline__ int local_sequence(const PolicyArgs& a, const Span& span, const int* ends,
                                              int64_t t0, int r, int lo) {
  int hi = span.sequences;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;  // lo + hi may pass 32 bits
    if (local_end(a, span, ends, t0, mid) <= r)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads)
    lp_policy_clear_kernel(Header* header, unsigned* counts, int64_t n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i == 0) header->counted = header->sequences = header->finished = 0;
  if (i < n && LP_CHECK(i >= 0, kChkStateIndex)) counts[i] = 0;
}

// Bit j: byte j of the word is not zero.
__device__ __forceinline__ unsigned nonzero_bytes(unsigned x) {
  const unsigned y = __vcmpne4(x, 0u) & 0x01010101u;
  return (y * 0x10204080u) >> 28;
}

// First pass: the rows that count, in all or by sequence.
__global__ void __launch_bounds__(kThreads)
    lp_policy_count_kernel(const __grid_constant__ PolicyArgs a, Header* header, unsigned* counts) {
  __shared__ int ends[kStaged];
  __shared__ int64_t found[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t t0 = int64_t(blockIdx.x) * kCountChunk, t1 = min(t0 + kCountChunk, a.T);
  if (!LP_CHECK(t0 < a.T, kChkRowIndex)) return;
  const int r = int(threadIdx.x) * kCountRun, rows = int(t1 - t0);
  // bit j: row r + j counts by the mask
  unsigned kept = r + kCountRun <= rows ? 0xffffu : r < rows ? (1u << (rows - r)) - 1u : 0u;
  if (a.mask != nullptr && kept != 0) {
    const uint8_t* mask = a.mask + t0 + r;
    if (kept == 0xffffu && reinterpret_cast<uintptr_t>(mask) % 16 == 0) {
      const uint4 m = __ldg(reinterpret_cast<const uint4*>(mask));
      kept = nonzero_bytes(m.x) | nonzero_bytes(m.y) << 4 | nonzero_bytes(m.z) << 8 |
             nonzero_bytes(m.w) << 12;
    } else {
      unsigned some = 0;
#pragma unroll
      for (int j = 0; j < kCountRun; ++j)
        if (kept >> j & 1u) some |= mask[j] != 0 ? 1u << j : 0u;
      kept = some;
    }
  }
  Span span{};
  if (a.cu_seqlens != nullptr) span = find_span(a, t0, t1, ends, found);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the counters are zero
  unsigned mine = 0, in_last = 0;
  int last = -1;  // the sequence of the thread's last row
  if (a.cu_seqlens == nullptr) {
    mine = __popc(kept);
  } else {
    if (r < span.begin) kept &= span.begin - r >= 32 ? 0u : ~0u << (span.begin - r);
    int i = kept != 0 ? local_sequence(a, span, ends, t0, r, 0) : span.sequences;
    unsigned left = kept;
    while (left != 0 && i < span.sequences) {
      const int run = local_end(a, span, ends, t0, i) - r;  // rows up to the sequence's end
      const unsigned here = run >= 32 ? left : left & ((1u << max(run, 0)) - 1u);
      left &= ~here;
      const unsigned n = __popc(here);
      if (!a.by_sequence) {
        mine += n;
      } else if (left == 0) {
        in_last = n;
        last = i;
      } else if (n > 0) {
        if (LP_CHECK(in_call(a, span, i), kChkStateIndex))
          mine += atomicAdd(&counts[span.first + i], n) == 0 ? 1u : 0u;
      }
      ++i;
      if (left != 0 && i < span.sequences) {  // past empty sequences the next row's is searched for
        const int row = r + __ffs(left) - 1;
        if (local_end(a, span, ends, t0, i) <= row) i = local_sequence(a, span, ends, t0, row, i + 1);
      }
    }
  }
  if (a.by_sequence) {
    // a warp's 512 rows mostly end in one sequence
    int same;
    __match_all_sync(0xffffffffu, last, &same);
    if (same) in_last = __reduce_add_sync(0xffffffffu, in_last);
    if (in_last > 0 && (!same || (threadIdx.x & 31) == 0) &&
        LP_CHECK(in_call(a, span, last), kChkStateIndex))
      mine += atomicAdd(&counts[span.first + last], in_last) == 0 ? 1u : 0u;
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if ((threadIdx.x & 31) == 0 && mine > 0)
    atomicAdd(a.by_sequence ? &header->sequences : &header->counted, mine);
}

// Second pass: weights, terms, gradients, and the sums by the CTA that finishes last.  A CTA has a
// stretch of neighbouring rows, so that it looks for its sequences once; the rows of its next turn
// (of its first, before the first pass is waited for) are on their way while it computes.
__global__ void __launch_bounds__(kThreads, 4)
    lp_policy_rows_kernel(const __grid_constant__ PolicyArgs a, int64_t chunk, Header* header,
                          const unsigned* counts, float4* partials) {
  __shared__ int ends[kStaged];
  __shared__ float weights[kStaged], advantages[kStaged];
  __shared__ int64_t found[2];
  __shared__ float slots[kThreads / 32][kStats];
  __shared__ bool last;
  const int64_t t0 = int64_t(blockIdx.x) * chunk, t1 = min(t0 + chunk, a.T);
  if (!LP_CHECK(t0 < a.T, kChkRowIndex)) return;
  const int rows = int(t1 - t0);
  int r = 4 * int(threadIdx.x);
  Four next;
  unsigned next_kept = load_mask4(a.mask, t0 + r, t1, a.wide);
  load_rows(a, t0 + r, t1, next);
  Span span{};
  if (a.cu_seqlens != nullptr) span = find_span(a, t0, t1, ends, found);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the counts are done
  const unsigned whole = __ldcg(a.by_sequence ? &header->sequences : &header->counted);
  if (a.cu_seqlens != nullptr && span.staged) {
    for (int i = threadIdx.x; i < span.sequences; i += kThreads) {
      if (!LP_CHECK(in_call(a, span, i), kChkStateIndex)) continue;
      weights[i] = weight_of(a.by_sequence, a.by_sequence ? __ldcg(counts + span.first + i) : 0u, whole);
      if (a.per_sequence) advantages[i] = __ldg(a.advantages + span.first + i);
    }
    __syncthreads();
  }
  const float of_all = weight_of(false, 0u, whole);
  float sum[kStats] = {0.f, 0.f, 0.f, 0.f};
  int i = 0;  // the sequence of the thread's next row, or one before it
  for (; r < rows; r += kTurn) {
    Four four = next;
    unsigned kept = next_kept;
    next_kept = load_mask4(a.mask, t0 + r + kTurn, t1, a.wide);
    load_rows(a, t0 + r + kTurn, t1, next);
    float w[4] = {of_all, of_all, of_all, of_all};
    if (a.cu_seqlens != nullptr && kept != 0) {
      if (i < span.sequences && local_end(a, span, ends, t0, i) <= r)
        i = local_sequence(a, span, ends, t0, r, i + 1);
      if (span.staged && i < span.sequences && r >= span.begin && r + 4 <= ends[i]) {
        const float weight = weights[i];  // mostly all four rows lie in one sequence
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = weight;
        if (a.per_sequence) {
          const float advantage = advantages[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) four.advantage[j] = advantage;
        }
      } else {
        int s = i;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if ((kept >> j & 1u) && s < span.sequences && local_end(a, span, ends, t0, s) <= r + j)
            s = local_sequence(a, span, ends, t0, r + j, s + 1);
          if (s == span.sequences || r + j < span.begin) {
            kept &= ~(1u << j);
          } else {
            if (!LP_CHECK(in_call(a, span, s), kChkStateIndex)) continue;
            const int64_t at = span.first + s;
            if (a.by_sequence) w[j] = weight_of(true, __ldcg(counts + at), whole);
            if (a.per_sequence) four.advantage[j] = __ldg(a.advantages + at);
          }
        }
      }
    }
    finish_rows(a, t0 + r, t1, four, kept, w, sum);
  }
  cta_sum<kThreads>(sum, slots);
  if (threadIdx.x == 0) {
    partials[blockIdx.x] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    __threadfence();
    last = atomicAdd(&header->finished, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
#pragma unroll
  for (int k = 0; k < kStats; ++k) sum[k] = 0.f;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < gridDim.x; i += kThreads) {
    const float4 p = __ldcg(partials + i);
    sum[0] += p.x, sum[1] += p.y, sum[2] += p.z, sum[3] += p.w;
  }
  cta_sum<kThreads>(sum, slots);
  if (threadIdx.x == 0) write_stats(a, sum);
}

bool one_cta(int64_t T, int64_t n_sequences) {
  return T <= kSmallRows && n_sequences <= kSmallSequences;
}
int64_t chunks_of(int64_t T) { return T > 0 ? (T + chunk_of(T) - 1) / chunk_of(T) : 0; }

template <class... Params, class... Args>
bool launch_dependent(void (*kernel)(Params...), int64_t blocks, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

}  // namespace

size_t policy_loss_workspace(int64_t T, int64_t n_sequences) {
  if (one_cta(T, n_sequences)) return kHeaderBytes;
  return kHeaderBytes + counts_bytes(n_sequences) + static_cast<size_t>(chunks_of(T)) * sizeof(float4);
}

lp_status launch_policy_loss(const PolicyArgs& args, cudaStream_t stream) {
  PolicyArgs a = args;
  const auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  a.wide = at16(a.logp) && at16(a.old_logp) && at16(a.ref_logp) && at16(a.entropy) &&
           (a.per_sequence || at16(a.advantages)) && at16(a.grad_logp) && at16(a.grad_entropy) &&
           reinterpret_cast<uintptr_t>(a.mask) % 4 == 0;
  if (a.T == 0) {  // nothing counts
    a.cu_seqlens = nullptr;
    a.n_sequences = 0;
  }
  if (one_cta(a.T, a.n_sequences)) {
    const int64_t groups = (a.T + 3) / 4;
    const int threads = int(std::min<int64_t>(kSmallThreads, std::max<int64_t>(1, (groups + 31) / 32) * 32));
    lp_policy_small_kernel<<<1, threads, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
  }
  char* p = static_cast<char*>(a.workspace);
  Header* header = reinterpret_cast<Header*>(p);
  unsigned* counts = reinterpret_cast<unsigned*>(p + kHeaderBytes);
  float4* partials = reinterpret_cast<float4*>(p + kHeaderBytes + counts_bytes(a.n_sequences));
  const int64_t cleared = a.by_sequence ? a.n_sequences : 0;
  const int64_t chunks = chunks_of(a.T);
  lp_policy_clear_kernel<<<unsigned(cleared / kThreads + 1), kThreads, 0, stream>>>(header, counts, cleared);
  if (cudaGetLastError() != cudaSuccess) return LP_ERR_CUDA;
  if (!launch_dependent(lp_policy_count_kernel, (a.T + kCountChunk - 1) / kCountChunk, stream, a, header,
                        counts) ||
      !launch_dependent(lp_policy_rows_kernel, chunks, stream, a, chunk_of(a.T), header,
                        static_cast<const unsigned*>(counts), partials))
    return LP_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

cudaError_t take_check_word_policy(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
