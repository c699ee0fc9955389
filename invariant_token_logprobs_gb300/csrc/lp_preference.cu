// lp_preference.cu: the preference loss of pairs of sequences and its gradient (include/lp_tune.h).
//
// A row's gradient needs its pair's loss, which needs the sums of two whole sequences, and the number
// of pairs that count.  Up to kSmallRows rows one CTA does all of it in one launch.  Beyond that there
// are three launches, each a programmatic dependent of the one before:
//   sums   a warp takes kChunk neighbouring rows, however they lie in sequences, and writes a sum for
//          each sequence that it meets: long sequences are split over many warps, short ones share one;
//   pairs  a few lanes a pair, or its warp where it is far longer than the mean, add its sequences' sums and
//          write its loss and both gradients;
//   rows   as in the first, a warp takes kChunk rows and writes their gradients.
// 9 bytes a row in, the mask again and 4 bytes out.  512 pairs of up to 8192 tokens (4.1 M rows) take 27
// to 29 us, where the bytes need 8: sums 13 to 16 us, pairs 7 to 9 and rows 13 to 15 when each runs alone.  What bounds them
// is each launch's chain of dependent loads (offsets, rows, the chunk's sums), and in sums the two-sums'
// instructions (issue slots 51%).  Larger batches come closer: 2048 pairs 80 us, 32 of them bytes.  Up
// to kSmallRows a call is its launch and the chain of loads and barriers: 4 pairs 6 us.
// All of it as one cooperative launch, with barriers over the grid, took 45 us instead of 28.7, and 18.4
// instead of 16.4 for two pairs of 98,000 tokens.
//
// The difference of two sums of 10^5 rows is what counts, to a few units of float32: sums, scores and
// z are float pairs (Knuth's two-sum and products by fma), 48 bits.  In float64, at 1/64 of the rate
// here, the same took 53 us instead of 28.7 for 512 pairs.  Every sum is taken in a fixed order: a
// lane's rows, the lanes' tree, the chunks of a sequence in order.
#include <cuda_runtime.h>

#include <algorithm>

#include "lp_check.cuh"
#include "lp_tune_internal.h"

namespace lp {
namespace {

// ---- one CTA
constexpr int kSmallThreads = 1024;
constexpr int64_t kSmallRows = 8192;
constexpr int kSmallSequences = 64;  // a lane of one warp for each pair

// ---- three launches
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = 4;                // of 4 rows, a lane
constexpr int kChunk = kGroups * 4 * 32;  // rows of a warp
constexpr int kPairThreads = 128;

// s + e is a value to about 48 bits, |e| at most some units in the last place of s.  Once s is no number or
// infinite, e is nothing.
struct Two {
  float s = 0.f, e = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = s + x, b = t - s;
    e += (s - (t - b)) + (x - b);
    s = t;
  }
  __device__ __forceinline__ void add(const Two& x) {
    add(x.s);
    e += x.e;
  }
  __device__ __forceinline__ bool finite() const { return fabsf(s) <= 0x1.fffffep127f; }
  __device__ __forceinline__ float value() const { return finite() ? s + e : s; }
  // the same value with |e| at most half a unit of s
  __device__ __forceinline__ Two settled() const {
    Two t;
    t.s = value();
    t.e = finite() && t.finite() ? e - (t.s - s) : 0.f;
    return t;
  }
  __device__ __forceinline__ Two negative() const {
    Two t;
    t.s = -s, t.e = -e;
    return t;
  }
  __device__ __forceinline__ Two times(const Two& x) const {
    Two t;
    t.s = s * x.s;
    t.e = __fmaf_rn(s, x.s, -t.s) + __fmaf_rn(s, x.e, e * x.s);
    return t.settled();
  }
  // n as a pair too: from 2^24 on float32 does not hold it
  __device__ __forceinline__ Two over(int64_t n) const {
    const float high = float(n), low = float(n - int64_t(high));
    Two t;
    t.s = s / high;
    t.e = (__fmaf_rn(-t.s, high, s) + __fmaf_rn(-t.s, low, e)) / high;
    return t.settled();
  }
  __device__ __forceinline__ Two from_lane(int distance) const {
    Two t;
    t.s = __shfl_xor_sync(0xffffffffu, s, distance);
    t.e = __shfl_xor_sync(0xffffffffu, e, distance);
    return t;
  }
};
__device__ __forceinline__ Two two_of(const Pair32& v) {
  Two t;
  t.s = v.high, t.e = v.low;
  return t;
}
// Sums over `lanes` lanes, the first lane's to use: the others add in another order.
__device__ __forceinline__ Two sum_over(Two v, int lanes) {
  for (int o = lanes / 2; o > 0; o /= 2) v.add(v.from_lane(o));
  return v;
}
__device__ __forceinline__ int64_t sum_over(int64_t v, int lanes) {
  for (int o = lanes / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A sequence's sums over its counted rows, whole or of one chunk.
struct __align__(16) Sums {
  Two logp, ref;
  int64_t count, unused;
};
static_assert(sizeof(Sums) == 32, "two accesses of 16 bytes");
// What a CTA of the pairs' kernel adds to the call's sums.
struct Part {
  Two loss, nll, right, chosen, rejected;
  int64_t count;
};

// The sequences of pair i.
__device__ __forceinline__ int64_t chosen_of(const PreferenceArgs& a, int64_t i) {
  return a.halves ? i : 2 * i;
}
__device__ __forceinline__ int64_t rejected_of(const PreferenceArgs& a, int64_t i) {
  return a.halves ? i + a.n_sequences / 2 : 2 * i + 1;
}
// An offset, whatever it holds, as a row of the call.
__device__ __forceinline__ int row_of(const PreferenceArgs& a, int64_t i) {
  if (!LP_CHECK(i >= 0 && i <= a.n_sequences, kChkRowIndex)) return 0;
  return int(min(max(__ldg(a.cu_seqlens + i), int64_t(0)), a.T));
}

struct Pair {
  Part part;               // the pair's, all zeros when it does not count
  float chosen, rejected;  // d loss / d logp of a counted row, times the number of pairs
  float reward[2];
};
__device__ __forceinline__ Two score_of(const PreferenceArgs& a, const Sums& s) {
  Two v = s.logp;
  if (a.ref_logp != nullptr) v.add(s.ref.negative());
  return a.average && s.count > 0 ? v.settled().over(s.count) : v.settled();
}
__device__ __forceinline__ Two one(float x) {
  Two t;
  t.s = x;
  return t;
}
__device__ __forceinline__ Pair pair_of(const PreferenceArgs& a, const Sums& c, const Sums& r) {
  Pair p{};
  const Two sc = score_of(a, c), sr = score_of(a, r), beta = two_of(a.beta);
  const Two rc = beta.times(sc), rr = beta.times(sr);
  p.reward[0] = rc.value();
  p.reward[1] = rr.value();
  if (c.count == 0 || r.count == 0) return p;
  Two gap = sc;
  gap.add(sr.negative());
  gap = gap.settled();
  Two z = beta.times(gap);
  z.add(two_of(a.margin).negative());
  z = z.settled();
  float loss, slope;
  if (a.kind == LP_PREFERENCE_SIGMOID) {
    // exp(-|z|) of z's leading part, and the rest to first order
    const float high = fabsf(z.s), low = z.s < 0.f ? -z.e : z.e;
    const float e = expf(-high), small = e - e * low;
    const float log_part = log1pf(small), near = 1.f / (1.f + small), far = small * near;
    // softplus(-z), softplus(z), and their derivatives' sizes
    const float down = z.s > 0.f ? log_part : high + (low + log_part);
    const float up = z.s > 0.f ? high + (low + log_part) : log_part;
    const float to_down = z.s > 0.f ? far : near, to_up = z.s > 0.f ? near : far;
    const float rest = 1.f - a.smoothing;
    loss = slope = 0.f;  // an infinite term without a weight is none
    if (rest != 0.f) {
      loss = rest * down;
      slope = -rest * to_down;
    }
    if (a.smoothing != 0.f) {
      loss += a.smoothing * up;
      slope += a.smoothing * to_up;
    }
    if (z.s != z.s) loss = slope = z.s;
  } else if (a.kind == LP_PREFERENCE_HINGE) {
    Two left = one(1.f);
    left.add(z.negative());
    const float v = left.value();  // 1 - z
    loss = v > 0.f ? v : v != v ? v : 0.f;
    slope = v > 0.f ? -1.f : v != v ? v : 0.f;
  } else {
    z.add(-0.5f);
    const Two off = z.settled().times(two_of(a.inverse_beta));
    loss = off.s * off.s;
    slope = 2.f * off.s;  // dz is beta times a score's, and off is z over beta
  }
  if (a.kind != LP_PREFERENCE_SQUARE) slope *= a.beta.high;
  const float nc = float(c.count), nr = float(r.count);
  p.part.loss = one(loss);
  p.part.nll = one(-(c.logp.value() / nc));
  p.part.right = one(gap.s > 0.f ? 1.f : 0.f);
  p.part.chosen = rc;
  p.part.rejected = rr;
  p.part.count = 1;
  p.chosen = a.average ? slope / nc : slope;
  p.rejected = a.average ? -slope / nr : -slope;
  if (a.nll_coef != 0.f) p.chosen -= a.nll_coef / nc;
  return p;
}
__device__ __forceinline__ float weight_of(int64_t pairs) { return pairs > 0 ? 1.f / float(pairs) : 0.f; }
__device__ __forceinline__ void write_stats(const PreferenceArgs& a, const Part& s) {
  const int64_t n = s.count > 0 ? s.count : 1;
  const auto mean = [&](const Two& v) { return v.settled().over(n).value(); };
  const float loss = mean(s.loss), nll = mean(s.nll);
  // a likelihood term with a coefficient of 0 is watched only
  a.stats[0] = a.nll_coef != 0.f ? __fmaf_rn(a.nll_coef, nll, loss) : loss;
  a.stats[1] = loss;
  a.stats[2] = nll;
  a.stats[3] = mean(s.right);
  a.stats[4] = mean(s.chosen);
  a.stats[5] = mean(s.rejected);
}
__device__ __forceinline__ void add_part(Part& s, const Part& o) {
  s.loss.add(o.loss), s.nll.add(o.nll), s.right.add(o.right), s.chosen.add(o.chosen), s.rejected.add(o.rejected);
  s.count += o.count;
}
__device__ __forceinline__ Part sum_parts(Part s, int lanes) {
  s.loss = sum_over(s.loss, lanes);
  s.nll = sum_over(s.nll, lanes);
  s.right = sum_over(s.right, lanes);
  s.chosen = sum_over(s.chosen, lanes);
  s.rejected = sum_over(s.rejected, lanes);
  s.count = sum_over(s.count, lanes);
  return s;
}

// A few rows: a team of warps a sequence, a lane a pair.
__global__ void __launch_bounds__(kSmallThreads)
    lp_preference_small_kernel(const __grid_constant__ PreferenceArgs a, int team) {
  __shared__ Sums parts[kSmallThreads / 32];
  __shared__ Sums sums[kSmallSequences];
  __shared__ float slopes[kSmallSequences];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  const int n = int(a.n_sequences), teams = warps / team, mine = warp / team;
  const int first = int(threadIdx.x) - mine * team * 32, stride = team * 32;
  const int from = n > 0 ? row_of(a, 0) : 0, to = n > 0 ? row_of(a, n) : 0;
  int begin = 0, end = 0;  // the team's last sequence's rows
  for (int i0 = 0; i0 < n; i0 += teams) {
    const int i = i0 + mine;
    Two logp, ref;
    int64_t count = 0;
    if (i < n) {
      begin = row_of(a, i), end = row_of(a, i + 1);
      for (int t = begin + first; t < end; t += stride) {
        if (!LP_CHECK(t >= 0 && t < a.T, kChkRowIndex)) break;
        if (a.mask != nullptr && a.mask[t] == 0) continue;
        logp.add(a.logp[t]);
        if (a.ref_logp != nullptr) ref.add(a.ref_logp[t]);
        ++count;
      }
    }
    Sums s;
    s.logp = sum_over(logp, 32);
    s.ref = sum_over(ref, 32);
    s.count = sum_over(count, 32);
    if (lane == 0) parts[warp] = s;
    __syncthreads();
    if (int(threadIdx.x) < teams && i0 + int(threadIdx.x) < n) {
      Sums whole = parts[threadIdx.x * team];
      for (int k = 1; k < team; ++k) {
        const Sums& p = parts[threadIdx.x * team + k];
        whole.logp.add(p.logp), whole.ref.add(p.ref);
        whole.count += p.count;
      }
      if (LP_CHECK(i0 + int(threadIdx.x) < kSmallSequences, kChkStateIndex)) sums[i0 + threadIdx.x] = whole;
    }
    __syncthreads();
  }
  if (warp == 0) {
    Pair p{};
    const int64_t c = chosen_of(a, lane), r = rejected_of(a, lane);
    if (2 * lane < n) {
      p = pair_of(a, sums[c], sums[r]);
      a.rewards[c] = p.reward[0];
      a.rewards[r] = p.reward[1];
    }
    const Part whole = sum_parts(p.part, 32);
    const float w = weight_of(whole.count);
    if (2 * lane < n) slopes[c] = p.chosen * w, slopes[r] = p.rejected * w;
    if (lane == 0) write_stats(a, whole);
  }
  __syncthreads();
  for (int i = mine; i < n; i += teams) {
    const float g = slopes[i];
    if (n > teams) begin = row_of(a, i), end = row_of(a, i + 1);
    for (int t = begin + first; t < end; t += stride)
      if (LP_CHECK(t >= 0 && t < a.T, kChkRowIndex))
        a.grad_logp[t] = a.mask == nullptr || a.mask[t] != 0 ? g : 0.f;
  }
  for (int t = threadIdx.x; t < int(a.T); t += blockDim.x)  // rows in no sequence
    if (t < from || t >= to) a.grad_logp[t] = 0.f;
}

// The first of n ascending offsets that is above t, in [0, n], by a whole warp: 32 probes a step.
__device__ __forceinline__ int warp_upper_bound(const int64_t* offsets, int n, int t) {
  const unsigned lane = threadIdx.x & 31;
  unsigned lo = 0, hi = unsigned(n);  // the answer is in [lo, hi]
  while (lo < hi) {
    const unsigned stride = (hi - lo + 31) / 32, at = lo + lane * stride;
    const bool below = at < hi && __ldg(offsets + at) <= t;
    const unsigned k = __popc(__ballot_sync(0xffffffffu, below));  // the probes below t come first
    if (k == 0) break;
    hi = min(hi, lo + k * stride);
    lo += (k - 1) * stride + 1;
  }
  return int(lo);
}

// Four values of an operand; rows from T on read as zero.
__device__ __forceinline__ void load4(const float* p, int64_t t, int64_t T, bool wide, float (&v)[4]) {
  if (wide && t + 4 <= T) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p + t));
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = t + j < T ? p[t + j] : 0.f;
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

// The sequences that have rows in [t0, t1), in order, 32 at a time; all of a warp together.  Runs of empty ones are
// passed by a search (100000 of them between two answers took 1536 us 32 at a time, 19 so).
struct Cursor {
  int first;      // sequence of lane 0
  int lo, hi;     // the lane's sequence's rows, counted from t0
  unsigned some;  // the lanes whose sequence has any
  bool more;      // whether the next 32 may have some
  __device__ __forceinline__ Cursor(const PreferenceArgs& a, int t0, int t1)
      : first(warp_upper_bound(a.cu_seqlens + 1, int(a.n_sequences), t0)) {
    look(a, t0, t1);
  }
  __device__ __forceinline__ void look(const PreferenceArgs& a, int t0, int t1) {
    const int lane = threadIdx.x & 31;
    const bool there = lane < int(a.n_sequences) - first;
    int begin = t1, end = t1;
    if (there) begin = row_of(a, first + int64_t(lane)), end = row_of(a, first + int64_t(lane) + 1);
    lo = max(begin, t0) - t0;
    hi = min(end, t1) - t0;
    some = __ballot_sync(0xffffffffu, there && begin < t1 && lo < hi);
    more = __all_sync(0xffffffffu, there && end < t1);
  }
  // f(i, lo, hi) for every sequence i, with its rows
  template <class F>
  __device__ __forceinline__ void each(const PreferenceArgs& a, int t0, int t1, F&& f) {
    while (true) {
      // where the rows passed so far end, if all 32 are empty: behind them the next one with rows is searched for
      const bool none = some == 0;
      for (; some != 0; some &= some - 1) {
        const int k = __ffs(some) - 1;
        f(first + k, __shfl_sync(0xffffffffu, lo, k), __shfl_sync(0xffffffffu, hi, k));
      }
      if (!more) return;
      const int passed = t0 + max(__shfl_sync(0xffffffffu, hi, 31), 0);
      first += 32;  // whatever the offsets hold, the search goes on
      if (none) first = max(first, warp_upper_bound(a.cu_seqlens + 1, int(a.n_sequences), passed));
      look(a, t0, t1);
    }
  }
};
// The first row of a warp's chunk, T past the last one.
__device__ __forceinline__ int chunk_begin(const PreferenceArgs& a, int64_t chunk) {
  return int(min(chunk * kChunk, a.T));
}
__device__ __forceinline__ int chunk_end(const PreferenceArgs& a, int t0) { return int(min(int64_t(t0) + kChunk, a.T)); }

// The place of a sequence's sums over a chunk: both go up along the rows, so no two meet.
__device__ __forceinline__ int64_t slot_of(int64_t chunk, int64_t sequence) { return chunk + sequence; }

__global__ void __launch_bounds__(kThreads, 8)
    lp_preference_sums_kernel(const __grid_constant__ PreferenceArgs a, Sums* slots, int64_t n_slots) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t chunk = int64_t(blockIdx.x) * kWarps + threadIdx.x / 32;
  const int t0 = chunk_begin(a, chunk), t1 = chunk_end(a, t0);
  if (t0 >= t1) return;
  float logp[kGroups][4], ref[kGroups][4];
  unsigned kept[kGroups];
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int64_t t = t0 + int64_t(128 * k + 4 * lane);
    if (!LP_CHECK(t >= 0, kChkRowIndex)) return;
    load4(a.logp, t, a.T, a.wide, logp[k]);
    if (a.ref_logp != nullptr) load4(a.ref_logp, t, a.T, a.wide, ref[k]);
    kept[k] = load_mask4(a.mask, t, a.T, a.wide);
  }
  Cursor cursor(a, t0, t1);
  cursor.each(a, t0, t1, [&](int i, int lo, int hi) {
    Two x, y;
    int count = 0;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      if (128 * (k + 1) <= lo || 128 * k >= hi) continue;  // the same for the warp
      unsigned in = kept[k];
      if (128 * k < lo || 128 * (k + 1) > hi) {  // some of these rows are others'
        const int from = lo - (128 * k + 4 * lane), to = hi - (128 * k + 4 * lane);
        if (from > 0) in &= from >= 4 ? 0u : ~0u << from;
        if (to < 4) in &= to <= 0 ? 0u : (1u << to) - 1u;
      }
      count += __popc(in);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x.add(in >> j & 1u ? logp[k][j] : 0.f);
        if (a.ref_logp != nullptr) y.add(in >> j & 1u ? ref[k][j] : 0.f);
      }
    }
    Sums s;
    s.logp = sum_over(x, 32);
    if (a.ref_logp != nullptr) s.ref = sum_over(y, 32);
    s.count = __reduce_add_sync(0xffffffffu, count);
    const int64_t at = slot_of(chunk, i);
    if (lane == 0 && LP_CHECK(at >= 0 && at < n_slots, kChkStateIndex)) slots[at] = s;
  });
}

// Chunks of a lane from which on a pair is its whole warp's: what four turns of fold take.
constexpr int kFewChunks = 8;

// Adds up, over `lanes` lanes, the chunks of a pair's sequences, in the slots from `at` to `end`, a lane's share of
// each: both sequences side by side, two turns at once, since the loads are most of the time.
__device__ __forceinline__ void fold(const Sums* slots, int64_t n_slots, const int64_t (&first)[2],
                                     const int64_t (&end)[2], int lane, int lanes, Sums (&sums)[2]) {
  int64_t at[2] = {first[0] + lane, first[1] + lane};
  while (at[0] < end[0] || at[1] < end[1]) {
    float4 v[2][2];
    long long count[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t slot = at[k] + q * lanes;
        v[k][q] = make_float4(0.f, 0.f, 0.f, 0.f);
        count[k][q] = 0;
        if (slot >= end[k] || !LP_CHECK(slot >= 0 && slot < n_slots, kChkStateIndex)) continue;
        v[k][q] = __ldcg(reinterpret_cast<const float4*>(slots + slot));
        count[k][q] = __ldcg(reinterpret_cast<const long long*>(&slots[slot].count));
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        Two logp, ref;
        logp.s = v[k][q].x, logp.e = v[k][q].y, ref.s = v[k][q].z, ref.e = v[k][q].w;
        sums[k].logp.add(logp);
        sums[k].ref.add(ref);
        sums[k].count += count[k][q];
      }
      at[k] += 2 * lanes;
    }
  }
}
__device__ __forceinline__ Sums sum_over(const Sums& v, int lanes) {
  Sums s;
  s.logp = sum_over(v.logp, lanes);
  s.ref = sum_over(v.ref, lanes);
  s.count = sum_over(v.count, lanes);
  return s;
}
__device__ __forceinline__ Two from_first_lane(const Two& v) {
  Two t;
  t.s = __shfl_sync(0xffffffffu, v.s, 0);
  t.e = __shfl_sync(0xffffffffu, v.e, 0);
  return t;
}

// `lanes` lanes a pair (a power of two), as many as sequences of the mean length have chunks.  Pairs of sequences far
// longer than that are left to the whole warp, one after the other: one answer of 131072 among 20000 pairs of up to 100
// took 112 us by one lane, 41 so, 38 without it; one of 2^20 among 2000 pairs of 16 564 us and 60.
__global__ void __launch_bounds__(kPairThreads)
    lp_preference_pairs_kernel(const __grid_constant__ PreferenceArgs a, const Sums* slots, int64_t n_slots,
                               int lanes, float* slopes, Part* parts) {
  __shared__ Part of_warp[kPairThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = int(threadIdx.x) & 31, sub = lane % lanes;
  const int64_t pair = (int64_t(blockIdx.x) * kPairThreads + threadIdx.x) / lanes;
  const bool there = 2 * pair < a.n_sequences;
  const int64_t both[2] = {chosen_of(a, pair), rejected_of(a, pair)};
  int64_t first[2] = {0, 0}, end[2] = {0, 0};  // slots
  bool is_long = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!there) continue;
    const int begin_row = row_of(a, both[k]), end_row = row_of(a, both[k] + 1);
    if (begin_row >= end_row) continue;
    first[k] = slot_of(begin_row / kChunk, both[k]);
    end[k] = slot_of((end_row - 1) / kChunk, both[k]) + 1;
    is_long = is_long || end[k] - first[k] > kFewChunks * lanes;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the sums are done
  Sums sums[2] = {};
  is_long = is_long && lanes < 32;
  if (!is_long) fold(slots, n_slots, first, end, sub, lanes, sums);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 2; ++k) sums[k] = sum_over(sums[k], lanes);
  for (unsigned left = __ballot_sync(0xffffffffu, is_long && sub == 0); left != 0; left &= left - 1) {
    const int of = __ffs(left) - 1;
    int64_t from[2], to[2];
    Sums whole[2] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k)
      from[k] = __shfl_sync(0xffffffffu, first[k], of), to[k] = __shfl_sync(0xffffffffu, end[k], of);
    fold(slots, n_slots, from, to, lane, 32, whole);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      whole[k] = sum_over(whole[k], 32);
      whole[k].logp = from_first_lane(whole[k].logp);
      whole[k].ref = from_first_lane(whole[k].ref);
      if (lane == of) sums[k] = whole[k];
    }
  }
  Pair p{};
  if (there && sub == 0) {
    p = pair_of(a, sums[0], sums[1]);
    if (LP_CHECK(both[0] < a.n_sequences && both[1] < a.n_sequences, kChkRowIndex)) {
      a.rewards[both[0]] = p.reward[0];
      a.rewards[both[1]] = p.reward[1];
      slopes[both[0]] = p.chosen;
      slopes[both[1]] = p.rejected;
    }
  }
  const Part s = sum_parts(p.part, 32);
  if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  Part whole = of_warp[0];
#pragma unroll
  for (int k = 1; k < kPairThreads / 32; ++k) {
    add_part(whole, of_warp[k]);
  }
  parts[blockIdx.x] = whole;
}

__global__ void __launch_bounds__(kThreads, 12)
    lp_preference_rows_kernel(const __grid_constant__ PreferenceArgs a, const float* slopes, const Part* parts,
                              int64_t n_parts) {
  __shared__ int64_t counts[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int t0 = chunk_begin(a, int64_t(blockIdx.x) * kWarps + warp), t1 = chunk_end(a, t0);
  unsigned kept[kGroups];
#pragma unroll
  for (int k = 0; k < kGroups; ++k)
    kept[k] = load_mask4(a.mask, t0 + int64_t(128 * k + 4 * lane), a.T, a.wide);
  Cursor cursor(a, t0, t1);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the pairs are done
  int64_t count = 0;
  for (int64_t i = threadIdx.x; i < n_parts; i += kThreads)
    count += __ldcg(reinterpret_cast<const long long*>(&parts[i].count));
  count = sum_over(count, 32);
  if (lane == 0) counts[warp] = count;
  __syncthreads();
  count = 0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) count += counts[k];
  if (blockIdx.x == 0 && warp == 0) {
    Part s{};
    for (int64_t i = lane; i < n_parts; i += 32) add_part(s, parts[i]);
    s = sum_parts(s, 32);
    s.count = count;
    if (lane == 0) write_stats(a, s);
  }
  if (t0 >= t1) return;
  const float w = weight_of(count);
  float g[kGroups][4] = {};  // rows in no sequence have none
  cursor.each(a, t0, t1, [&](int i, int lo, int hi) {
    if (!LP_CHECK(i >= 0 && i < a.n_sequences, kChkStateIndex)) return;
    const float slope = __ldcg(slopes + i) * w;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      if (128 * (k + 1) <= lo || 128 * k >= hi) continue;  // the same for the warp
      const int r = 128 * k + 4 * lane;
      const bool whole = 128 * k >= lo && 128 * (k + 1) <= hi;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (whole || (r + j >= lo && r + j < hi)) g[k][j] = kept[k] >> j & 1u ? slope : 0.f;
    }
  });
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int64_t t = t0 + int64_t(128 * k + 4 * lane);
    if (!LP_CHECK(t >= 0, kChkRowIndex)) return;
    if (a.wide && t + 4 <= a.T) {
      *reinterpret_cast<float4*>(a.grad_logp + t) = make_float4(g[k][0], g[k][1], g[k][2], g[k][3]);
      continue;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t + j < a.T) a.grad_logp[t + j] = g[k][j];
  }
}

bool one_cta(int64_t T, int64_t n) { return T <= kSmallRows && n <= kSmallSequences; }

// The workspace of the three launches.
struct Layout {
  int64_t chunks, slots, parts;
  int lanes;
  size_t slopes_at, parts_at, bytes;
};
Layout layout_of(int64_t T, int64_t n) {
  Layout l;
  l.chunks = (T + kChunk - 1) / kChunk;
  l.slots = l.chunks + n;
  // lanes of a pair: one for each chunk of a sequence of the mean length
  const int64_t pieces = T / (kChunk * std::max<int64_t>(n, 1)) + 1;
  l.lanes = 1;
  while (l.lanes < 32 && l.lanes < pieces) l.lanes *= 2;
  l.parts = (n / 2 * l.lanes + kPairThreads - 1) / kPairThreads;
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  l.slopes_at = up(size_t(l.slots) * sizeof(Sums));
  l.parts_at = l.slopes_at + up(size_t(n) * sizeof(float));
  l.bytes = l.parts_at + up(size_t(l.parts) * sizeof(Part));
  return l;
}

template <class... Params, class... Args>
bool launch_dependent(void (*kernel)(Params...), int64_t blocks, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = stream;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

}  // namespace

size_t preference_loss_workspace(int64_t T, int64_t n_sequences) {
  return one_cta(T, n_sequences) ? 256 : layout_of(T, n_sequences).bytes;
}

lp_status launch_preference_loss(const PreferenceArgs& args, cudaStream_t stream) {
  PreferenceArgs a = args;
  const auto at16 = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  a.wide = at16(a.logp) && at16(a.ref_logp) && at16(a.grad_logp) &&
           reinterpret_cast<uintptr_t>(a.mask) % 4 == 0;
  if (one_cta(a.T, a.n_sequences)) {
    // as many warps as there are rows for, a power of two of them a sequence
    int warps = 1, team = 1;
    while (warps < kSmallThreads / 32 && (warps * 32 < a.T || warps < a.n_sequences)) warps *= 2;
    while (2 * team * std::max<int64_t>(a.n_sequences, 1) <= warps) team *= 2;
    lp_preference_small_kernel<<<1, warps * 32, 0, stream>>>(a, std::min(team, warps));
    return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
  }
  const Layout l = layout_of(a.T, a.n_sequences);
  char* ws = static_cast<char*>(a.workspace);
  Sums* slots = reinterpret_cast<Sums*>(ws);
  float* slopes = reinterpret_cast<float*>(ws + l.slopes_at);
  Part* parts = reinterpret_cast<Part*>(ws + l.parts_at);
  const int64_t blocks = std::max<int64_t>(1, (l.chunks + kWarps - 1) / kWarps);
  lp_preference_sums_kernel<<<unsigned(blocks), kThreads, 0, stream>>>(a, slots, l.slots);
  if (cudaGetLastError() != cudaSuccess) return LP_ERR_CUDA;
  if (l.parts > 0 &&
      !launch_dependent(lp_preference_pairs_kernel, l.parts, kPairThreads, stream, a,
                        static_cast<const Sums*>(slots), l.slots, l.lanes, slopes, parts))
    return LP_ERR_CUDA;
  if (!launch_dependent(lp_preference_rows_kernel, blocks, kThreads, stream, a,
                        static_cast<const float*>(slopes), static_cast<const Part*>(parts), l.parts))
    return LP_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

cudaError_t take_check_word_preference(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
