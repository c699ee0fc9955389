// lp_muon.cu: one step of Muon over many matrices (include/lp_tune.h).
//
// A matrix is taken as X of m <= n, transposed where it is tall.  Every Newton-Schulz step is three
// products, each one launch over the tiles of all matrices of a batch:
//     G = X X^T                      symmetric: the tiles on and below the diagonal
//     P = a I + b G + c G G          symmetric too, from G in the same way
//     X = P X
// Operands are pairs of float16, x = hi + lo (22 bits), scaled by 2^14, which holds them inside
// float16's range: after the division by the Frobenius norm no singular value passes 1.21 (the
// polynomial's largest value on [0, 1]), so no element of X, G or P passes 3.45.  (Where eps leaves X
// small, a power of two more keeps its bits; an element below 2^-16 of the norm has fewer than 22, to 2^-39
// of the norm.)  A product is hi hi + hi lo + lo hi with float32 accumulators (lo lo is 2^-22 of it):
// three tensor-core products where one of float16 would lose what a step multiplies by 3.4 in the
// small singular directions, five times over.  (tests/test_gpu_muon.py derives what is left.)
//
// The pairs lie in memory as the tensor core reads them from shared memory: blocks of 128 x 64
// with 128-byte swizzled rows, 16 KB of hi and 16 KB of lo side by side, so a tile is fetched as
// plain rows of 128 bytes, and the same block serves as a K-major operand (G) and as an N-major one
// (P X).  Of G and P the blocks above the diagonal are never written: they are read where they mirror
// to, as M- or N-major operands.
//
// A CTA takes tiles of 128 x 128 in turn: one warp fetches stages of 64 of K (64 KB), one issues the
// products, hi x [hi; lo] as one of N = 256, then lo x hi onto its second half, and eight warps, half
// a row of the tile a thread, take finished chunks of K out of tensor memory, two of which alternate,
// and add them up in registers.
//
// Bound by the tensor cores and their power: 4096 x 4096 takes 2.8 to 3.1 ms a step, of which the
// three products of each float16 pair cannot do without 2.14 ms at the measured bfloat16 rate; the
// last of 528 tiles' turns on 152 SMs costs a tenth of it.  The tensor pipe is active for 56 to 58% of
// the products' time at 2048 x 2048 (442 us a step), where the symmetric products have 136 tiles for
// 152 SMs; the fetches alone take 2.2 ms at 4096 x 4096, the products alone 2.6 to 2.8.  Small
// matrices are bound by their 17 dependent launches, 6 to 7 us each: four of 256 x 256 118 us.
// Pairs of CTAs with tiles of 256 x 128 were no faster, tiles of 256 x 256 had no room in tensor memory
// for two accumulators of every term; orders of the tiles by groups gained nothing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <vector>

#include "lp_check.cuh"
#include "lp_tcgen05.cuh"
#include "lp_tune_internal.h"

namespace lp {
namespace {

using namespace tc;

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScale = 16384.f;           // of the operands
constexpr float kUnscale = 1.f / kScale;
// X is held times 2^e besides, which takes its norm |u| / (|u| + eps) to 1/2 and above: an eps far above |u|
// would leave its elements among float16's subnormals, and five steps multiply what they lose by 485.  No step
// grows X by more than kA < 2^1.7844, so that e comes down with the steps and X stays below what it has without.
constexpr int kMaxExponent = 60;
__device__ __forceinline__ int exponent_of(float norm, float eps) {
  const float share = norm / (norm + eps);
  return share > 0.f ? min(max(-1 - ilogbf(share), 0), kMaxExponent) : 0;
}
__device__ __forceinline__ int exponent_at(int first, int step) { return max(first - (17844 * step + 9999) / 10000, 0); }
__device__ __forceinline__ float power_of_2(int e) { return __int_as_float((e + 127) << 23); }  // |e| <= 126
// From this exponent on b G and c G G are below 2^-28 of a I, and P is a I.
constexpr int kLinear = 15;

constexpr int kTile = 128;                  // rows and columns of a tile, rows of a block
constexpr int kBlockK = 64;                 // columns of a block, K of a stage
constexpr uint32_t kHalf = kTile * kBlockK * 2;  // bytes of a block's hi (or lo) part
constexpr uint32_t kBlock = 2 * kHalf;
// K blocks that are summed in tensor memory before the sum is added to the tile's in registers.  The
// tensor core cuts sums off where an addition would round: over K of 1000 the singular values came
// out 8e-6 off, five times what float32 products give; in chunks it is what 32 of its steps cut off.  That is
// always downwards: where a gradient's rows are of one sign, it adds up to 1e-5 of X (float32 products 2e-6).
constexpr int kChunk = 8;
// K blocks from which on a tile's K is in segments: 1024 x 1024 takes 183 us with four, 201 with one; 64
// such matrices, which need no split, 3.7 ms and 3.5.  (The bits are not to depend on the company.)
constexpr int kSplitBlocks = 16;
constexpr uint32_t kAccumulator = 2 * kTile;     // tensor-memory columns
constexpr int kOutThreads = 256;                 // of the epilogue: two a row of the tile
constexpr int kOutWarps = kOutThreads / 32;
constexpr int kProductThreads = 128 + kOutThreads;
// Registers of a thread: what the launch gives, and how the epilogue's two warpgroups, which hold the
// tile's sums, take from the other: 56 + 2 * 224 = 3 * 168.
constexpr int kFewRegisters = 56, kManyRegisters = 224;
constexpr int kNormThreads = 256;
constexpr int kSplitThreads = 256;

enum Product { kGram, kPoly, kApply };

// The word of the workspace's header that says, behind the four that are read back, whether a wait of the batch
// has given up.
constexpr int kBatchError = 4;

// A record's buffers in the workspace.
__device__ __forceinline__ int64_t block_at(int64_t row_block, int64_t col_block, int64_t col_blocks) {
  return (row_block * col_blocks + col_block) * int64_t(kBlock);
}
__host__ __device__ __forceinline__ int64_t padded_to(int64_t v, int64_t by) { return (v + by - 1) / by * by; }

// ------------------------------------------------------------------ momentum, norm, X

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
// f(gradient's pointer of its type)
template <class F>
__device__ __forceinline__ void with_grad(const MuonRecord& t, F&& f) {
  if (t.grad_bf16)
    f(static_cast<const __nv_bfloat16*>(t.grad));
  else
    f(static_cast<const float*>(t.grad));
}
// The new momentum and what is orthogonalised.
__device__ __forceinline__ float momentum_of(const MuonArgs& a, float g, float m) {
  return __fmaf_rn(a.momentum, m, g);
}
__device__ __forceinline__ float update_of(const MuonArgs& a, float g, float m) {
  return a.nesterov ? __fmaf_rn(a.momentum, m, g) : m;
}

// Four neighbouring elements of the gradient, and of the momentum, at once.
__device__ __forceinline__ void load_wide(const __nv_bfloat16* p, float* v) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xffff0000u);
  v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xffff0000u);
}
__device__ __forceinline__ void load_wide(const float* p, float* v) {
  const float4 w = *reinterpret_cast<const float4*>(p);
  v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
}
// The sum of a value over the CTA's 256 threads, the same bits for all of them.
__device__ __forceinline__ float sum256(float s, float* slots) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x / 32] = s;
  __syncthreads();
  s = slots[threadIdx.x & 7];
#pragma unroll
  for (int o = 4; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// The squares' sum of a part of a matrix.
__global__ void __launch_bounds__(kNormThreads)
    lp_muon_norm_kernel(const __grid_constant__ MuonArgs a, const MuonUnit* units, float* partials, int first) {
  __shared__ float slots[kNormThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the words that are read back, of all batches, and the batch's own
  if (blockIdx.x == 0 && threadIdx.x <= kBatchError && (first || threadIdx.x == kBatchError)) a.err[threadIdx.x] = 0u;
  const MuonUnit u = units[blockIdx.x];
  if (!LP_CHECK(u.tensor >= 0 && u.tensor < a.n_tensors, kChkPlan)) return;
  const MuonRecord t = a.records[u.tensor];
  const int64_t n = t.rows * t.cols, from = int64_t(u.part) * t.part;
  if (!LP_CHECK(from >= 0 && from < n, kChkCopyIndex)) return;
  const int count = int(min(t.part, n - from));
  constexpr int kTurn = 4;  // groups of four elements of a thread at once
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  with_grad(t, [&](const auto* grad) {
    for (int first_of = 4 * int(threadIdx.x); first_of < count; first_of += kTurn * 4 * kNormThreads) {
      float g[kTurn][4], m[kTurn][4];
#pragma unroll
      for (int k = 0; k < kTurn; ++k) {
        const int at = first_of + k * 4 * kNormThreads;
        if (t.wide && at + 4 <= count) {
          load_wide(grad + from + at, g[k]);
          load_wide(t.momentum + from + at, m[k]);
          continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g[k][j] = at + j < count ? to_float(grad[from + at + j]) : 0.f;
          m[k][j] = at + j < count ? t.momentum[from + at + j] : 0.f;
        }
      }
#pragma unroll
      for (int k = 0; k < kTurn; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x = update_of(a, g[k][j], momentum_of(a, g[k][j], m[k][j]));
          sum[j] = __fmaf_rn(x, x, sum[j]);
        }
    }
  });
  const float s = sum256((sum[0] + sum[1]) + (sum[2] + sum[3]), slots);
  if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

// hi and lo of eight scaled values, as a block holds them.
__device__ __forceinline__ void split8(const float (&v)[8], uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 two = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    const float2 back = __half22float2(two);
    const __half2 rest = __floats2half2_rn(v[2 * i] - back.x, v[2 * i + 1] - back.y);
    h[i] = *reinterpret_cast<const uint32_t*>(&two);
    l[i] = *reinterpret_cast<const uint32_t*>(&rest);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// Where columns 8 chunk .. 8 chunk + 7 of row r lie in a block's half.
__device__ __forceinline__ uint32_t chunk_at(int r, int chunk) {
  return uint32_t(r) * 128u + (uint32_t(chunk ^ (r & 7)) << 4);
}

// A block of the first X, and the new momentum of its elements.  A thread has four groups of eight columns;
// their loads are all on their way before the norm is there.  (float64 for the norm's last steps, 1/64 of the
// rate, took longer than the block.)
__global__ void __launch_bounds__(kSplitThreads, 2)
    lp_muon_split_kernel(const __grid_constant__ MuonArgs a, const MuonUnit* units, const float* partials) {
  constexpr int kGroups = kTile * kBlockK / 8 / kSplitThreads;
  __shared__ float slots[kSplitThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const MuonUnit u = units[blockIdx.x];
  if (!LP_CHECK(u.tensor >= 0 && u.tensor < a.n_tensors, kChkPlan)) return;
  const MuonRecord t = a.records[u.tensor];
  // Neighbouring threads go along the matrix's rows, which are X's columns where it is tall.  A thread's next
  // group is 32 rows on, or 16 columns.
  const int tid = int(threadIdx.x);
  const int r = t.tall ? tid % kTile : tid / 8, chunk = t.tall ? tid / kTile : tid % 8;
  const int next_r = t.tall ? 0 : kSplitThreads / 8, next_chunk = t.tall ? kSplitThreads / kTile : 0;
  const int rows_left = int(t.m - int64_t(u.i) * kTile) - r, cols_left = int(t.n - int64_t(u.j) * kBlockK) - 8 * chunk;
  const int64_t row = int64_t(u.i) * kTile + r, col = int64_t(u.j) * kBlockK + 8 * chunk;
  const int64_t at = t.tall ? col * t.cols + row : row * t.cols + col, step = t.tall ? t.cols : 1;
  const int64_t next = (t.tall ? 8 * next_chunk : next_r) * t.cols;
  const auto left_of = [&](int k) {  // columns of group k
    return k * next_r < rows_left ? min(max(cols_left - 8 * k * next_chunk, 0), 8) : 0;
  };
  const bool wide = !t.tall && t.wide;
  float g[kGroups][8], m[kGroups][8];
  with_grad(t, [&](const auto* grad) {
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int left = left_of(k);
      const int64_t i = at + k * next;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[k][j] = m[k][j] = 0.f;
      if (!LP_CHECK(left == 0 || (i >= 0 && i + (left - 1) * step < t.rows * t.cols), kChkCopyIndex)) continue;
      if (wide) {
        if (left == 8)
#pragma unroll
          for (int q = 0; q < 8; q += 4) load_wide(grad + i + q, g[k] + q), load_wide(t.momentum + i + q, m[k] + q);
        else
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < left) g[k][j] = to_float(grad[i + j]), m[k][j] = t.momentum[i + j];
        continue;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) g[k][j] = to_float(grad[i + j * step]), m[k][j] = t.momentum[i + j * step];
    }
  });
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are written
  float s = 0.f;
  for (int k = tid; k < int(t.parts); k += kSplitThreads) s += __ldcg(partials + t.first_part + k);
  const float norm = sqrtf(sum256(s, slots));
  const bool fine = norm <= 0x1.fffffep127f;
  const int exponent = fine ? exponent_of(norm, a.eps) : 0;
  if (u.i == 0 && u.j == 0 && tid == 0) a.levels[u.tensor] = fine ? 1 + exponent : 0;
  const float scale = kScale * power_of_2(exponent) / (norm + a.eps);
  unsigned char* block = a.workspace + t.x[0] + block_at(u.i, u.j, padded_to(t.n, kTile) / kBlockK);
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int left = left_of(k);
    const int64_t i = at + k * next;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[k][j] = momentum_of(a, g[k][j], m[k][j]);
      v[j] = fine ? update_of(a, g[k][j], m[k][j]) * scale : 0.f;
    }
    uint4 hi, lo;
    split8(v, hi, lo);
    const uint32_t in = chunk_at(r + k * next_r, chunk + k * next_chunk);
    *reinterpret_cast<uint4*>(block + in) = hi;
    *reinterpret_cast<uint4*>(block + kHalf + in) = lo;
    if (!fine || !LP_CHECK(left == 0 || (i >= 0 && i + (left - 1) * step < t.rows * t.cols), kChkCopyIndex)) continue;
    if (wide && left == 8) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<float4*>(t.momentum + i + 4 * q) =
            make_float4(m[k][4 * q], m[k][4 * q + 1], m[k][4 * q + 2], m[k][4 * q + 3]);
      continue;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) t.momentum[i + j * step] = m[k][j];
  }
}

// ------------------------------------------------------------------------- products

// A stage of the ring: 64 of K of A's and of B's tile.
constexpr int kStages = 3;
constexpr uint32_t kStage = 2 * kBlock;
constexpr int kBars = 2 * kStages + 6;
constexpr uint32_t kOut = kStages * kStage;  // the epilogue's 32 KB
constexpr int kSmem = 1024 + int(kOut + kBlock) + kBars * 8 + 16;
static_assert(kSmem <= 232448, "shared memory of a CTA");

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// kind::f16 with float16 operands and float32 accumulators, M = 128; bits 15 and 16 say that A and B are M-
// and N-major.
__host__ __device__ constexpr uint32_t idesc_half(int n) {
  return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(kTile >> 4) << 24);
}

// 32 consecutive columns of this thread's tensor-memory lane; tmem_wait before they are used.
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Where a unit's operands lie, in rows of 128 bytes of the workspace.
constexpr int kRow = 128;
constexpr int kBlockRows = int(kBlock) / kRow;
struct Operands {
  int a, b;                // A and B (of X X^T and G G, the same)
  int a_blocks, b_blocks;  // blocks of a row of blocks
  int k_blocks;
};
template <int kProduct>
__device__ __forceinline__ Operands operands_of(const MuonRecord& t, int from) {
  const int x_blocks = int(padded_to(t.n, kTile)) / kBlockK, g_blocks = int(padded_to(t.m, kTile)) / kBlockK;
  const int x = int(t.x[from] / kRow), g = int(t.g / kRow), p = int(t.p / kRow);
  const int k = int(((kProduct == kGram ? t.n : t.m) + kBlockK - 1) / kBlockK);
  if (kProduct == kGram) return {x, x, x_blocks, x_blocks, k};
  if (kProduct == kPoly) return {g, g, g_blocks, g_blocks, k};
  return {p, x, g_blocks, x_blocks, k};
}
// K in segments, by its length alone, whose sums are added in order: a tile's bits are the same whether one CTA
// goes through them or each is another CTA's.
constexpr int kSplits = 4;
struct Segments {
  int blocks, shift;
  __device__ __forceinline__ explicit Segments(int k_blocks) : blocks(k_blocks), shift(k_blocks >= kSplitBlocks ? 2 : 0) {}
  __device__ __forceinline__ int count() const { return 1 << shift; }
  __device__ __forceinline__ int begin(int s) const { return s * blocks >> shift; }
  // those of a CTA: all, or of a cluster each CTA one
  template <bool kSplit>
  __device__ __forceinline__ int first(uint32_t rank) const { return kSplit ? min(int(rank), count()) : 0; }
  template <bool kSplit>
  __device__ __forceinline__ int last(uint32_t rank) const { return kSplit ? min(int(rank) + 1, count()) : count(); }
};
static_assert(kSplits == 1 << 2, "the shift");
// G and P are symmetric, and only the blocks of their tiles on and below the diagonal are written.  Whether
// columns 64 kb on of row block i lie above it: they are then read where they mirror to, as an operand that is
// contiguous along M or N.
__device__ __forceinline__ bool mirrored(int i, int kb) { return kb / 2 > i; }

// Whether `go` holds for all of the epilogue's warps.
__device__ __forceinline__ bool epilogue_all(int go) {
  int all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 256, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(go)
      : "memory");
  return all != 0;
}
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void bulk_store(void* to, uint32_t from, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(from), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ uint32_t half2_of(float x, float y) {
  const __half2 two = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&two);
}
// hi of two values, or lo: what hi leaves.
__device__ __forceinline__ uint32_t part_of(float x, float y, bool lo) {
  const uint32_t h = half2_of(x, y);
  if (!lo) return h;
  const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return half2_of(x - back.x, y - back.y);
}

// The tile, of which x holds 64 columns from column 64 half on of the thread's row r, into its two blocks:
// first the hi parts of both, then the lo parts, through shared memory.
__device__ __forceinline__ void write_tile(const float (&x)[kTile / 2], int r, int half, unsigned char* to,
                                           uint8_t* out, bool first_thread) {
  const uint32_t out_at = smem_u32(out);
#pragma unroll
  for (int lo = 0; lo < 2; ++lo) {
    if (first_thread) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the buffer is free
    epilogue_sync();
#pragma unroll
    for (int q = 0; q < kTile / 16; ++q) {
      uint4 v;
      v.x = part_of(x[8 * q], x[8 * q + 1], lo);
      v.y = part_of(x[8 * q + 2], x[8 * q + 3], lo);
      v.z = part_of(x[8 * q + 4], x[8 * q + 5], lo);
      v.w = part_of(x[8 * q + 6], x[8 * q + 7], lo);
      *reinterpret_cast<uint4*>(out + half * kHalf + chunk_at(r, q)) = v;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    epilogue_sync();
    if (first_thread) {
#pragma unroll
      for (int q = 0; q < 2; ++q) bulk_store(to + q * int64_t(kBlock) + lo * kHalf, out_at + q * kHalf, kHalf);
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
}

// The step's last product: the parameters from the 64 columns in x, rows `row` on and columns `col` on of X,
// lanes along the parameters' rows.  The record's entries are read before the first store, which might be to
// them as far as the compiler knows, and all loads of a turn are on their way before its first store: with
// both left to the compiler a tile took 35 us.  slots: 4 KB of the warp's own.
__device__ __forceinline__ void write_params(const MuonArgs& a, const MuonRecord& t, bool fine, float unscale, int row,
                                             int col, int lane, const float (&x)[kTile / 2], float* slots, bool poison) {
  if (!fine) return;
  const double l = a.lr * double(t.lr_scale);
  const float keep = float(1.0 - l * double(t.weight_decay));
  const float rate = poison ? __int_as_float(0x7fc00000)
                            : float(l * double(t.update_scale)) * unscale;
  const bool tall = t.tall != 0;
  const int64_t cols = t.cols;
  // X's rows and columns from here on; lanes go along `across`
  const int rows_left = int(t.m) - row, cols_left = int(t.n) - col;
  if (!LP_CHECK(row >= 0 && col >= 0 && rows_left <= t.m, kChkOutBox)) return;
  float* const param = t.param + (tall ? int64_t(col) * cols + row : int64_t(row) * cols + col) + lane;
  __nv_bfloat16* copy = t.copy;
  if (copy != nullptr) copy += param - t.param;
  constexpr int kTurn = 16;
  // `n` rows of the parameters, a lane's element of each: their loads, then their stores
  const auto turn = [&](float* p, __nv_bfloat16* c, int n, const float (&v)[kTurn]) {
    float old[kTurn];
#pragma unroll
    for (int j = 0; j < kTurn; ++j) old[j] = j < n ? p[j * cols] : 0.f;
#pragma unroll
    for (int j = 0; j < kTurn; ++j) old[j] = __fmaf_rn(-rate, v[j], old[j] * keep);
#pragma unroll
    for (int j = 0; j < kTurn; ++j)
      if (j < n) p[j * cols] = old[j];
    if (c == nullptr) return;
#pragma unroll
    for (int j = 0; j < kTurn; ++j)
      if (j < n) c[j * cols] = __float2bfloat16_rn(old[j]);
  };
  if (tall) {  // X's rows are the parameters' columns: so are the lanes
    const bool mine = lane < rows_left;
#pragma unroll
    for (int c = 0; c < kTile / 2; c += kTurn) {
      float v[kTurn];
#pragma unroll
      for (int j = 0; j < kTurn; ++j) v[j] = x[c + j];
      turn(param + c * cols, copy != nullptr ? copy + c * cols : nullptr, mine ? cols_left - c : 0, v);
    }
    return;
  }
  // a warp's 32 rows, 32 columns at a time, through shared memory
#pragma unroll
  for (int c = 0; c < kTile / 2; c += 32) {
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q)
      *reinterpret_cast<float4*>(slots + lane * 32 + ((q ^ (lane & 7)) << 2)) =
          make_float4(x[c + 4 * q], x[c + 4 * q + 1], x[c + 4 * q + 2], x[c + 4 * q + 3]);
    __syncwarp();
    const bool mine = c + lane < cols_left;
#pragma unroll
    for (int from = 0; from < 32; from += kTurn) {
      float v[kTurn];
#pragma unroll
      for (int j = 0; j < kTurn; ++j)
        v[j] = slots[(from + j) * 32 + (((lane >> 2) ^ (j & 7)) << 2) + (lane & 3)];
      turn(param + from * cols + c, copy != nullptr ? copy + from * cols + c : nullptr, mine ? rows_left - from : 0, v);
    }
  }
}

// Bounded wait for the phase of `bar` with parity `parity`, as wait_bar but by clock64: the epilogue waits
// once a chunk, and reading %globaltimer would be most of it.
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                              uint32_t role) {
  constexpr long long kLimit = 2000000000;  // a second
  const long long t0 = clock64();
  while (true) {
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kLimit) {
      *abort_flag = 1;
      atomicOr(err, role);
      atomicOr(err + kBatchError, role);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                         uint32_t role) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_long(bar, parity, abort_flag, err, role);
}

// A cluster's way out.  CTA q takes columns 16 q .. 16 q + 15 of each half of the tile: every CTA writes its
// segment's sums of them into that one's ring, which nothing reads any more, and each adds up what it has got,
// in the segments' order, to its own x.
template <int kProduct>
__device__ __forceinline__ void write_split(const MuonArgs& a, const MuonRecord& t, const MuonUnit& u,
                                            const Segments& segments, uint32_t rank, float unscale, const float (&x)[kTile / 2],
                                            const float (&y)[kTile / 2], int r, int half, uint8_t* ring, int64_t block) {
  constexpr int kSlice = kTile / 2 / kSplits;
  const int thread = half * kTile + r;
  cluster_sync();  // every CTA's products are done
  const uint32_t mine = smem_u32(ring) + thread * 16;
  // [segment][four columns][thread]
  constexpr uint32_t kGroup = kOutThreads * 16, kPart = kSlice / 4 * kGroup;
  if (int(rank) < segments.count())
#pragma unroll
    for (int q = 0; q < kSplits; ++q) {
      const uint32_t to = cluster_addr(mine + rank * kPart, q);
#pragma unroll
      for (int k = 0; k < kSlice / 4; ++k)
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + k * kGroup),
                     "f"(y[q * kSlice + 4 * k]), "f"(y[q * kSlice + 4 * k + 1]), "f"(y[q * kSlice + 4 * k + 2]),
                     "f"(y[q * kSlice + 4 * k + 3])
                     : "memory");
    }
  cluster_sync();
  float e[kSlice];
#pragma unroll
  for (int q = 0; q < kSplits; ++q)
    if (q == int(rank))
#pragma unroll
      for (int j = 0; j < kSlice; ++j) e[j] = x[q * kSlice + j];
  for (int s = 0; s < segments.count(); ++s)
#pragma unroll
    for (int k = 0; k < kSlice / 4; ++k) {
      float v[4];
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                   : "r"(mine + s * kPart + k * kGroup)
                   : "memory");
#pragma unroll
      for (int j = 0; j < 4; ++j) e[4 * k + j] += v[j];
    }
  const int column = half * (kTile / 2) + int(rank) * kSlice, diagonal = (u.i - u.j) * kTile + r - column;
#pragma unroll
  for (int j = 0; j < kSlice; ++j) {
    e[j] *= unscale;
    if (kProduct == kPoly && j == diagonal) e[j] += kA * kScale;
  }
  unsigned char* to = a.workspace + (kProduct == kGram ? t.g : t.p) + block + half * int64_t(kBlock);
  if (!LP_CHECK(block >= 0, kChkOutBox)) return;
#pragma unroll
  for (int q = 0; q < kSlice / 8; ++q) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e[8 * q + j];
    uint4 hi, lo;
    split8(v, hi, lo);
    const uint32_t in = chunk_at(r, int(rank) * (kSlice / 8) + q);
    *reinterpret_cast<uint4*>(to + in) = hi;
    *reinterpret_cast<uint4*>(to + kHalf + in) = lo;
  }
}

// One product over `units` tiles.  iteration: of the steps, the even ones read the first X, the odd ones the
// other; last: P X goes into the parameters instead of the other X.  map_a, map_b: the workspace as rows of 128
// bytes, in boxes of 256 and of 64.  withhold (tests of the bounded waits only): the first copy is announced and
// not made.
// kSplit: a cluster of kSplits CTAs a tile, each with a segment of K; they trade sums, so that each writes 16 of
// each 64 columns.  (The grid has a cluster for every unit.)
template <int kProduct, bool kSplit>
__global__ void __launch_bounds__(kProductThreads, 1)
    lp_muon_product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                           const __grid_constant__ MuonArgs a, const MuonUnit* units, int n_units,
                           int iteration, int last, int withhold) {
  constexpr int kMine = kTile / 2;  // columns of an epilogue thread
  const int from = iteration & 1;
  uint8_t* smem = pipeline_smem_base();
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOut + kBlock);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  const auto full_bar = [&](int s) { return bar0 + 8u * s; };
  const auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  const auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
  const auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * kStages + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 4), tile_bar = drain_bar + 8u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = kSplit ? blockIdx.x / kSplits : blockIdx.x, step = kSplit ? gridDim.x / kSplits : gridDim.x;
  const uint32_t rank = kSplit ? cluster_rank() : 0u;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(full_bar(s), 1), mbar_init(empty_bar(s), 1);
    for (int b = 0; b < 2; ++b) mbar_init(tfull_bar(b), 1), mbar_init(tempty_bar(b), kOutWarps);
    mbar_init(drain_bar, 1);
    mbar_init(tile_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_b)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(2 * kAccumulator)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // the plan does not depend on the launch before: its first entries come on chip meanwhile
  if (first < n_units && lane == 0) {
    const int tensor = *reinterpret_cast<const volatile int*>(&units[first].tensor);
    if (LP_CHECK(tensor >= 0 && tensor < a.n_tensors, kChkPlan))
      asm volatile("prefetch.global.L1 [%0];" ::"l"(a.records + tensor) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kSplit) cluster_sync();  // the cluster's CTAs are there
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the operands are written

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegisters));
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ loader
      int stage = 0;
      uint32_t phase = 0, pending = 0, pending_parity = 0;
      bool ok = true;
      for (int n = first; ok && n < n_units; n += step) {
        const MuonUnit u = units[n];
        if (!LP_CHECK(u.tensor >= 0 && u.tensor < a.n_tensors, kChkPlan)) break;
        const Operands o = operands_of<kProduct>(a.records[u.tensor], from);
        const bool same = kProduct != kApply && u.i == u.j;
        const Segments segments(o.k_blocks);
        const int kb_end = segments.begin(segments.template last<kSplit>(rank));
        for (int kb = segments.begin(segments.template first<kSplit>(rank)); kb < kb_end; ++kb) {
          if (!wait_for(empty_bar(stage), phase ^ 1u, abort_flag, a.err, kErrLoader)) {
            ok = false;
            break;
          }
          const uint32_t sa = smem_u32(smem + stage * kStage), bar = full_bar(stage);
          mbar_arrive_expect_tx(bar, same ? kBlock : kStage);
          pending |= 1u << stage;
          pending_parity = (pending_parity & ~(1u << stage)) | (phase << stage);
          // 64 columns of row block i, or where they mirror to: 64 rows of two neighbouring blocks, the hi parts,
          // then the lo parts
          const auto load = [&](uint32_t to, int base, int blocks, int i, bool mirror) {
            const int row = base + (mirror ? (kb / 2 * blocks + 2 * i) * kBlockRows + (kb & 1) * 64
                                           : (i * blocks + kb) * kBlockRows);
            if (!LP_CHECK(row >= 0, kChkTmaCoord)) return;
            if (!mirror) {
              tma_load_2d_local(to, &map_a, 0, row, bar);
              return;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
              tma_load_2d_local(to + q * (kHalf / 2), &map_b, 0, row + (q & 1) * kBlockRows + (q / 2) * kTile, bar);
          };
          if (!(withhold != 0 && n == 0 && kb == 0)) {
            load(sa, o.a, o.a_blocks, u.i, kProduct != kGram && mirrored(u.i, kb));
            if (!same)
              load(sa + kBlock, o.b, o.b_blocks, u.j, kProduct == kApply || (kProduct == kPoly && mirrored(u.j, kb)));
          }
          if (++stage == kStages) stage = 0, phase ^= 1u;
        }
      }
      if (!ok)  // let every issued copy land before the CTA can exit
        for (int s = 0; s < kStages; ++s)
          if (pending & (1u << s)) drain_wait(full_bar(s), (pending_parity >> s) & 1u);
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------ products
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int n = first; ok && n < n_units; n += step) {
        const MuonUnit u = units[n];
        if (!LP_CHECK(u.tensor >= 0 && u.tensor < a.n_tensors, kChkPlan)) break;
        const int k_blocks = operands_of<kProduct>(a.records[u.tensor], from).k_blocks;
        const bool same = kProduct != kApply && u.i == u.j;
        const Segments segments(k_blocks);
        const int to = segments.template last<kSplit>(rank);
        for (int segment = segments.template first<kSplit>(rank); ok && segment < to; ++segment) {
          const int end = segments.begin(segment + 1);
          int kb = segments.begin(segment);
          while (ok && kb < end) {  // a chunk
            const int chunk_end = min(kb + kChunk, end);
            const uint32_t d = tmem_base + uint32_t(acc) * kAccumulator;
            uint32_t adds = 0;
            if (!wait_for(tempty_bar(acc), acc_phase ^ 1u, abort_flag, a.err, kErrMma)) ok = false;
            for (; ok && kb < chunk_end; ++kb) {
              if (!wait_for(full_bar(stage), phase, abort_flag, a.err, kErrMma)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t sa = smem_u32(smem + stage * kStage), sb = same ? sa : sa + kBlock;
              const bool a_mn = kProduct != kGram && mirrored(u.i, kb);
              const bool b_mn = kProduct == kApply || (kProduct == kPoly && mirrored(u.j, kb));
              const uint64_t hi = a_mn ? sw128_mn_desc(sa, kHalf / 2) : sw128_desc(sa), lo = hi + (kHalf >> 4);
              const uint64_t b = b_mn ? sw128_mn_desc(sb, kHalf / 2) : sw128_desc(sb);
              // of a step of 16 of K, in the descriptors' units: 8 rows of 128 bytes twice, or 32 bytes of a row
              const uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
              const uint32_t major = uint32_t(a_mn) << 15 | uint32_t(b_mn) << 16;
#pragma unroll
              for (int k = 0; k < kBlockK / kUmmaK; ++k) {
                // hi x [hi; lo] as one of N = 256, and lo x hi onto its second half
                tc_mma_single(d, hi + k * a_step, b + k * b_step, adds, idesc_half(2 * kTile) | major);
                tc_mma_single(d + kTile, lo + k * a_step, b + k * b_step, 1u, idesc_half(kTile) | major);
                adds = 1;
              }
              tc_commit_local(empty_bar(stage));
              if (++stage == kStages) stage = 0, phase ^= 1u;
            }
            if (!ok) break;
            tc_commit_local(tfull_bar(acc));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
          }
        }
      }
      tc_commit_local(drain_bar);
      drain_wait(drain_bar, 0);
    }
    if (kSplit && first < n_units) {  // the epilogues' meetings over the cluster's one unit
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    // -------------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegisters));
    // the thread's row of the tile, and which half of its columns
    const int group = warp & 3, half = warp / 4 - 1, r = group * 32 + lane;
    const uint32_t t_lane = tmem_base + (uint32_t(group * 32) << 16) + half * kMine;
    const bool first_thread = threadIdx.x == 128;
    uint8_t* out = smem + kOut;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool poison = last && *reinterpret_cast<volatile uint32_t*>(a.err + kBatchError) != 0u;
    for (int n = first; n < n_units; n += step) {
      const MuonUnit u = units[n];
      if (!LP_CHECK(u.tensor >= 0 && u.tensor < a.n_tensors, kChkPlan)) {
        if constexpr (kSplit) cluster_sync(), cluster_sync();  // the cluster's other warps wait there
        break;
      }
      const MuonRecord& t = a.records[u.tensor];
      const int k_blocks = operands_of<kProduct>(t, from).k_blocks;
      const int64_t cols = padded_to(kProduct == kApply ? t.n : t.m, kTile) / kBlockK;
      const int64_t block = block_at(u.i, 2 * int64_t(u.j), cols);
      // the matrix's exponent here, and what takes the sums to what is written
      int level = 1;
      if (kProduct != kGram) level = __ldcg(a.levels + u.tensor);
      const int exponent = exponent_at(max(level - 1, 0), iteration);
      const float unscale =
          kProduct == kGram   ? kUnscale
          : kProduct == kPoly ? (exponent < kLinear ? kC * kUnscale * power_of_2(-4 * exponent) : 0.f)
          : last              ? kUnscale * kUnscale * power_of_2(-exponent)
                              : kUnscale * power_of_2(exponent_at(max(level - 1, 0), iteration + 1) - exponent);
      float x[kMine];  // the chunks' sums, rounded to nearest
      int go = 1;
      if (kProduct == kPoly) {
        // c (G G + b / c G), and of a G that is held times 4^e c 16^-e (G G + 4^e b / c G): what G adds comes in while
        // the first products run, the hi parts of both blocks, then the lo parts, through the tile's way out.  (Read
        // from global memory, 16 bytes a lane of 32 rows, it took 4 us of a launch's 13.)
        const float linear = kB / kC * kScale * power_of_2(2 * min(exponent, kLinear));
#pragma unroll
        for (int lo = 0; lo < 2; ++lo) {
          if (first_thread) {
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the buffer is free
            mbar_arrive_expect_tx(tile_bar, kBlock);
#pragma unroll
            for (int q = 0; q < 2; ++q)
              bulk_load(smem_u32(out) + q * kHalf, a.workspace + t.g + block + q * int64_t(kBlock) + lo * kHalf, kHalf,
                        tile_bar);
          }
          // every lane waits itself: what it reads has come by the barrier alone
          go = __all_sync(0xffffffffu, go && wait_for(tile_bar, lo, abort_flag, a.err, kErrEpilogue));
#pragma unroll
          for (int q = 0; q < kMine / 8; ++q) {
            uint32_t h[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                         : "r"(smem_u32(out) + half * kHalf + chunk_at(r, q))
                         : "memory");
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
              if (lo == 0) x[8 * q + 2 * i] = f.x, x[8 * q + 2 * i + 1] = f.y;
              else {
                x[8 * q + 2 * i] = (x[8 * q + 2 * i] + f.x) * linear;
                x[8 * q + 2 * i + 1] = (x[8 * q + 2 * i + 1] + f.y) * linear;
              }
            }
          }
          epilogue_sync();  // the buffer has been read
        }
      } else {
#pragma unroll
        for (int j = 0; j < kMine; ++j) x[j] = 0.f;
      }
      const Segments segments(k_blocks);
      float y[kMine];  // a segment's
      for (int segment = segments.template first<kSplit>(rank); segment < segments.template last<kSplit>(rank) && go;
           ++segment) {
#pragma unroll
        for (int j = 0; j < kMine; ++j) y[j] = 0.f;
        for (int kb = segments.begin(segment); kb < segments.begin(segment + 1); kb += kChunk) {
          if (lane == 0) go = *abort_flag == 0 && wait_for(tfull_bar(acc), acc_phase, abort_flag, a.err, kErrEpilogue);
          go = __shfl_sync(0xffffffffu, go, 0);
          if (!go) break;
          tc_fence_after();
          const uint32_t at = t_lane + uint32_t(acc) * kAccumulator;
#pragma unroll
          for (int c = 0; c < kMine; c += 32) {
            uint32_t v[32], w[32];  // hi hi, and the rest
            tmem_load32(at + c, v);
            tmem_load32(at + kTile + c, w);
            tmem_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) y[c + j] += __uint_as_float(v[j]) + __uint_as_float(w[j]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_local(tempty_bar(acc));
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
        if constexpr (!kSplit) {
#pragma unroll
          for (int j = 0; j < kMine; ++j) x[j] += y[j];
        }
      }
      if constexpr (kSplit) {
        write_split<kProduct>(a, t, u, segments, rank, unscale, x, y, r, half, smem, block);
        continue;  // the grid's clusters have a unit each
      }
      // every warp of the CTA goes on, or none does: they meet at the tile's way out
      if (!epilogue_all(go)) {  // the tiles that are left have no result
        if (!last) break;
        poison = true;
      }
      if (kProduct == kApply && last) {
        write_params(a, t, level != 0, unscale, u.i * kTile + group * 32, u.j * kTile + half * kMine, lane, x,
                     reinterpret_cast<float*>(out) + (warp - 4) * 1024, poison);
        continue;
      }
      const int diagonal = (u.i - u.j) * kTile + r - half * kMine;  // where the row meets it in x
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        x[j] *= unscale;
        if (kProduct == kPoly && j == diagonal) x[j] += kA * kScale;
      }
      unsigned char* to = a.workspace + (kProduct == kGram ? t.g : kProduct == kPoly ? t.p : t.x[from ^ 1]);
      if (LP_CHECK(block >= 0, kChkOutBox)) write_tile(x, r, half, to + block, out, first_thread);
    }
    if (first_thread) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // all is written
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(2 * kAccumulator)
                 : "memory");
  }
}

// ------------------------------------------------------------------------- host

template <class... Params, class... Args>
bool launch_next(void (*kernel)(Params...), int64_t blocks, int threads, int smem, bool dependent, int cluster,
                 cudaStream_t stream,
                 const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  cfg.attrs = attrs;
  if (dependent) {
    attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attrs[cfg.numAttrs].val.clusterDim.x = unsigned(cluster);
    attrs[cfg.numAttrs].val.clusterDim.y = attrs[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// Elements of the X of a batch's matrices: enough to fill the GPU many times over.
constexpr int64_t kBatchElements = int64_t(1) << 26;

// The plan as it grows.
struct Building {
  std::vector<MuonBatch> batches;
  std::vector<MuonRecord> records;
  std::vector<MuonUnit> parts, blocks, gram, apply;
  size_t workspace = 0;
};

int k_of(const Building& b, const MuonUnit& u, bool gram) {
  const MuonRecord& t = b.records[size_t(u.tensor)];
  return int(gram ? t.n : t.m);
}

Building build_plan(const lp_muon_tensor* tensors, int64_t n_tensors) {
  Building b;
  int64_t i = 0;
  while (i < n_tensors) {
    MuonBatch batch{};
    batch.first_part = int64_t(b.parts.size());
    batch.first_block = int64_t(b.blocks.size());
    batch.first_gram = int64_t(b.gram.size());
    batch.first_apply = int64_t(b.apply.size());
    int64_t elements = 0;
    std::vector<int32_t> in;
    for (; i < n_tensors; ++i) {
      const lp_muon_tensor& t = tensors[i];
      MuonRecord r{};
      r.param = t.param;
      r.copy = static_cast<__nv_bfloat16*>(t.copy);
      r.grad = t.grad;
      r.momentum = t.momentum;
      r.rows = t.rows;
      r.cols = t.cols;
      r.tall = t.rows > t.cols;
      r.m = std::min(t.rows, t.cols);
      r.n = std::max(t.rows, t.cols);
      r.lr_scale = t.lr_scale;
      r.weight_decay = t.weight_decay;
      r.update_scale = t.update_scale;
      r.grad_bf16 = t.grad_dtype == LP_BFLOAT16;
      const auto at = [](const void* p, uintptr_t by) { return reinterpret_cast<uintptr_t>(p) % by == 0; };
      r.wide = at(t.grad, r.grad_bf16 ? 8 : 16) && at(t.momentum, 16) && at(t.param, 16) && t.cols % 4 == 0;
      const int64_t padded = padded_to(r.m, kTile) * padded_to(r.n, kTile);
      if (r.m > 0 && !in.empty() && elements + padded > kBatchElements) break;
      b.records.push_back(r);
      if (r.m == 0) continue;
      elements += padded;
      in.push_back(int32_t(i));
    }
    if (in.empty()) break;  // only matrices without elements are left
    int64_t parts = 0;
    for (int32_t k : in) {
      MuonRecord& r = b.records[size_t(k)];
      r.first_part = parts;
      // at least kMuonPart elements, and no more than 1024 parts
      r.part = padded_to(std::max(kMuonPart, (r.rows * r.cols + 1023) / 1024), 4);
      r.parts = (r.rows * r.cols + r.part - 1) / r.part;
      parts += r.parts;
      batch.most_m = std::max(batch.most_m, r.m);
      batch.most_n = std::max(batch.most_n, r.n);
      for (int64_t p = 0; p < r.parts; ++p) b.parts.push_back({k, int32_t(p), 0, 0});
      const int64_t mb = padded_to(r.m, kTile) / kTile, nb = padded_to(r.n, kTile) / kTile;
      for (int64_t x = 0; x < mb; ++x)
        for (int64_t y = 0; y < 2 * nb; ++y) b.blocks.push_back({k, 0, int16_t(x), int16_t(y)});
    }
    for (int32_t k : in) {
      const MuonRecord& r = b.records[size_t(k)];
      const int64_t mb = padded_to(r.m, kTile) / kTile, nb = padded_to(r.n, kTile) / kTile;
      for (int64_t x = 0; x < mb; ++x)
        for (int64_t y = 0; y <= x; ++y) b.gram.push_back({k, 0, int16_t(x), int16_t(y)});
      for (int64_t y = 0; y < nb; ++y)
        for (int64_t x = 0; x < mb; ++x) b.apply.push_back({k, 0, int16_t(x), int16_t(y)});
    }
    // the longest products first, so that the last ones to start are short
    std::stable_sort(b.gram.begin() + batch.first_gram, b.gram.end(),
                     [&](const MuonUnit& x, const MuonUnit& y) { return k_of(b, x, true) > k_of(b, y, true); });
    std::stable_sort(b.apply.begin() + batch.first_apply, b.apply.end(),
                     [&](const MuonUnit& x, const MuonUnit& y) { return k_of(b, x, false) > k_of(b, y, false); });
    batch.parts = int64_t(b.parts.size()) - batch.first_part;
    batch.blocks = int64_t(b.blocks.size()) - batch.first_block;
    batch.grams = int64_t(b.gram.size()) - batch.first_gram;
    batch.applies = int64_t(b.apply.size()) - batch.first_apply;
    // the workspace: header, the matrices' flags, partial sums, then each matrix's buffers
    const auto up = [](size_t v) { return (v + 1023) / 1024 * 1024; };
    size_t at = up(kWorkspaceHeader + size_t(n_tensors) * 4);
    batch.partials_at = int64_t(at);
    at += up(size_t(parts) * sizeof(float));
    for (int32_t k : in) {
      MuonRecord& r = b.records[size_t(k)];
      const int64_t mp = padded_to(r.m, kTile), np = padded_to(r.n, kTile);
      for (int64_t* p : {&r.x[0], &r.x[1]}) *p = int64_t(at), at += size_t(mp * np) * 4;
      for (int64_t* p : {&r.g, &r.p}) *p = int64_t(at), at += size_t(mp * mp) * 4;
    }
    b.workspace = std::max(b.workspace, at);
    b.batches.push_back(batch);
  }
  return b;
}

MuonHeader header_of(const Building& b) {
  MuonHeader h{};
  const auto up = [](size_t v) { return int64_t((v + 255) / 256 * 256); };
  h.magic = kMuonMagic;
  h.n_tensors = int64_t(b.records.size());
  h.n_batches = int64_t(b.batches.size());
  h.workspace = int64_t(b.workspace);
  h.batches_at = up(sizeof(MuonHeader));
  h.records_at = h.batches_at + up(b.batches.size() * sizeof(MuonBatch));
  h.parts_at = h.records_at + up(b.records.size() * sizeof(MuonRecord));
  h.blocks_at = h.parts_at + up(b.parts.size() * sizeof(MuonUnit));
  h.gram_at = h.blocks_at + up(b.blocks.size() * sizeof(MuonUnit));
  h.apply_at = h.gram_at + up(b.gram.size() * sizeof(MuonUnit));
  h.bytes = h.apply_at + up(b.apply.size() * sizeof(MuonUnit));
  return h;
}

template <class T>
void put_all(char* to, const std::vector<T>& v) {
  if (!v.empty()) std::copy_n(reinterpret_cast<const char*>(v.data()), v.size() * sizeof(T), to);
}

}  // namespace

size_t muon_plan_bytes(const lp_muon_tensor* tensors, int64_t n_tensors) {
  return size_t(header_of(build_plan(tensors, n_tensors)).bytes);
}

void write_muon_plan(const lp_muon_tensor* tensors, int64_t n_tensors, void* plan, size_t bytes) {
  const Building b = build_plan(tensors, n_tensors);
  const MuonHeader h = header_of(b);
  if (bytes < size_t(h.bytes)) return;
  char* p = static_cast<char*>(plan);
  std::fill_n(p, h.bytes, char(0));
  std::copy_n(reinterpret_cast<const char*>(&h), sizeof(h), p);
  put_all(p + h.batches_at, b.batches);
  put_all(p + h.records_at, b.records);
  put_all(p + h.parts_at, b.parts);
  put_all(p + h.blocks_at, b.blocks);
  put_all(p + h.gram_at, b.gram);
  put_all(p + h.apply_at, b.apply);
}

// The three products of every step of a batch.
static lp_status launch_products(const Device& dev, const CUtensorMap& map_a, const CUtensorMap& map_b,
                                 const MuonArgs& a, const MuonBatch& b, const MuonUnit* gram, const MuonUnit* apply,
                                 int steps, bool withhold, cudaStream_t stream) {
  static PerContextOnce once;
  if (once.run(dev.ctx_id, [] {
        for (const void* k : {reinterpret_cast<const void*>(lp_muon_product_kernel<kGram, false>),
                              reinterpret_cast<const void*>(lp_muon_product_kernel<kPoly, false>),
                              reinterpret_cast<const void*>(lp_muon_product_kernel<kApply, false>),
                              reinterpret_cast<const void*>(lp_muon_product_kernel<kGram, true>),
                              reinterpret_cast<const void*>(lp_muon_product_kernel<kPoly, true>)}) {
          const cudaError_t e = set_smem_limit(k, kSmem);
          if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
      }) != cudaSuccess)
    return LP_ERR_CUDA;
  for (int s = 0; s < steps; ++s) {
    const int last = s == steps - 1;
    const auto launch = [&](auto* kernel, int64_t grid, int cluster, const MuonUnit* units, int64_t n, int is_last,
                            int first) {
      return launch_next(kernel, grid, kProductThreads, kSmem, true, cluster, stream, map_a, map_b, a, units, int(n),
                         s, is_last, first);
    };
    const int withheld = s == 0 && withhold;
    const int64_t few = single_grid(dev.sm_count, b.grams), many = single_grid(dev.sm_count, b.applies);
    // A cluster a tile while all clusters fit, where there is a K to split: 2047 x 1021 (36 tiles of K 2048 and
    // 1024) takes 208 us a step so, 268 with a CTA a tile.
    const bool split = b.grams * kSplits <= dev.sm_count && few == b.grams;
    const bool split_gram = split && b.most_n > (kSplitBlocks - 1) * kBlockK,
               split_poly = split && b.most_m > (kSplitBlocks - 1) * kBlockK;
    if (!(split_gram ? launch(lp_muon_product_kernel<kGram, true>, b.grams * kSplits, kSplits, gram, b.grams, 0, withheld)
                     : launch(lp_muon_product_kernel<kGram, false>, few, 1, gram, b.grams, 0, withheld)) ||
        !(split_poly ? launch(lp_muon_product_kernel<kPoly, true>, b.grams * kSplits, kSplits, gram, b.grams, 0, 0)
                     : launch(lp_muon_product_kernel<kPoly, false>, few, 1, gram, b.grams, 0, 0)) ||
        !launch(lp_muon_product_kernel<kApply, false>, many, 1, apply, b.applies, last, 0))
      return LP_ERR_CUDA;
  }
  return LP_OK;
}

lp_status launch_muon_step(const Device& dev, const void* plan_host, const void* plan, const MuonArgs& args,
                           int steps, cudaStream_t stream) {
  const char* host = static_cast<const char*>(plan_host);
  const char* device = static_cast<const char*>(plan);
  const MuonHeader& h = *reinterpret_cast<const MuonHeader*>(host);
  MuonArgs a = args;
  a.records = reinterpret_cast<const MuonRecord*>(device + h.records_at);
  a.n_tensors = h.n_tensors;
  a.err = reinterpret_cast<uint32_t*>(a.workspace);
  a.levels = reinterpret_cast<int32_t*>(a.workspace + kWorkspaceHeader);
  CUtensorMap map_a, map_b;
  const int64_t rows = h.workspace / kRow;
  if (!encode_rows128(&map_a, a.workspace, rows, 256) || !encode_rows128(&map_b, a.workspace, rows, 64))
    return LP_ERR_CUDA;
  const auto units_at = [&](int64_t at, int64_t first) {
    return reinterpret_cast<const MuonUnit*>(device + at) + first;
  };
  for (int64_t k = 0; k < h.n_batches; ++k) {
    const MuonBatch& b = reinterpret_cast<const MuonBatch*>(host + h.batches_at)[k];
    float* partials = reinterpret_cast<float*>(a.workspace + b.partials_at);
    if (!launch_next(lp_muon_norm_kernel, b.parts, kNormThreads, 0, false, 1, stream, a,
                     units_at(h.parts_at, b.first_part), partials, int(k == 0)) ||
        !launch_next(lp_muon_split_kernel, b.blocks, kSplitThreads, 0, true, 1, stream, a,
                     units_at(h.blocks_at, b.first_block), static_cast<const float*>(partials)))
      return LP_ERR_CUDA;
    const lp_status st = launch_products(
        dev, map_a, map_b, a, b, units_at(h.gram_at, b.first_gram), units_at(h.apply_at, b.first_apply), steps,
        k == 0 && fault_injection() == 1, stream);
    if (st != LP_OK) return st;
  }
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

cudaError_t take_check_word_muon(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
