// lp_adamw.cu: AdamW over many tensors, the norm of their gradients, and the values
// of 8-bit moments (include/lp_train.h).
//
// Every element is computed alone, so the step is bound by its bytes: with 32-bit moments, float32
// gradients and a bfloat16 copy 30 an element, and 622 M elements take 2.63 ms, 7.1 TB/s.  With
// 8-bit moments the bytes halve and the codes' integer work comes to light: 300 M elements with
// float32 gradients took 926 us at 106 instructions an element and take 880 at 84, of 795 us at
// the copy rate (issue slots 73%, ALU pipe 58% busy).  The values of 311 M elements' 8-bit moments
// are written in 448 us, 6.9 TB/s.  300 tensors of 64 to 4 M elements, 113 M in all, take 578 us with
// their norm, of which the step is 490 and reading the gradients for the norm 77.  Tensors off a
// 16-byte boundary go through shared memory: 40 M elements take 363 us instead of 175 with 32 bits, 340
// instead of 122 with 8.  Where each warp has one block, no copy runs ahead: 4.9 M elements of 8 bits
// take 19.4 us of 11.6.
//
// One launch: a table gives each CTA's row its tensor, and a tensor's blocks of 256 elements are a
// warp's.  The moments' products are each rounded (no fused multiplication), so that 8-bit moments,
// which are rounded by comparing bits, do not depend on how the arithmetic was compiled.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "lp_check.cuh"
#include "lp_device.cuh"
#include "lp_train_internal.h"

namespace lp {
namespace {

constexpr int kThreads = 256;
constexpr int kRow = LP_ADAMW_ALIGN;    // state elements of a CTA
constexpr int kBlock = LP_ADAMW_BLOCK;  // elements of a warp, with one scale
static_assert(kRow == kBlock * kThreads / 32, "one block of elements a warp");

// The magnitude codes of 8-bit moments: code c > 0 is the float of bits (c + kFirst) << kShift.
// The code of a float is its own leading bits, so both ways are a few integer operations on
// bytes where they lie in a word of four.
template <bool kSigned>
struct Code {
  static constexpr int kShift = kSigned ? 20 : 19;
  static constexpr uint32_t kFirst = kSigned ? 889 : 1777;
  static constexpr uint32_t kMask = kSigned ? 127 : 255;
  static constexpr uint32_t kLowest = (kFirst + 1) << kShift;  // bits of the value of code 1
  // that value over 2^kShift: what a random number below 2^kShift is scaled by to round a
  // magnitude below that value to it or to zero
  static constexpr float kLow = kSigned ? 0x1.4p-36f : 0x1.2p-35f;

  // Whether no byte of the word is a code for zero.
  static __device__ __forceinline__ bool none_zero(uint32_t word) {
    if (kSigned) return ((word & 0x7f7f7f7fu) + 0x7f7f7f7fu & 0x80808080u) == 0x80808080u;
    return (word - 0x01010101u & ~word & 0x80808080u) == 0u;
  }
  // Byte j of the word.  For the first moment the sign's bit, multiplied up with the code, adds
  // 16 to the exponent, which the factor of a negative value takes back.
  template <int j, bool kZeros>
  static __device__ __forceinline__ float decode(uint32_t word, float scale) {
    const uint32_t byte = __byte_perm(word, 0u, 0x4440u + j);
    const float value = __uint_as_float(byte * (1u << kShift) + (kFirst << kShift));
    float factor = kSigned && byte >= 128u ? scale * -0x1p-16f : scale;
    if (kZeros && (byte & kMask) == 0u) factor = 0.f * scale;
    return value * factor;
  }
  template <bool kZeros>
  static __device__ __forceinline__ void decode4(uint32_t word, float scale, float* v) {
    v[0] = decode<0, kZeros>(word, scale), v[1] = decode<1, kZeros>(word, scale);
    v[2] = decode<2, kZeros>(word, scale), v[3] = decode<3, kZeros>(word, scale);
  }
  // |x| over the block's largest magnitude, at most 1
  static __device__ __forceinline__ float part(float x, float inverse) {
    return fminf(fabsf(x) * inverse, 1.f);
  }
  // A part with its random bits added, moved up so that the code, plus the low byte of kFirst, is
  // the top byte; of a part below the lowest code's value, the top byte for zero.
  static __device__ __forceinline__ uint32_t rounded(float part, uint32_t word) {
    const uint32_t bits = __float_as_uint(part);
    const uint32_t random = __byte_perm(word, 0u, kSigned ? 0x4104u : 0x4324u);  // 16 bits, << 8
    return bits >= kLowest ? bits * (1u << (24 - kShift)) + random : kFirst << 24;
  }
  // The codes of four elements x with these rounded parts.
  static __device__ __forceinline__ uint32_t encode4(const uint32_t (&rounded)[4], const float* x) {
    uint32_t codes = top_bytes(rounded[0], rounded[1], rounded[2], rounded[3]);
    if (!kSigned)  // minus 0xf1 in every byte, without a carry between them
      return (codes & 0x7f7f7f7fu) + 0x0f0f0f0fu ^ (codes & 0x80808080u);
    codes -= 0x79797979u;  // every byte is 0x79 at least
    const uint32_t signs = top_bytes(__float_as_uint(x[0]), __float_as_uint(x[1]),
                                     __float_as_uint(x[2]), __float_as_uint(x[3]));
    return codes | (signs & codes + 0x7f7f7f7fu & 0x80808080u);  // zero has none
  }
  static __device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073u), __byte_perm(c, d, 0x0073u), 0x5410u);
  }
  // The code of an element whose part lies between zero and the lowest code's value, in its byte;
  // nothing for others.
  static __device__ __forceinline__ uint32_t encode_between(float x, float part, uint32_t word, int j) {
    if (__float_as_uint(part) - 1u >= kLowest - 1u) return 0u;
    const uint32_t random = kSigned ? (word & 0xffffu) << 4 : (word >> 16) << 3;
    if (!(part > static_cast<float>(random) * kLow)) return 0u;
    return (1u | (kSigned && x < 0.f ? 128u : 0u)) << 8 * j;
  }
};
static_assert((Code<true>::kFirst & 255u) == 0x79u && (Code<false>::kFirst & 255u) == 0xf1u,
              "the low bytes that encode4 takes off");

// Philox 4x32 with 7 rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers:
// as easy as 1, 2, 3", SC11) at counter (group, step), with the rounds' keys at hand.
__device__ __forceinline__ void random_words(uint64_t group, uint64_t step,
                                             const uint32_t (&keys)[7][2], uint32_t (&w)[4]) {
  uint32_t c0 = uint32_t(group), c1 = uint32_t(group >> 32), c2 = uint32_t(step),
           c3 = uint32_t(step >> 32);
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    c0 = uint32_t(b >> 32) ^ c1 ^ keys[i][0];
    c1 = uint32_t(b);
    c2 = uint32_t(a >> 32) ^ c3 ^ keys[i][1];
    c3 = uint32_t(a);
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

// The largest of a warp's values, NaN when one is.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// A block's scale from its largest magnitude: 0 below 2^-100, NaN when not finite.
__device__ __forceinline__ float scale_of(float largest) {
  if (!(largest <= 0x1.fffffep127f)) return __int_as_float(0x7fffffff);
  return largest < 0x1p-100f ? 0.f : largest;
}

// Two products or sums an instruction, each rounded as by itself.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; "
      "mov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 z, x, y; "
      "mov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two elements: the moments from m, v and the gradient, the new param, and the roots of v.
__device__ __forceinline__ float2 update(const AdamwArgs& a, float2 g, float kept, float step_size,
                                         float2* p, float2* m, float2* v) {
  // the products in pairs and the sums one by one: a pair's product and sum would be fused into
  // one rounding, and the moments' products are each rounded
  const float2 m0 = mul2(both(a.beta1), *m), m1 = mul2(both(a.rest1), g);
  const float2 v0 = mul2(both(a.beta2), *v), v1 = mul2(both(a.rest2), mul2(g, g));
  *m = make_float2(__fadd_rn(m0.x, m1.x), __fadd_rn(m0.y, m1.y));
  *v = make_float2(__fadd_rn(v0.x, v1.x), __fadd_rn(v0.y, v1.y));
  const float2 u = make_float2(sqrtf(v->x), sqrtf(v->y));
  const float2 below = add2(mul2(u, both(a.root_scale)), both(a.eps));
  // the quotient by an approximate reciprocal, within 3 units in the last place: it is far below
  // the param that it changes
  const float2 change = mul2(*m, make_float2(reciprocal(below.x), reciprocal(below.y)));
  *p = add2(mul2(*p, both(kept)), mul2(both(-step_size), change));
  return u;
}

// A lane's 8 elements of a block: 4 lane + {0..3} and 128 + 4 lane + {0..3}, 16 bytes of
// float32 or 8 of bfloat16 an access.  Where the tensor is not aligned for that, or the block
// is its ragged end, they go through a warp's stretch of shared memory, 32 neighbours an access.
__device__ __forceinline__ void load8(const float* p, int count, bool wide, float* stretch,
                                      float (&v)[8]) {
  const int lane = threadIdx.x & 31;
  if (wide && count >= kBlock) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[4 * h]), "=f"(v[4 * h + 1]), "=f"(v[4 * h + 2]), "=f"(v[4 * h + 3])
                   : "l"(p + 128 * h + 4 * lane)
                   : "memory");
    return;
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = 32 * k + lane;
    stretch[e] = e < count ? p[e] : 0.f;
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = stretch[(k >> 2) * 128 + lane * 4 + (k & 3)];
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int count, bool wide, float* stretch,
                                      float (&v)[8]) {
  const int lane = threadIdx.x & 31;
  if (wide && count >= kBlock) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a, b;
      asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];"
                   : "=r"(a), "=r"(b)
                   : "l"(p + 128 * h + 4 * lane)
                   : "memory");
      v[4 * h] = __uint_as_float(a << 16), v[4 * h + 1] = __uint_as_float(a & 0xffff0000u);
      v[4 * h + 2] = __uint_as_float(b << 16), v[4 * h + 3] = __uint_as_float(b & 0xffff0000u);
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = 32 * k + lane;
    stretch[e] = e < count ? __bfloat162float(p[e]) : 0.f;
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = stretch[(k >> 2) * 128 + lane * 4 + (k & 3)];
}
__device__ __forceinline__ void store8(float* p, __nv_bfloat16* copy, int count, bool wide,
                                       float* stretch, const float (&v)[8]) {
  const int lane = threadIdx.x & 31;
  if (wide && count >= kBlock) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = 128 * h + 4 * lane;
      *reinterpret_cast<float4*>(p + e) =
          make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
      if (copy == nullptr) continue;
      __nv_bfloat162 two[2] = {__floats2bfloat162_rn(v[4 * h], v[4 * h + 1]),
                               __floats2bfloat162_rn(v[4 * h + 2], v[4 * h + 3])};
      *reinterpret_cast<uint2*>(copy + e) = *reinterpret_cast<const uint2*>(two);
    }
    return;
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) stretch[(k >> 2) * 128 + lane * 4 + (k & 3)] = v[k];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int e = 32 * k + lane;
    if (e >= count) continue;
    p[e] = stretch[e];
    if (copy != nullptr) copy[e] = __float2bfloat16_rn(stretch[e]);
  }
}

// A block on its way into shared memory; a lane copies what it reads.
struct Stage {
  float p[kBlock];
  float g[kBlock];  // float32 or bfloat16
  uint32_t m[kBlock / 4], u[kBlock / 4];
};
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(to))),
               "l"(from)
               : "memory");
}
template <int kBytes>
__device__ __forceinline__ void copy_few(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(to))),
               "l"(from), "n"(kBytes)
               : "memory");
}

// One row of a tensor a CTA, its blocks in turn a warp.  The moments' buffers are padded to whole
// blocks, and what lies past a tensor's end in them stays zero.
//
// With 32-bit moments a block is 7 KB of traffic and 32 warps an SM keep the memory busy.  With
// 8-bit ones it is half of that and some 90 instructions an element, so the next block is
// copied while one is computed.
template <bool kSmall, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 32 / kWarps)
    lp_adamw_kernel(const __grid_constant__ AdamwArgs a) {
  constexpr int kStretch = (kSmall ? 2 * sizeof(Stage) : kBlock * sizeof(float)) / sizeof(float);
  __shared__ __align__(16) float stretches[kWarps][kStretch];
  const int64_t row = blockIdx.x;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int32_t index = a.table[row];
  if (!LP_CHECK(row < a.rows && index >= 0 && index < a.n_tensors, kChkPlan)) return;
  const AdamwRecord rec = a.records[index];
  if (!LP_CHECK(row >= rec.first_row && (row - rec.first_row) * kRow < rec.n, kChkPlan)) return;
  const float clip = a.grad_scale != nullptr ? *a.grad_scale : 1.f;
  if (clip != clip) return;
  const float lr = a.lr * rec.lr_scale;
  const float kept = 1.f - lr * rec.weight_decay, step_size = a.step_size * rec.lr_scale;
  float* stretch = stretches[warp];
  const int64_t first = (row - rec.first_row) * kRow;  // of the row in the tensor
  const int left = int(min(rec.n - first, int64_t(kRow)));
  // every access below is of the row's first `left` elements, or of its kRow in the moments
  if (!LP_CHECK(left > 0 && first >= 0 && first + left <= rec.n && rec.first_row >= 0 &&
                    rec.first_row + (rec.n + kRow - 1) / kRow <= a.rows,
                kChkPlan))
    return;
  const bool is_wide = rec.wide != 0;
  float* const params = rec.param + first;
  __nv_bfloat16* const copies = rec.copy != nullptr ? rec.copy + first : nullptr;
  constexpr int step = kWarps * kBlock;
  // starts the copy of the block at `at`, where it is whole and aligned
  const auto fetch = [&](int at, Stage* to) {
    if (is_wide && left - at >= kBlock) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = 128 * h + 4 * lane;
        copy16(to->p + e, params + at + e);
        if (rec.grad_bf16)
          copy_few<8>(reinterpret_cast<__nv_bfloat16*>(to->g) + e,
                      static_cast<const __nv_bfloat16*>(rec.grad) + first + at + e);
        else
          copy16(to->g + e, static_cast<const float*>(rec.grad) + first + at + e);
        copy_few<4>(to->m + e / 4, static_cast<const uint32_t*>(a.exp_avg) + (row * kRow + at + e) / 4);
        copy_few<4>(to->u + e / 4, static_cast<const uint32_t*>(a.exp_avg_sq) + (row * kRow + at + e) / 4);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  Stage* stage = reinterpret_cast<Stage*>(stretch);
  Stage* other = stage + 1;
  if (kSmall) fetch(warp * kBlock, stage);
  for (int at = warp * kBlock; at < left; at += step) {
    const int count = min(left - at, kBlock);
    const int64_t flat = row * kRow + at;
    float p[8], g[8], m[8], v[8];
    uint32_t old_m[2], old_u[2];
    float old_scale_m = 0.f, old_scale_u = 0.f;
    if (kSmall) {
      old_scale_m = a.exp_avg_scale[flat / kBlock];
      old_scale_u = a.exp_avg_sq_scale[flat / kBlock];
      fetch(at + step, other);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    }
    if (kSmall && is_wide && count == kBlock) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = 128 * h + 4 * lane;
        const float4 x = *reinterpret_cast<const float4*>(stage->p + e);
        p[4 * h] = x.x, p[4 * h + 1] = x.y, p[4 * h + 2] = x.z, p[4 * h + 3] = x.w;
        if (rec.grad_bf16) {
          const uint2 y = *reinterpret_cast<const uint2*>(
              reinterpret_cast<const __nv_bfloat16*>(stage->g) + e);
          g[4 * h] = __uint_as_float(y.x << 16), g[4 * h + 1] = __uint_as_float(y.x & 0xffff0000u);
          g[4 * h + 2] = __uint_as_float(y.y << 16);
          g[4 * h + 3] = __uint_as_float(y.y & 0xffff0000u);
        } else {
          const float4 y = *reinterpret_cast<const float4*>(stage->g + e);
          g[4 * h] = y.x, g[4 * h + 1] = y.y, g[4 * h + 2] = y.z, g[4 * h + 3] = y.w;
        }
        old_m[h] = stage->m[e / 4];
        old_u[h] = stage->u[e / 4];
      }
    } else {
      load8(params + at, count, is_wide, stretch, p);
      if (rec.grad_bf16)
        load8(static_cast<const __nv_bfloat16*>(rec.grad) + first + at, count, is_wide, stretch, g);
      else
        load8(static_cast<const float*>(rec.grad) + first + at, count, is_wide, stretch, g);
      if (kSmall) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          old_m[h] = static_cast<const uint32_t*>(a.exp_avg)[flat / 4 + 32 * h + lane];
          old_u[h] = static_cast<const uint32_t*>(a.exp_avg_sq)[flat / 4 + 32 * h + lane];
        }
      } else {
        load8(static_cast<const float*>(a.exp_avg) + flat, kBlock, true, stretch, m);
        load8(static_cast<const float*>(a.exp_avg_sq) + flat, kBlock, true, stretch, v);
      }
    }
    if (a.grad_scale != nullptr)
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] *= clip;
    if (kSmall) {
      // a lane whose bytes are none of them zero, as mostly, does not ask each
      if (Code<true>::none_zero(old_m[0]) && Code<true>::none_zero(old_m[1]) &&
          Code<false>::none_zero(old_u[0]) && Code<false>::none_zero(old_u[1])) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          Code<true>::decode4<false>(old_m[h], old_scale_m, m + 4 * h);
          Code<false>::decode4<false>(old_u[h], old_scale_u, v + 4 * h);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          Code<true>::decode4<true>(old_m[h], old_scale_m, m + 4 * h);
          Code<false>::decode4<true>(old_u[h], old_scale_u, v + 4 * h);
        }
      }
    }
    float u[8];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      float2 mk = make_float2(m[k], m[k + 1]), vk = make_float2(v[k], v[k + 1]),
             pk = make_float2(p[k], p[k + 1]);
      if (kSmall) vk = mul2(vk, vk);
      const float2 uk = update(a, make_float2(g[k], g[k + 1]), kept, step_size, &pk, &mk, &vk);
      m[k] = mk.x, m[k + 1] = mk.y, v[k] = vk.x, v[k + 1] = vk.y, p[k] = pk.x, p[k + 1] = pk.y;
      u[k] = uk.x, u[k + 1] = uk.y;
    }
    store8(params + at, copies != nullptr ? copies + at : nullptr, count, is_wide, stretch, p);
    if (!kSmall) {
      store8(static_cast<float*>(a.exp_avg) + flat, nullptr, kBlock, true, stretch, m);
      store8(static_cast<float*>(a.exp_avg_sq) + flat, nullptr, kBlock, true, stretch, v);
      continue;
    }
    float top_m = 0.f, top_u = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      top_m = fmax_nan(top_m, fabsf(m[k]));
      top_u = fmax_nan(top_u, u[k]);
    }
    const float scale_m = scale_of(warp_max(top_m)), scale_u = scale_of(warp_max(top_u));
    const float inv_m = scale_m > 0.f ? 1.f / scale_m : 0.f;
    const float inv_u = scale_u > 0.f ? 1.f / scale_u : 0.f;
    if (lane == 0) {
      a.exp_avg_scale[flat / kBlock] = scale_m;
      a.exp_avg_sq_scale[flat / kBlock] = scale_u;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4], rounded_m[4], rounded_u[4];
      random_words(uint64_t(flat / 4 + h * 32 + lane), a.step, a.round_keys, w);
      float part_m[4], part_u[4];
      uint32_t least_m = ~0u, least_u = ~0u;  // the smallest parts' bits, less one
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        part_m[j] = Code<true>::part(m[4 * h + j], inv_m);
        part_u[j] = Code<false>::part(u[4 * h + j], inv_u);
        rounded_m[j] = Code<true>::rounded(part_m[j], w[j]);
        rounded_u[j] = Code<false>::rounded(part_u[j], w[j]);
        least_m = min(least_m, __float_as_uint(part_m[j]) - 1u);
        least_u = min(least_u, __float_as_uint(part_u[j]) - 1u);
      }
      uint32_t new_m = Code<true>::encode4(rounded_m, m + 4 * h);
      uint32_t new_u = Code<false>::encode4(rounded_u, u + 4 * h);
      if (least_m < Code<true>::kLowest - 1u || least_u < Code<false>::kLowest - 1u) {
        // rare: a magnitude below 2^-16 of its block's largest
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          new_m |= Code<true>::encode_between(m[4 * h + j], part_m[j], w[j], j);
          new_u |= Code<false>::encode_between(u[4 * h + j], part_u[j], w[j], j);
        }
      }
      static_cast<uint32_t*>(a.exp_avg)[flat / 4 + 32 * h + lane] = new_m;
      static_cast<uint32_t*>(a.exp_avg_sq)[flat / 4 + 32 * h + lane] = new_u;
    }
    Stage* const next = other;
    other = stage;
    stage = next;
  }
}

// One row of a tensor a warp, whose squares are summed by lane in order and then by shuffles.
__global__ void __launch_bounds__(kThreads)
    lp_adamw_square_sum_kernel(const AdamwRecord* records, const int32_t* table, int64_t n_tensors,
                               int64_t rows, float* sums) {
  __shared__ __align__(16) float stretches[kThreads / 32][kBlock];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x / 32;
  const int64_t row = int64_t(blockIdx.x) * (kThreads / 32) + warp;
  if (row >= rows) return;
  const int32_t index = table[row];
  if (!LP_CHECK(index >= 0 && index < n_tensors, kChkPlan)) return;
  const AdamwRecord rec = records[index];
  if (!LP_CHECK(row >= rec.first_row && (row - rec.first_row) * kRow < rec.n, kChkPlan)) return;
  const int64_t first = (row - rec.first_row) * kRow;
  const int count = int(min(rec.n - first, int64_t(kRow)));
  float s = 0.f;
#pragma unroll 8
  for (int b = 0; b < kRow; b += kBlock) {
    if (b >= count) break;
    float g[8];
    if (rec.grad_bf16)
      load8(static_cast<const __nv_bfloat16*>(rec.grad) + first + b, count - b, rec.wide != 0,
            stretches[warp], g);
    else
      load8(static_cast<const float*>(rec.grad) + first + b, count - b, rec.wide != 0,
            stretches[warp], g);
#pragma unroll
    for (int k = 0; k < 8; ++k) s += g[k] * g[k];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) sums[row] = s;
}

constexpr int kNormThreads = 1024;
// A sum and what its roundings lost (the error of a sum of two floats is a float: Knuth's two-sum).
// float64 additions would take longer than the loads.
struct Pair {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float sum = hi + x, back = sum - hi;
    lo += (hi - (sum - back)) + (x - back);
    hi = sum;
  }
};
__global__ void __launch_bounds__(kNormThreads)
    lp_adamw_norm_kernel(const float* sums, int64_t rows, float max_norm, float* norm_out) {
  __shared__ Pair slots[kNormThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Pair s{0.f, 0.f};
  const int64_t quads = rows / 4;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < quads; i += kNormThreads) {
    if (!LP_CHECK(4 * i + 4 <= rows, kChkStateIndex)) break;
    const float4 x = __ldcg(reinterpret_cast<const float4*>(sums) + i);
    s.add(x.x), s.add(x.y), s.add(x.z), s.add(x.w);
  }
  if (threadIdx.x < rows % 4) s.add(__ldcg(sums + quads * 4 + threadIdx.x));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, s.hi, o), lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
    s.add(hi);
    s.lo += lo;
  }
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < kNormThreads / 32; ++i) {
    s.add(slots[i].hi);
    s.lo += slots[i].lo;
  }
  // beside an infinite sum the part that was lost is no number
  const float norm = sqrtf(s.hi <= 0x1.fffffep127f ? s.hi + s.lo : s.hi);
  norm_out[0] = norm;
  norm_out[1] = norm <= 0x1.fffffep127f ? fminf(max_norm / (norm + 1e-6f), 1.f)
                                        : __int_as_float(0x7fffffff);
}

__global__ void __launch_bounds__(kThreads)
    lp_adamw_values_kernel(const uint32_t* m, const uint32_t* u, const float* m_scale,
                           const float* u_scale, float4* m_out, float4* v_out) {
#pragma unroll
  for (int k = 0; k < kRow / 4 / kThreads; ++k) {
    const int64_t i = int64_t(blockIdx.x) * (kRow / 4) + k * kThreads + threadIdx.x;
    if (!LP_CHECK(i >= 0 && i < int64_t(gridDim.x) * (kRow / 4), kChkStateIndex)) return;
    const uint32_t cm = __ldg(m + i), cu = __ldg(u + i);
    const float sm = __ldg(m_scale + i / (kBlock / 4)), su = __ldg(u_scale + i / (kBlock / 4));
    float a[4], b[4];
    Code<true>::decode4<true>(cm, sm, a);
    Code<false>::decode4<true>(cu, su, b);
    m_out[i] = make_float4(a[0], a[1], a[2], a[3]);
    v_out[i] = make_float4(b[0] * b[0], b[1] * b[1], b[2] * b[2], b[3] * b[3]);
  }
}

// From this many rows on, of 8-bit moments, a warp takes a whole row instead of a block of it: its
// copies then run ahead of seven blocks in eight.  12 M elements: 49.7 us against 47.3 with a
// block a warp; 24 M: 85 against 91; 300 M: 926 against 1087.
constexpr int64_t kManyRows = 152 * 48;

template <class... Params, class... Args>
bool launch_dependent(void (*kernel)(Params...), int64_t blocks, int threads, cudaStream_t stream,
                      Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

}  // namespace

lp_status launch_adamw_step(const AdamwArgs& args, cudaStream_t stream) {
  AdamwArgs a = args;
  for (int i = 0; i < 7; ++i) {
    a.round_keys[i][0] = uint32_t(a.seed) + uint32_t(i) * 0x9E3779B9u;
    a.round_keys[i][1] = uint32_t(a.seed >> 32) + uint32_t(i) * 0xBB67AE85u;
  }
  const auto launch = [&](auto* kernel, int warps) {
    kernel<<<unsigned(a.rows), 32 * warps, 0, stream>>>(a);
  };
  if (a.exp_avg_scale == nullptr)
    launch(lp_adamw_kernel<false, 8>, 8);
  else if (a.rows >= kManyRows)
    launch(lp_adamw_kernel<true, 1>, 1);
  else
    launch(lp_adamw_kernel<true, 8>, 8);
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

size_t adamw_grad_norm_workspace(int64_t rows) {
  return static_cast<size_t>(rows > 0 ? rows : 1) * 4;
}

lp_status launch_adamw_grad_norm(const AdamwRecord* records, const int32_t* table,
                                 int64_t n_tensors, int64_t rows, float max_norm, float* norm_out,
                                 void* workspace, cudaStream_t stream) {
  float* sums = static_cast<float*>(workspace);
  constexpr int kRowsOfCta = kThreads / 32;
  if (rows > 0) {
    lp_adamw_square_sum_kernel<<<unsigned((rows + kRowsOfCta - 1) / kRowsOfCta), kThreads, 0,
                                 stream>>>(records, table, n_tensors, rows, sums);
    if (cudaGetLastError() != cudaSuccess) return LP_ERR_CUDA;
  }
  if (!launch_dependent(lp_adamw_norm_kernel, 1, kNormThreads, stream,
                        static_cast<const float*>(sums), rows, max_norm, norm_out))
    return LP_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

lp_status launch_adamw_state_values(const void* exp_avg, const void* exp_avg_sq,
                                    const float* exp_avg_scale, const float* exp_avg_sq_scale,
                                    int64_t rows, float* m_out, float* v_out,
                                    cudaStream_t stream) {
  lp_adamw_values_kernel<<<unsigned(rows), kThreads, 0, stream>>>(
      static_cast<const uint32_t*>(exp_avg), static_cast<const uint32_t*>(exp_avg_sq),
      exp_avg_scale, exp_avg_sq_scale, reinterpret_cast<float4*>(m_out),
      reinterpret_cast<float4*>(v_out));
  return cudaGetLastError() == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

cudaError_t take_check_word_adamw(uint32_t* out) { return take_check_word(out); }

}  // namespace lp
