// lp_layer_norm.cuh: what the layer norm's kernels add to lp_norm.cuh.
#pragma once

#include "lp_norm.cuh"

namespace lp {
namespace {

__device__ __forceinline__ float2 add(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_bits(a)), "l"(as_bits(b)));
  return as_pair(r);
}

}  // namespace
}  // namespace lp
