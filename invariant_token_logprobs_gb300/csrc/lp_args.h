// lp_args.h: what the front ends of lp_train.h and lp_tune.h check their arguments with.
#pragma once

#include <cstdint>

#include "../../include/lp_train.h"

namespace lp {
namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxStride = int64_t(1) << 40;  // keeps row offsets inside 64 bits

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool is_dtype(int t) { return t == LP_FLOAT32 || t == LP_BFLOAT16; }
int64_t size_of(bool bf16) { return bf16 ? 2 : 4; }

// Bytes [p, p + (rows - 1) * pitch + width): a row operand's extent.
struct Extent {
  uintptr_t p = 0;
  uintptr_t pitch = 0, width = 0, rows = 0;
};
Extent extent(const void* p, int64_t rows, int64_t ld, int64_t width, int64_t size) {
  Extent e;
  if (p == nullptr || rows == 0) return e;
  e.p = reinterpret_cast<uintptr_t>(p);
  e.pitch = static_cast<uintptr_t>(ld * size);
  e.width = static_cast<uintptr_t>(width * size);
  e.rows = static_cast<uintptr_t>(rows);
  return e;
}
// Whether two operands share a byte.  Operands of one pitch may interleave (columns
// of one wide buffer); with other pitches the whole ranges must be apart.
bool overlap(const Extent& a, const Extent& b) {
  if (a.rows == 0 || b.rows == 0) return false;
  const uintptr_t a1 = a.p + (a.rows - 1) * a.pitch + a.width;
  const uintptr_t b1 = b.p + (b.rows - 1) * b.pitch + b.width;
  if (a.p >= b1 || b.p >= a1) return false;
  if (a.pitch != b.pitch || a.pitch == 0) return true;
  const uintptr_t lag = a.p <= b.p ? (b.p - a.p) % a.pitch
                                   : (a.pitch - (a.p - b.p) % a.pitch) % a.pitch;
  return lag < a.width || lag + b.width > a.pitch;
}

bool bad_rows(int64_t ld, int64_t d) { return ld < d || ld > kMaxStride; }

// Rows operand present and well formed, or absent; `required` says which.
bool mismatch(const void* p, bool required) { return (p != nullptr) != required; }

}  // namespace
}  // namespace lp
