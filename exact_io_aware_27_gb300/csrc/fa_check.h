// Argument checks shared by the C entry points (host only).
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "fa.h"
#include "fa_internal.h"

namespace fa {

inline bool is_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// `rows` rows of `width` bytes, `stride` bytes from row to row (stride >= width).
struct Rows {
  uintptr_t lo;
  size_t rows, width, stride;
  uintptr_t hi() const { return rows ? lo + (rows - 1) * stride + width : lo; }
};
inline Rows rows_of(const void* p, size_t rows, size_t width, size_t stride) {
  return {reinterpret_cast<uintptr_t>(p), rows, width, stride};
}
inline Rows bytes_of(const void* p, size_t bytes) { return rows_of(p, 1, bytes, bytes); }

// True when the two may share a byte. Views side by side in one buffer (equal strides,
// disjoint columns) do not overlap although their address ranges do.
inline bool rows_overlap(const Rows& a, const Rows& b) {
  if (!a.rows || !b.rows || !a.width || !b.width) return false;
  if (a.hi() <= b.lo || b.hi() <= a.lo) return false;
  if (a.stride != b.stride || a.rows == 1 || b.rows == 1) return true;
  const size_t s = a.stride;
  const size_t off = b.lo >= a.lo ? (size_t)(b.lo - a.lo) % s : (s - (size_t)(a.lo - b.lo) % s) % s;
  return off < a.width || off + b.width > s;
}

// FA_OK when the current device is one the kernels run on.
int require_device();

inline int check_scale_value(float scale) {
  return (std::isfinite(scale) && scale > 0.f) ? FA_OK : FA_ERR_INVALID_ARG;
}

}  // namespace fa
