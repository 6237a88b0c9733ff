// What the host-side argument checks of the C ABI share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/convrot.h"

namespace convrot {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

inline bool aligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
inline bool aligned16(const void* p) { return aligned(p, 16); }

// The addresses of [rows, cols] values with a row stride, from the first byte to
// behind the last; none without an element.
struct Range {
  uintptr_t lo, hi;
};
inline Range range_of(const void* p, int64_t rows, int64_t stride, int64_t cols, unsigned size) {
  if (!p || rows < 1 || cols < 1) return {0, 0};
  const uintptr_t at = reinterpret_cast<uintptr_t>(p), most = UINTPTR_MAX - at;
  const __int128 bytes = ((__int128)(rows - 1) * stride + cols) * size;
  return {at, at + (bytes < (__int128)most ? uintptr_t(bytes) : most)};
}
inline bool meet(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

inline convrot_status from_hip(hipError_t e) {
  return e == hipSuccess ? CONVROT_OK : CONVROT_ERR_HIP;
}

}  // namespace convrot
