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

inline convrot_status from_hip(hipError_t e) {
  return e == hipSuccess ? CONVROT_OK : CONVROT_ERR_HIP;
}

}  // namespace convrot
