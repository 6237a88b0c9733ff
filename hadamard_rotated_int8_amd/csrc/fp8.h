// E4M3 blocks with power-of-two scales: what the FP8 kernels share.
#pragma once

#include "common.h"

namespace convrot {

constexpr int kFp8Block = 128;         // features (and weight rows) that share one scale
constexpr unsigned kFp8ScaleNan = 255;  // the E8M0 code of NaN
constexpr unsigned kFp8CodeNan = 0x7F7F7F7Fu;  // four E4M3 NaNs

// The E8M0 byte of a block whose largest magnitude has the float32 bits `a`:
// the least e in [-126, 127] with a <= 448 2^e, as e + 127.  448 = 1.75 2^8,
// so e is a's exponent less 8, and one more where a's significand is above
// 1.75.  A zero block takes 2^0, one that holds an infinity or a NaN the NaN.
CR_DEVICE unsigned fp8_scale_of(unsigned a) {
  const int e = int(a >> 23) - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  const unsigned s = unsigned(e > 1 ? e : 1);
  return a >= 0x7F800000u ? kFp8ScaleNan : a == 0 ? 127u : s;
}

// 2^-e of a finite scale byte; the product with any value of the block is
// exact, or so small that its code is zero either way.
CR_DEVICE float fp8_inverse_scale(unsigned s) { return __uint_as_float((254u - s) << 23); }

// Four values (already divided by the scale) to E4M3, to nearest even.
CR_DEVICE unsigned fp8_codes4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return unsigned(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

CR_DEVICE unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int kCtrl>
CR_DEVICE unsigned dpp_u32(unsigned v) {
  return unsigned(__builtin_amdgcn_update_dpp(0, int(v), kCtrl, 0xF, 0xF, false));
}

}  // namespace convrot
