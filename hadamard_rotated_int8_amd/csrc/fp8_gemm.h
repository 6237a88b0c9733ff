// What the FP8 GEMM kernels share: their parameters, the order of the output
// tiles and the output's stores.
#pragma once

#include "fp8.h"
#include "kernels.h"

namespace convrot {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kBK = 128;  // features (bytes) per step: one scale block
constexpr int kGroupM = 4;
constexpr int kMaxBlocks = 1042;  // CONVROT_MAX_K / 128, rounded up to pairs

struct Fp8Params {
  const uint8_t* qx;
  const uint8_t* sx;
  int64_t lds;
  int M, K, kb;
  int nseg;
  int tiles_m, tiles_n;
  int y_bf16, gelu;
  int first;  // tile of the launch's first workgroup
  struct Seg {
    const uint8_t* qw;
    const void* sw;
    const float* bias;
    void* y;
    int64_t ldy;
    int n, tn0;
  } seg[kMaxGemmGroup];
};

struct Fp8Tile {
  int m0, n0, seg;
};

// Tile t of the output: groups of kGroupM tile rows are walked column by
// column, so that consecutive tiles (dealt XCD by XCD) share an L2.
template <int BM, int BN>
CR_DEVICE Fp8Tile fp8_tile(const Fp8Params& p, int t) {
  const int per_group = kGroupM * p.tiles_n;
  const int first = t / per_group * kGroupM;
  const int gm = p.tiles_m - first < kGroupM ? p.tiles_m - first : kGroupM;
  const int in = t % per_group;
  const int tm = first + in % gm, tn = in / gm;
  int s = 0, tn0 = 0;
#pragma unroll
  for (int i = 1; i < kMaxGemmGroup; ++i)
    if (i < p.nseg && tn >= p.seg[i].tn0) {
      s = i;
      tn0 = p.seg[i].tn0;
    }
  return {tm * BM, (tn - tn0) * BN, s};
}

// The kernel's parameters for BM x BN tiles.
template <int BM, int BN>
inline Fp8Params fp8_params(const Fp8GemmArgs& a) {
  Fp8Params p{};
  p.qx = a.qx;
  p.sx = a.sx;
  p.lds = a.lds;
  p.M = int(a.m);
  p.K = int(a.k);
  p.kb = int((a.k + kFp8Block - 1) / kFp8Block);
  p.nseg = a.count;
  p.y_bf16 = a.y_bf16;
  p.gelu = a.gelu;
  p.tiles_m = int((a.m + BM - 1) / BM);
  for (int i = 0; i < a.count; ++i) {
    p.seg[i] = {a.w[i].q, a.w[i].scale, a.w[i].bias, a.w[i].y, a.w[i].ldy, int(a.w[i].n), p.tiles_n};
    p.tiles_n += int((a.w[i].n + BN - 1) / BN);
  }
  return p;
}

CR_DEVICE unsigned bf16_pair(float a, float b) {  // two values to nearest even
  return unsigned(__builtin_bit_cast(uint16_t, (__bf16)a)) |
         unsigned(__builtin_bit_cast(uint16_t, (__bf16)b)) << 16;
}

// Four consecutive columns of one output row; `whole` when all four exist and
// the row allows a vector store.
CR_DEVICE void store4(void* y, int64_t at, const float* v, int left, bool bf16, bool whole) {
  if (bf16) {
    uint16_t* p = static_cast<uint16_t*>(y) + at;
    const u32x2 w = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    if (whole) {
      *reinterpret_cast<u32x2*>(p) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = uint16_t(w[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    float* p = static_cast<float*>(y) + at;
    if (whole) {
      *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = v[i];
    }
  }
}

// The float32 value of an E8M0 byte (255 is NaN; 0 is 2^-127, a subnormal).
CR_DEVICE float e8m0_value(unsigned s) {
  return __uint_as_float(s == 0 ? 0x400000u : s == kFp8ScaleNan ? 0x7FC00000u : s << 23);
}

// 32 E4M3 codes times a power of two, as four bfloat16 operands.
struct Bf16Frag {
  bf16x8 v[4];
};
CR_DEVICE Bf16Frag to_bf16(v8i q, float scale) {
  Bf16Frag r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(q[i]), scale, false);
    const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(unsigned(q[i]), scale, true);
    r.v[i / 2][4 * (i & 1)] = lo[0];
    r.v[i / 2][4 * (i & 1) + 1] = lo[1];
    r.v[i / 2][4 * (i & 1) + 2] = hi[0];
    r.v[i / 2][4 * (i & 1) + 3] = hi[1];
  }
  return r;
}
}  // namespace convrot
