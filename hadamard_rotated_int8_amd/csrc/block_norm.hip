// The norms around a transformer block:
//   h = residual_scale x + gate * post(branch)
//   y = pre(h) * (1 + scale) + shift
// in one pass: each row stays in registers between the two norms, and y can
// leave as the FP8 packed activation of the linear that follows.
//
// Bound by HBM: x (and the branch) are read once, h and y written once.
// Statistics are float32; a layer norm's variance is taken of the
// differences from the mean (a second sum over the registers).  A float32
// mean is itself off by some 2^-24 of the rows' common part, and so is every
// difference; the differences' own mean, summed with their squares, takes
// that off again, so a large common part costs no digits.
#include <type_traits>

#include "fp8.h"
#include "kernels.h"

namespace convrot {
namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kMaxWaves = 16;
enum { kBf16 = 0, kF32 = 1, kAbsent = 2 };  // types of x and branch

// ROW_HALF_MIRROR and ROW_MIRROR: lane i of each 8 reads lane 7 - i, of each
// 16 lane 15 - i.
constexpr int kDppHalfMirror = 0x141, kDppMirror = 0x140;

// Every step adds two sums that both lanes of a pair hold, so all lanes get
// the same bits.  (A rotation by 4 would add in another order in every lane,
// and lanes would take off different means.)
CR_DEVICE float wave_sum(float v) {
  v += dpp_f32<kDppQuadSwap1>(v);
  v += dpp_f32<kDppQuadSwap2>(v);
  v += dpp_f32<kDppHalfMirror>(v);
  v += dpp_f32<kDppMirror>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// Sums over the row's waves.  Every sum of a row has a `part` of its own, so
// one barrier suffices.
CR_DEVICE float row_sum(float v, float2* part, int waves) {
  v = wave_sum(v);
  if (waves > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6].x = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < waves; ++w) v += part[w].x;
  }
  return v;
}
CR_DEVICE float2 row_sums(float u, float v, float2* part, int waves) {
  u = wave_sum(u);
  v = wave_sum(v);
  if (waves > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_float2(u, v);
    __syncthreads();
    u = v = 0.f;
    for (int w = 0; w < waves; ++w) {
      u += part[w].x;
      v += part[w].y;
    }
  }
  return make_float2(u, v);
}

// Eight consecutive values; loads need only the type's own alignment.
CR_DEVICE void load_bf16x8(float* v, const uint16_t* s) {
  u32x4 w;
  __builtin_memcpy(&w, s, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}
CR_DEVICE void load_f32x8(float* v, const float* s) {
  f32x4 w0, w1;
  __builtin_memcpy(&w0, s, 16);
  __builtin_memcpy(&w1, s + 4, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = w0[i];
    v[4 + i] = w1[i];
  }
}
CR_DEVICE float load1(const void* p, bool bf16, int64_t at) {
  return bf16 ? __uint_as_float(unsigned(static_cast<const uint16_t*>(p)[at]) << 16)
              : static_cast<const float*>(p)[at];
}

// Where the vector of a row starts.
CR_DEVICE int64_t vector_at(const VectorArgs& v, int64_t row) { return row / v.rows * v.stride; }

// Lane l of wave w of a row (of W waves) holds features 8 (l + 64 w + 64 W c)
// .. +7 for c < CPT; a row of k % 8 == 0 features (WHOLE) has no chunk that is
// partly outside.  A row's W waves are one workgroup, or (W = 1) a workgroup
// is four rows that never wait for one another.
template <int CPT, int XT, int BT, bool WHOLE, int MAXT>
__global__ __launch_bounds__(MAXT) void block_norm_kernel(const BlockNormArgs a) {
  __shared__ float2 part[4][kMaxWaves];
  const bool alone = MAXT == 256 && a.waves == 1;
  const int T = 64 * a.waves;
  const int t0 = alone ? int(threadIdx.x & 63) : int(threadIdx.x);
  const int64_t block = a.first + blockIdx.x;
  const int64_t row = alone ? block * 4 + (threadIdx.x >> 6) : block;
  if (row >= a.m) return;  // (whole waves, and with W > 1 none)
  const int k = int(a.k);
  const float inv_k = 1.f / float(k);

  auto feature = [&](int c) { return 8 * (t0 + T * c); };
  // Values of one row or vector; those outside are zero.
  auto load = [&](float (&v)[CPT][8], const void* p, bool bf16, int64_t at) {
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int f = feature(c);
      if constexpr (WHOLE) {
        const int64_t i = at + (f < k ? f : 0);
        if (bf16)
          load_bf16x8(v[c], static_cast<const uint16_t*>(p) + i);
        else
          load_f32x8(v[c], static_cast<const float*>(p) + i);
        if (f >= k) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] = 0.f;
        }
      } else if (f + 8 <= k) {
        if (bf16)
          load_bf16x8(v[c], static_cast<const uint16_t*>(p) + at + f);
        else
          load_f32x8(v[c], static_cast<const float*>(p) + at + f);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = f + i < k ? load1(p, bf16, at + f + i) : 0.f;
      }
    }
  };
  auto store = [&](void* p, bool bf16, int64_t at, int c, const float* v) {
    const int f = feature(c);
    if (WHOLE ? f < k : f + 8 <= k) {
      if (bf16) {
        uint16_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
        __builtin_memcpy(static_cast<uint16_t*>(p) + at + f, w, 16);
      } else {
        __builtin_memcpy(static_cast<float*>(p) + at + f, v, 32);
      }
    } else if (!WHOLE) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (f + i < k) {
          if (bf16)
            static_cast<uint16_t*>(p)[at + f + i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
          else
            static_cast<float*>(p)[at + f + i] = v[i];
        }
    }
  };
  auto normalise = [&](float (&v)[CPT][8], const NormArgs& n, int slot) {
    const bool layer = n.kind == kNormLayer;
    float mean = 0.f;
    if (layer) {
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[c][i];
      mean = row_sum(sum, part[slot], a.waves) * inv_k;
    }
    float sum = 0.f, sq = 0.f;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int left = k - feature(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float d = v[c][i] - mean;
        v[c][i] = d;
        d = (WHOLE ? left > 0 : i < left) ? d : 0.f;
        sum += d;
        sq += d * d;
      }
    }
    const float2 s = row_sums(sum, sq, part[slot + 1], a.waves);
    const float rest = layer ? s.x * inv_k : 0.f;  // of the mean
    const float var = s.y * inv_k - rest * rest;
    const float r = 1.f / sqrtf((var < 0.f ? 0.f : var) + n.eps);  // (a NaN stays one)
    const float back = rest != 0.f ? -rest * r : -0.f;             // (r may be infinite)
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = __builtin_fmaf(v[c][i], r, back);
    if (n.weight.p) {
      float w[CPT][8];
      load(w, n.weight.p, n.weight.bf16, 0);
#pragma unroll
      for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= w[c][i];
    }
    if (n.bias.p) {
      float w[CPT][8];
      load(w, n.bias.p, n.bias.bf16, 0);
#pragma unroll
      for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += w[c][i];
    }
  };

  float h[CPT][8];
  load(h, a.x, XT == kBf16, row * a.ldx);
  if constexpr (BT != kAbsent) {
    float b[CPT][8];
    load(b, a.branch, BT == kBf16, row * a.ldb);
    if (a.post.kind != kNormNone) normalise(b, a.post, 0);
    if (a.gate.p) {
      float g[CPT][8];
      load(g, a.gate.p, a.gate.bf16, vector_at(a.gate, row));
#pragma unroll
      for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) b[c][i] *= g[c][i];
    }
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int left = k - feature(c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = __builtin_fmaf(h[c][i], a.residual_scale, b[c][i]);
        h[c][i] = (WHOLE ? left > 0 : i < left) ? v : 0.f;
      }
      if (a.h) store(a.h, XT == kBf16, row * a.ldh, c, h[c]);
    }
    if (!a.y && !a.q) return;
  }
  if (a.pre.kind != kNormNone) normalise(h, a.pre, 2);
  if (a.scale.p) {
    float w[CPT][8];
    load(w, a.scale.p, a.scale.bf16, vector_at(a.scale, row));
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] *= 1.f + w[c][i];
  }
  if (a.shift.p) {
    float w[CPT][8];
    load(w, a.shift.p, a.shift.bf16, vector_at(a.shift, row));
#pragma unroll
    for (int c = 0; c < CPT; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] += w[c][i];
  }
  if (!a.q) {
#pragma unroll
    for (int c = 0; c < CPT; ++c) store(a.y, a.y_bf16, row * a.ldy, c, h[c]);
    return;
  }
#pragma unroll
  for (int c = 0; c < CPT; ++c) {  // 16 neighbouring lanes hold one block of 128; k % 16 == 0
    const int f = feature(c);
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, f < k ? abs_bits(h[c][i]) : 0u);
    top = max(top, dpp_u32<kDppQuadSwap1>(top));
    top = max(top, dpp_u32<kDppQuadSwap2>(top));
    top = max(top, dpp_u32<kDppRowRor4>(top));
    top = max(top, dpp_u32<kDppRowRor8>(top));
    const unsigned s = fp8_scale_of(top);
    const float inv = fp8_inverse_scale(s);
    u32x2 codes;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      codes[i] = s == kFp8ScaleNan ? kFp8CodeNan
                                   : fp8_codes4(h[c][4 * i] * inv, h[c][4 * i + 1] * inv,
                                                h[c][4 * i + 2] * inv, h[c][4 * i + 3] * inv);
    if (f < k) {
      *reinterpret_cast<u32x2*>(a.q + row * k + f) = codes;
      if ((threadIdx.x & 15) == 0) a.q_scale[(f / kFp8Block) * a.lds + row] = uint8_t(s);
    }
  }
}

template <int CPT, int XT, int BT, int MAXT>
void launch_t(const BlockNormArgs& a, hipStream_t stream) {
  const bool alone = a.waves == 1;
  const int threads = alone ? 256 : 64 * a.waves;
  in_launches(alone ? (a.m + 3) / 4 : a.m, threads, [&](int64_t first, unsigned count) {
    BlockNormArgs part = a;
    part.first = first;
    if (a.k % 8 == 0)
      hipLaunchKernelGGL((block_norm_kernel<CPT, XT, BT, true, MAXT>), dim3(count), dim3(threads), 0, stream, part);
    else
      hipLaunchKernelGGL((block_norm_kernel<CPT, XT, BT, false, MAXT>), dim3(count), dim3(threads), 0, stream, part);
  });
}

template <int CPT, int MAXT>
void launch_types(const BlockNormArgs& a, hipStream_t stream) {
  auto branch = [&](auto xt) {
    constexpr int XT = decltype(xt)::value;
    if (!a.branch)
      launch_t<CPT, XT, kAbsent, MAXT>(a, stream);
    else if (a.branch_bf16)
      launch_t<CPT, XT, kBf16, MAXT>(a, stream);
    else
      launch_t<CPT, XT, kF32, MAXT>(a, stream);
  };
  if (a.x_bf16)
    branch(std::integral_constant<int, kBf16>{});
  else
    branch(std::integral_constant<int, kF32>{});
}

}  // namespace

// Two chunks per thread and as many waves per row as that takes, up to 16:
// a row of 5120 features has 5 waves.  Measured at 32760 x 5120 (float32
// branch and gate onto a bfloat16 stream, both norms, shift and scale) with
// 1, 2, 3, 4, 5 and 10 waves per row: 497, 332, 434, 326, 327 and 365 us;
// norm, shift and scale of 4096 x 5120 bfloat16: 22.1, 19.5, 24.1, 19.3, 18.5
// and 26.7 us.  (One wave holds 80 values a lane and few rows are in flight;
// ten wait for one another longer; three leave a third of the last chunk's
// lanes idle.  The mean's own correction came later and costs 1 to 2 %: 332 us
// and 19.1 with 5 waves.)
hipError_t launch_block_norm(const BlockNormArgs& args, hipStream_t stream) {
  BlockNormArgs a = args;
  const int chunks = int((a.k + 7) / 8);
  a.waves = (chunks + 127) / 128 < kMaxWaves ? (chunks + 127) / 128 : kMaxWaves;
  const int cpt = (chunks + 64 * a.waves - 1) / (64 * a.waves);
  if (cpt <= 1)
    launch_types<1, 256>(a, stream);
  else if (cpt <= 2 && a.waves <= 4)
    launch_types<2, 256>(a, stream);
  else if (cpt <= 2)
    launch_types<2, 1024>(a, stream);
  else
    launch_types<4, 1024>(a, stream);
  return hipGetLastError();
}

}  // namespace convrot
