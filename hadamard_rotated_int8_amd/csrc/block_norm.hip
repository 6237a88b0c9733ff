// The norms around a transformer block:
//   h = residual_scale x + gate * post(branch)
//   y = pre(h) * (1 + scale) + shift
// in one pass: each row stays in registers between the two norms, and y can
// leave as the FP8 packed activation of the linear that follows.
//
// Bound by HBM: x (and the branch) are read once, h and y written once.
// Statistics are float32; a layer norm's variance is taken of the
// differences from the mean (a second sum over the registers), so a large
// common offset costs no digits.
#include "fp8.h"
#include "kernels.h"

namespace convrot {
namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

constexpr int kMaxWaves = 16;

// Sum over the workgroup.  Every sum of a row has a `part` of its own, so one
// barrier suffices.
CR_DEVICE float group_sum(float v, float* part, int waves) {
  v += dpp_f32<kDppQuadSwap1>(v);
  v += dpp_f32<kDppQuadSwap2>(v);
  v += dpp_f32<kDppRowRor4>(v);
  v += dpp_f32<kDppRowRor8>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  if (waves > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < waves; ++w) v += part[w];
  }
  return v;
}

// Eight consecutive values from `at`, `left` of them inside the row (the
// rest are zero); loads need only the type's own alignment.
CR_DEVICE void load8(float* v, const void* p, bool bf16, int64_t at, int left) {
  if (bf16) {
    const uint16_t* s = static_cast<const uint16_t*>(p) + at;
    if (left >= 8) {
      u32x4 w;
      __builtin_memcpy(&w, s, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? __uint_as_float(unsigned(s[i]) << 16) : 0.f;
    }
  } else {
    const float* s = static_cast<const float*>(p) + at;
    if (left >= 8) {
      f32x4 w0, w1;
      __builtin_memcpy(&w0, s, 16);
      __builtin_memcpy(&w1, s + 4, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = w0[i];
        v[4 + i] = w1[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? s[i] : 0.f;
    }
  }
}

CR_DEVICE void store8(void* p, bool bf16, int64_t at, const float* v, int left) {
  if (bf16) {
    uint16_t* d = static_cast<uint16_t*>(p) + at;
    uint16_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
    if (left >= 8) {
      __builtin_memcpy(d, w, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) d[i] = w[i];
    }
  } else {
    float* d = static_cast<float*>(p) + at;
    if (left >= 8) {
      __builtin_memcpy(d, v, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) d[i] = v[i];
    }
  }
}

// Where the vector of a row starts.
CR_DEVICE int64_t vector_at(const VectorArgs& v, int64_t row) { return row / v.rows * v.stride; }

// Thread t holds features 8 (t + T c) .. +7 for c < CPT, T the workgroup size.
template <int CPT>
__global__ __launch_bounds__(1024) void block_norm_kernel(const BlockNormArgs a) {
  __shared__ float part[4][kMaxWaves];
  const int T = blockDim.x, waves = T >> 6, k = int(a.k);
  const float inv_k = 1.f / float(k);
  const int64_t row = blockIdx.x;

  auto normalise = [&](float (&v)[CPT][8], const NormArgs& n, int slot) {
    float mean = 0.f;
    if (n.kind == kNormLayer) {
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += v[c][i];
      mean = group_sum(sum, part[slot], waves) * inv_k;
    }
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int left = k - 8 * (int(threadIdx.x) + T * c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = v[c][i] - mean;
        v[c][i] = d;
        sq += i < left ? d * d : 0.f;
      }
    }
    const float r = 1.f / sqrtf(group_sum(sq, part[slot + 1], waves) * inv_k + n.eps);
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int f = 8 * (int(threadIdx.x) + T * c);
      if (f >= k) break;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= r;
      if (n.weight.p) {
        load8(w, n.weight.p, n.weight.bf16, f, k - f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= w[i];
      }
      if (n.bias.p) {
        load8(w, n.bias.p, n.bias.bf16, f, k - f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += w[i];
      }
    }
  };

  float h[CPT][8];
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int f = 8 * (int(threadIdx.x) + T * c);
    load8(h[c], a.x, a.x_bf16, row * a.ldx + f, f < k ? k - f : 0);
  }
  if (a.branch) {
    float b[CPT][8];
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int f = 8 * (int(threadIdx.x) + T * c);
      load8(b[c], a.branch, a.branch_bf16, row * a.ldb + f, f < k ? k - f : 0);
    }
    if (a.post.kind != kNormNone) normalise(b, a.post, 0);
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const int f = 8 * (int(threadIdx.x) + T * c);
      if (f >= k) break;
      float g[8];
      if (a.gate.p) {
        load8(g, a.gate.p, a.gate.bf16, vector_at(a.gate, row) + f, k - f);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = 1.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        h[c][i] = f + i < k ? __builtin_fmaf(g[i], b[c][i], h[c][i] * a.residual_scale) : 0.f;
      if (a.h) store8(a.h, a.x_bf16, row * a.ldh + f, h[c], k - f);
    }
  }
  if (!a.y && !a.q) return;
  if (a.pre.kind != kNormNone) normalise(h, a.pre, 2);
#pragma unroll
  for (int c = 0; c < CPT; ++c) {
    const int f = 8 * (int(threadIdx.x) + T * c);
    float w[8];
    if (f < k) {
      if (a.scale.p) {
        load8(w, a.scale.p, a.scale.bf16, vector_at(a.scale, row) + f, k - f);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] *= 1.f + w[i];
      }
      if (a.shift.p) {
        load8(w, a.shift.p, a.shift.bf16, vector_at(a.shift, row) + f, k - f);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] += w[i];
      }
    }
    if (a.q) {  // 16 neighbouring lanes hold one block of 128; k % 16 == 0
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
    } else if (f < k) {
      store8(a.y, a.y_bf16, row * a.ldy + f, h[c], k - f);
    }
  }
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream) {
  const int chunks = int((a.k + 7) / 8);
  const int cpt = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
  const int threads = ((chunks + cpt - 1) / cpt + 63) / 64 * 64;
  const dim3 grid(unsigned(a.m));
  if (cpt == 1)
    hipLaunchKernelGGL(block_norm_kernel<1>, grid, dim3(threads), 0, stream, a);
  else if (cpt == 2)
    hipLaunchKernelGGL(block_norm_kernel<2>, grid, dim3(threads), 0, stream, a);
  else
    hipLaunchKernelGGL(block_norm_kernel<4>, grid, dim3(threads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace convrot
