// FP8 linear for few rows of X (one token, a small batch): the weights are
// read once, straight into registers, and that is what takes the time.
//
// A workgroup owns 32 rows of W; its 8 waves share the blocks of 128 features
// round robin (so that they read neighbouring lines) and add their sums in
// LDS in wave order.  Each wave requests kAhead blocks of W at once, two
// 16-byte loads per lane and 16 rows, each instruction 16 rows x 64 bytes;
// with 16 waves on a CU that is far more than HBM needs in flight.
//
// One instruction of 16 x 16 x 128 (or, for float32 outputs, four of bfloat16
// on converted codes, see fp8_gemm.hip) multiplies 16 rows of W with 16 rows
// of X.  X comes packed, or, for up to 16 rows, as it is: each wave then
// quantises its own blocks in registers while W is on its way, which is less
// than a second launch costs.
#include <type_traits>

#include "fp8_gemm.h"

namespace convrot {
namespace {

constexpr int kWaves = 8;
constexpr int kRows = 32;   // of W per workgroup
constexpr int kNT = kRows / 16;
constexpr int kAhead = 4;   // blocks requested at once
enum { kPacked = 0, kRawBf16 = 1, kRawF32 = 2 };

// The maximum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
CR_DEVICE unsigned max_over_groups(unsigned a) {
  const auto h = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  a = max(h[0], h[1]);
  const auto q = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  return max(q[0], q[1]);
}

template <int MT, int XSRC, bool F32SCALE, bool EXACT>
__global__ __launch_bounds__(kWaves * 64) void fp8_rows_kernel(const Fp8Params p, const void* x, int64_t ldx) {
  __shared__ float part[kWaves][kNT * MT][64][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fg = lane >> 4;
  const int K = p.K, kb = p.kb;
  int s = 0;
  for (int i = 1; i < p.nseg; ++i)
    if (int(blockIdx.x) >= p.seg[i].tn0) s = i;
  const Fp8Params::Seg& sg = p.seg[s];
  const int n0 = (int(blockIdx.x) - sg.tn0) * kRows;
  const int cols = sg.n - n0 < kRows ? sg.n - n0 : kRows;
  const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(sg.qw + (int64_t)n0 * K, cols * K);

  // Lane l: row l % 16 of 16, features 16 g .. +15 and 64 + 16 g .. +15 of a
  // block, g = l / 16 (both operands alike).
  f32x4 acc[kNT][MT] = {};
  for (int b0 = wave; b0 < kb; b0 += kWaves * kAhead) {
    v4i w[kAhead][kNT][2];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int t = 0; t < kNT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int f = (b0 + kWaves * u) * kBK + 64 * c + 16 * fg;
          w[u][t][c] = __builtin_bit_cast(
              v4i, __builtin_amdgcn_raw_buffer_load_b128(
                       wr, f < K ? unsigned((16 * t + fr) * K + f) : kOutOfRange, 0, 0));
        }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int b = b0 + kWaves * u;
      if (b >= kb) break;
      v8i xq[MT];
      unsigned sx[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int row = 16 * t + fr;
        if constexpr (XSRC == kPacked) {
          v4i q[2] = {};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int f = b * kBK + 64 * c + 16 * fg;
            if (row < p.M && f < K) q[c] = *reinterpret_cast<const v4i*>(p.qx + (int64_t)row * K + f);
          }
          xq[t] = v8i{q[0][0], q[0][1], q[0][2], q[0][3], q[1][0], q[1][1], q[1][2], q[1][3]};
          sx[t] = row < p.M ? p.sx[b * p.lds + row] : 127u;
        } else {
          float v[2][16];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int f = b * kBK + 64 * c + 16 * fg;
            if (row < p.M && f < K) {  // K % 16 == 0
              if constexpr (XSRC == kRawBf16) {
                const u32x4* src = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + row * ldx + f);
                const u32x4 a0 = src[0], a1 = src[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  v[c][2 * i] = bf16_lo(a0[i]);
                  v[c][2 * i + 1] = bf16_hi(a0[i]);
                  v[c][8 + 2 * i] = bf16_lo(a1[i]);
                  v[c][9 + 2 * i] = bf16_hi(a1[i]);
                }
              } else {
                const f32x4* src = reinterpret_cast<const f32x4*>(static_cast<const float*>(x) + row * ldx + f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const f32x4 a = src[i];
#pragma unroll
                  for (int e = 0; e < 4; ++e) v[c][4 * i + e] = a[e];
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[c][i] = 0.f;
            }
          }
          unsigned top = 0;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = max(top, abs_bits(v[c][i]));
          top = max_over_groups(top);
          sx[t] = fp8_scale_of(top);
          const float inv = fp8_inverse_scale(sx[t]);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              xq[t][4 * c + i] = int(sx[t] == kFp8ScaleNan
                                         ? kFp8CodeNan
                                         : fp8_codes4(v[c][4 * i] * inv, v[c][4 * i + 1] * inv,
                                                      v[c][4 * i + 2] * inv, v[c][4 * i + 3] * inv));
        }
      }
      const int64_t at = (int64_t)(n0 / kFp8Block) * kb + b;
      float sf = 1.f;
      int se = 127;
      if constexpr (F32SCALE)
        sf = static_cast<const float*>(sg.sw)[at];
      else
        se = static_cast<const uint8_t*>(sg.sw)[at];
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        const v4i* q = w[u][j];
        const v8i wq = {q[0][0], q[0][1], q[0][2], q[0][3], q[1][0], q[1][1], q[1][2], q[1][3]};
        if constexpr (EXACT) {
          const Bf16Frag wf = to_bf16(wq, F32SCALE ? 1.f : e8m0_value(se));
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const Bf16Frag xf = to_bf16(xq[t], e8m0_value(sx[t]));
            f32x4 c = F32SCALE ? f32x4{} : acc[j][t];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf.v[i], xf.v[i], c, 0, 0, 0);
            if constexpr (F32SCALE) {
#pragma unroll
              for (int e = 0; e < 4; ++e) c[e] = __builtin_fmaf(c[e], sf, acc[j][t][e]);
            }
            acc[j][t] = c;
          }
        } else {
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            if constexpr (F32SCALE) {
              const f32x4 c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wq, xq[t], f32x4{}, 0, 0, 0, 127,
                                                                               0, int(sx[t]));
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[j][t][e] = __builtin_fmaf(c[e], sf, acc[j][t][e]);
            } else {
              acc[j][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wq, xq[t], acc[j][t], 0, 0, 0, se, 0,
                                                                           int(sx[t]));
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kNT; ++j)
#pragma unroll
    for (int t = 0; t < MT; ++t) *reinterpret_cast<f32x4*>(part[wave][j * MT + t][lane]) = acc[j][t];
  __syncthreads();
  // Element e of lane l in group (j, t): column 16 j + 4 (l / 16) + e, row 16 t + l % 16.
  for (int g = wave; g < kNT * MT; g += kWaves) {
    f32x4 v = *reinterpret_cast<const f32x4*>(part[0][g][lane]);
#pragma unroll
    for (int i = 1; i < kWaves; ++i) v += *reinterpret_cast<const f32x4*>(part[i][g][lane]);
    const int n = n0 + 16 * (g / MT) + 4 * fg, row = 16 * (g % MT) + fr;
    if (row < p.M && n < sg.n) {
      float o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[e] = v[e];
        if (sg.bias && n + e < sg.n) o[e] += sg.bias[n + e];
        if (p.gelu) o[e] = gelu_erf(o[e]);
      }
      const bool vec = (sg.ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(sg.y) & (p.y_bf16 ? 7 : 15)) == 0;
      store4(sg.y, row * sg.ldy + n, o, sg.n - n, p.y_bf16, vec && n + 4 <= sg.n);
    }
  }
}

template <int MT, int XSRC>
void launch_t(const Fp8GemmArgs& a, const Fp8Params& p, dim3 grid, hipStream_t stream) {
  auto go = [&](auto f32, auto exact) {
    hipLaunchKernelGGL((fp8_rows_kernel<MT, XSRC, decltype(f32)::value, decltype(exact)::value>), grid,
                       dim3(kWaves * 64), 0, stream, p, a.x, a.ldx);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  if (a.f32_scale) {
    if (a.y_bf16) go(Yes{}, No{}); else go(Yes{}, Yes{});
  } else {
    if (a.y_bf16) go(No{}, No{}); else go(No{}, Yes{});
  }
}

}  // namespace

hipError_t launch_fp8_gemm_rows(const Fp8GemmArgs& a, hipStream_t stream) {
  const Fp8Params p = fp8_params<16, kRows>(a);
  const dim3 grid(unsigned(p.tiles_n));
  if (a.x)
    a.x_bf16 ? launch_t<1, kRawBf16>(a, p, grid, stream) : launch_t<1, kRawF32>(a, p, grid, stream);
  else if (a.m <= 16)
    launch_t<1, kPacked>(a, p, grid, stream);
  else if (a.m <= 32)
    launch_t<2, kPacked>(a, p, grid, stream);
  else
    launch_t<4, kPacked>(a, p, grid, stream);
  return hipGetLastError();
}

}  // namespace convrot
