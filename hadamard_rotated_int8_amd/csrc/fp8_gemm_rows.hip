// FP8 linear for a few rows of X as they are (one token, a small batch), in one
// launch: the weights are read once, straight into registers, and that is what
// takes the time.
//
// A workgroup owns 32 rows of W (16 where that leaves CUs without one); its 8
// waves share the blocks of 128 features round robin (so that they read
// neighbouring lines) and add their sums in LDS in wave order.  Each wave
// requests kAhead blocks of W at once, two 16-byte loads per lane and 16 rows,
// each instruction 16 rows x 64 bytes.
//
// Every workgroup quantises X into LDS while its first W loads are on their
// way, which is less than a second launch costs.  (Each wave quantising its
// own blocks in registers took 6 us more for one row of 5120 through 13824.)
// One instruction of 16 x 16 x 128 (or, for float32 outputs, four of bfloat16
// on converted codes, see fp8_gemm.hip) multiplies 16 rows of W with up to 16
// rows of X.
//
// One row, 5120 -> 13824 (71 MB): 15.3 us, 4.6 TB/s.  With 1, 2 and 4 blocks
// requested at once instead of 3 it took about the same or spilled; 16 rows
// of W per workgroup: 16.7; 4096 -> 4096: 8.1 us with 32 rows, 6.5 with 16.
#include <type_traits>

#include "fp8_gemm.h"

namespace convrot {
namespace {

constexpr int kWaves = 8;
constexpr int kAhead = 3;   // blocks requested at once

// ROW_HALF_MIRROR: lane i of each group of 8 reads lane 7 - i.
constexpr int kDppHalfMirror = 0x141;

// Sixteen consecutive features of X, 16-byte aligned.
CR_DEVICE void load16(float* v, const void* x, bool bf16, int64_t at) {
  if (bf16) {
    const u32x4* src = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at);
    const u32x4 a[2] = {src[0], src[1]};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = bf16_lo(a[i / 4][i % 4]);
      v[2 * i + 1] = bf16_hi(a[i / 4][i % 4]);
    }
  } else {
    const f32x4* src = reinterpret_cast<const f32x4*>(static_cast<const float*>(x) + at);
    const f32x4 a[4] = {src[0], src[1], src[2], src[3]};
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = a[i / 4][i % 4];
  }
}

// NT: 16-row groups of W.
template <int NT, bool F32SCALE, bool EXACT>
__global__ __launch_bounds__(kWaves * 64, 4) void fp8_rows_kernel(const Fp8Params p, const void* x, int64_t ldx,
                                                                  bool x_bf16) {
  constexpr int kRows = 16 * NT;
  __shared__ float part[kWaves][NT][64][4];
  __shared__ __attribute__((aligned(16))) uint8_t xlds[kFp8RawBytes];  // codes [M][128 kb]
  __shared__ uint8_t slds[kFp8RawBytes / kBK];                         // scales [M][kb]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fg = lane >> 4;
  const int K = p.K, kb = p.kb;
  const int tile = p.first + int(blockIdx.x);
  int s = 0;
  for (int i = 1; i < p.nseg; ++i)
    if (tile >= p.seg[i].tn0) s = i;
  const Fp8Params::Seg& sg = p.seg[s];
  const int n0 = (tile - sg.tn0) * kRows;
  const int cols = sg.n - n0 < kRows ? sg.n - n0 : kRows;
  const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(sg.qw + (int64_t)n0 * K, cols * K);

  // Lane l: row l % 16 of 16, features 16 g .. +15 and 64 + 16 g .. +15 of a
  // block, g = l / 16 (both operands alike).
  f32x4 acc[NT] = {};
  v4i w[kAhead][NT][2];
  auto load_w = [&](int b0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int f = (b0 + kWaves * u) * kBK + 64 * c + 16 * fg;
          w[u][t][c] = __builtin_bit_cast(
              v4i, __builtin_amdgcn_raw_buffer_load_b128(
                       wr, f < K ? unsigned((16 * t + fr) * K + f) : kOutOfRange, 0, 0));
        }
  };
  load_w(wave);
  // X: 8 threads to a block, 16 features each.
  for (int i = threadIdx.x >> 3; i < p.M * kb; i += kWaves * 8) {
    const int row = i / kb, b = i - row * kb, f = b * kBK + 16 * int(threadIdx.x & 7);
    float v[16];
    if (f < K) {
      load16(v, x, x_bf16, row * ldx + f);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = 0.f;
    }
    unsigned top = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) top = max(top, abs_bits(v[e]));
    top = max(top, dpp_u32<kDppQuadSwap1>(top));
    top = max(top, dpp_u32<kDppQuadSwap2>(top));
    top = max(top, dpp_u32<kDppHalfMirror>(top));
    const unsigned sc = fp8_scale_of(top);
    const float inv = fp8_inverse_scale(sc);
    u32x4 q;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      q[e] = sc == kFp8ScaleNan ? kFp8CodeNan
                                : fp8_codes4(v[4 * e] * inv, v[4 * e + 1] * inv, v[4 * e + 2] * inv,
                                             v[4 * e + 3] * inv);
    *reinterpret_cast<u32x4*>(xlds + (row * kb + b) * kBK + 16 * (threadIdx.x & 7)) = q;
    if ((threadIdx.x & 7) == 0) slds[row * kb + b] = uint8_t(sc);
  }
  wait_lgkm0();  // (not __syncthreads, which may wait for W)
  barrier();
  for (int b0 = wave; b0 < kb; b0 += kWaves * kAhead) {
    if (b0 != wave) load_w(b0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int b = b0 + kWaves * u;
      if (b >= kb) break;
      v4i x0 = {}, x1 = {};
      int sx = 127;
      if (fr < p.M) {
        const uint8_t* src = xlds + (fr * kb + b) * kBK + 16 * fg;
        x0 = *reinterpret_cast<const v4i*>(src);
        x1 = *reinterpret_cast<const v4i*>(src + 64);
        sx = slds[fr * kb + b];
      }
      const v8i xq = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
      const int64_t at = (int64_t)(n0 / kFp8Block) * kb + b;
      float sf = 1.f;
      int se = 127;
      if constexpr (F32SCALE)
        sf = static_cast<const float*>(sg.sw)[at];
      else
        se = static_cast<const uint8_t*>(sg.sw)[at];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const v4i* q = w[u][j];
        const v8i wq = {q[0][0], q[0][1], q[0][2], q[0][3], q[1][0], q[1][1], q[1][2], q[1][3]};
        if constexpr (EXACT) {
          const Bf16Frag wf = to_bf16(wq, F32SCALE ? 1.f : e8m0_value(se));
          const Bf16Frag xf = to_bf16(xq, e8m0_value(sx));
          f32x4 c = F32SCALE ? f32x4{} : acc[j];
#pragma unroll
          for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf.v[i], xf.v[i], c, 0, 0, 0);
          if constexpr (F32SCALE) {
#pragma unroll
            for (int e = 0; e < 4; ++e) c[e] = __builtin_fmaf(c[e], sf, acc[j][e]);
          }
          acc[j] = c;
        } else if constexpr (F32SCALE) {
          const f32x4 c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wq, xq, f32x4{}, 0, 0, 0, 127, 0, sx);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = __builtin_fmaf(c[e], sf, acc[j][e]);
        } else {
          acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wq, xq, acc[j], 0, 0, 0, se, 0, sx);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) *reinterpret_cast<f32x4*>(part[wave][j][lane]) = acc[j];
  __syncthreads();
  // Element e of lane l in group j: column 16 j + 4 (l / 16) + e, row l % 16.
  if (wave < NT) {
    f32x4 v = *reinterpret_cast<const f32x4*>(part[0][wave][lane]);
#pragma unroll
    for (int i = 1; i < kWaves; ++i) v += *reinterpret_cast<const f32x4*>(part[i][wave][lane]);
    const int n = n0 + 16 * wave + 4 * fg, row = fr;
    if (row < p.M && n < sg.n) {
      float o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[e] = v[e];
        if (sg.bias && n + e < sg.n) o[e] += sg.bias[n + e];
        if (p.gelu) o[e] = gelu_erf(o[e]);
      }
      const bool vec = (sg.ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(sg.y) & (p.y_bf16 ? 7 : 15)) == 0;
      store4(sg.y, row * sg.ldy + n, o, sg.n - n, p.y_bf16, vec && sg.n - n >= 4);
    }
  }
}

template <int NT>
void launch_t(const Fp8GemmArgs& a, hipStream_t stream) {
  Fp8Params p = fp8_params<16, 16 * NT>(a);
  auto go = [&](auto f32, auto exact) {
    in_launches(p.tiles_n, kWaves * 64, [&](int64_t first, unsigned count) {
      p.first = int(first);
      hipLaunchKernelGGL((fp8_rows_kernel<NT, decltype(f32)::value, decltype(exact)::value>), dim3(count),
                         dim3(kWaves * 64), 0, stream, p, a.x, a.ldx, a.x_bf16);
    });
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
  int64_t groups = 0;
  for (int i = 0; i < a.count; ++i) groups += (a.w[i].n + 31) / 32;
  if (groups < device_cu_count())
    launch_t<1>(a, stream);
  else
    launch_t<2>(a, stream);
  return hipGetLastError();
}

}  // namespace convrot
