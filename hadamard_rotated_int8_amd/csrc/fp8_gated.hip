// The gated pair of projections with many tiles, act(X Wg^T + bg) * (X Wu^T +
// bu) in one kernel (fp8_wide.h), its way back to the projections, and the
// weights' transpose, on which the way back to X is a linear like any other.
// 4096 x 5120 -> 13824, 1728 tiles on 256 CUs: 490 us with both projections
// kept (2.4 PFLOP/s), bound by power (1.96 of 2.4 GHz) and the stores of 340 MB
// of outputs: the matrix cores are busy in 54 % of the cycles (72 % in the wide
// kernel without them).
#include "fp8_wide.h"

namespace convrot {
namespace {

template <bool F32, int MODE>
__global__ __launch_bounds__(256, 1) void fp8_gated_wide_kernel(const Fp8Params p, int total) {
  fp8_wide<false, F32, MODE>(p, total);
}

template <bool F32, int MODE>
void launch_wide_t(const Fp8GemmArgs& a, hipStream_t stream) {
  const Fp8Params p = fp8_params<kBM, WideCfg<F32, MODE>::BN>(a);
  const int total = p.tiles_m * p.tiles_n;
  const int cus = device_cu_count();
  hipLaunchKernelGGL((fp8_gated_wide_kernel<F32, MODE>), dim3(total < cus ? total : cus), dim3(256), 0, stream, p,
                     total);
}

// ROW_HALF_MIRROR: lane i of each group of 8 reads lane 7 - i.
constexpr int kDppHalfMirror = 0x141;

// Sixteen features from f of row r, of n; those behind are zero.
template <bool BF16>
CR_DEVICE void load16(float* v, const void* p, int64_t at, int left) {
  if (left >= 16) {
    if constexpr (BF16) {
      u32x4 w[2];  // (loads need only the type's own alignment)
      __builtin_memcpy(w, static_cast<const uint16_t*>(p) + at, 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[2 * i] = bf16_lo(w[i / 4][i % 4]);
        v[2 * i + 1] = bf16_hi(w[i / 4][i % 4]);
      }
    } else {
      __builtin_memcpy(v, static_cast<const float*>(p) + at, 64);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      v[i] = i >= left ? 0.f
             : BF16    ? __uint_as_float(unsigned(static_cast<const uint16_t*>(p)[at + i]) << 16)
                       : static_cast<const float*>(p)[at + i];
  }
}
CR_DEVICE void store16(uint16_t* p, int64_t at, const float* v, int left) {
  unsigned w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
  if (left >= 16) {
    __builtin_memcpy(p + at, w, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < left) p[at + i] = uint16_t(w[i / 2] >> (16 * (i & 1)));
  }
}

// One 128-feature block of a row in 8 lanes, 16 features each, as
// fp8_pack.hip does it.
CR_DEVICE void pack16(const float* v, uint8_t* q, uint8_t* scale) {
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, abs_bits(v[i]));
  top = max(top, dpp_u32<kDppQuadSwap1>(top));
  top = max(top, dpp_u32<kDppQuadSwap2>(top));
  top = max(top, dpp_u32<kDppHalfMirror>(top));
  const unsigned s = fp8_scale_of(top);
  const float inv = fp8_inverse_scale(s);
  u32x4 codes;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    codes[i] = s == kFp8ScaleNan
                   ? kFp8CodeNan
                   : fp8_codes4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
  *reinterpret_cast<u32x4*>(q) = codes;
  if ((threadIdx.x & 7) == 0) *scale = uint8_t(s);
}

// dgate = dy up act'(gate), dup = dy act(gate), as bfloat16 and, from the
// unrounded values, packed for the linear that leads back to X: the gate's
// blocks of a row, then the up projection's.  Bound by memory: three tensors
// are read once, two and their codes written (4096 x 13824: 680 MB in 115 us,
// 5.9 TB/s, some of it from the last-level cache).
//   silu' = s (1 + g (1 - s)),  s = 1 / (1 + exp(-g))
//   gelu' = Phi(g) + g phi(g)
template <bool BF16>
__global__ __launch_bounds__(256) void gated_back_kernel(const GatedBackArgs a) {
  const int nb = int((a.n + kFp8Block - 1) / kFp8Block), chunks = nb * 8;
  const int64_t total = a.m * chunks;
  for (int64_t c0 = (int64_t)blockIdx.x * 256; c0 < total; c0 += (int64_t)gridDim.x * 256) {
    const int64_t c = c0 + threadIdx.x;
    if (c >= total) break;  // (whole blocks)
    const int64_t row = c / chunks;
    const int f = int(c - row * chunks) * 16;
    const int left = int(a.n) - f;
    float dy[16], g[16], u[16];
    load16<BF16>(dy, a.dy, row * a.lddy + f, left);
    load16<true>(g, a.gate, row * a.ldk + f, left);
    load16<true>(u, a.up, row * a.ldk + f, left);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float act, slope;
      if (a.act == kActGelu) {
        const float phi = 0.5f * erfcf(-0.70710678f * g[i]);
        act = g[i] * phi;
        slope = __builtin_fmaf(g[i] * 0.39894228f, __builtin_amdgcn_exp2f(-0.72134752f * g[i] * g[i]), phi);
      } else {
        const float s = sigmoid_rough(g[i]);
        act = g[i] * s;
        slope = s * __builtin_fmaf(g[i], 1.f - s, 1.f);
      }
      g[i] = dy[i] * u[i] * slope;
      u[i] = dy[i] * act;
    }
    if (left > 0) {
      store16(a.dgate, row * a.ldd + f, g, left);
      store16(a.dup, row * a.ldd + f, u, left);
    }
    uint8_t* q = a.q + row * (2 * nb * kFp8Block) + f;
    uint8_t* s = a.q_scale + f / kFp8Block * a.lds + row;
    pack16(g, q, s);
    pack16(u, q + nb * kFp8Block, s + nb * a.lds);
  }
}

// One 64 x 64 tile of codes through LDS, byte by byte.  Offline: once for a
// weight (2 x 13824 x 5120 148 us, 2.6 times a copy).
__global__ __launch_bounds__(256) void fp8_transpose_kernel(const uint8_t* q, int64_t n, int64_t k, uint8_t* out,
                                                            int64_t ldq, int tiles, int64_t first) {
  __shared__ uint8_t tile[64][68];
  const int64_t at = first + blockIdx.x;
  const int64_t n0 = at % tiles * 64, k0 = at / tiles * 64;
  const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 16;
  for (int i = 0; i < 16; ++i)
    tile[r][c + i] = n0 + r < n && k0 + c + i < k ? q[(n0 + r) * k + k0 + c + i] : 0;
  __syncthreads();
  if (k0 + r < k) {
    uint8_t v[16];
    for (int i = 0; i < 16; ++i) v[i] = tile[c + i][r];
    __builtin_memcpy(out + (k0 + r) * ldq + n0 + c, v, 16);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void scale_transpose_kernel(const T* s, int nb, int kb, T* out, int lds) {
  for (int i = blockIdx.x * 256 + threadIdx.x; i < nb * kb; i += gridDim.x * 256)
    out[int64_t(i % kb) * lds + i / kb] = s[i];
}

}  // namespace

hipError_t launch_fp8_gated_wide(const Fp8GemmArgs& a, hipStream_t stream) {
  if (a.f32_scale)
    a.kept[0] ? launch_wide_t<true, kGatedKept>(a, stream) : launch_wide_t<true, kGated>(a, stream);
  else
    a.kept[0] ? launch_wide_t<false, kGatedKept>(a, stream) : launch_wide_t<false, kGated>(a, stream);
  return hipGetLastError();
}

hipError_t launch_gated_back(const GatedBackArgs& a, hipStream_t stream) {
  const int64_t groups = (a.m * ((a.n + kFp8Block - 1) / kFp8Block * 8) + 255) / 256;
  const dim3 grid(unsigned(groups < (1 << 20) ? groups : (1 << 20)));
  if (a.dy_bf16)
    hipLaunchKernelGGL(gated_back_kernel<true>, grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(gated_back_kernel<false>, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_fp8_transpose(const Fp8TransposeArgs& a, hipStream_t stream) {
  const int nb = int((a.n + kFp8Block - 1) / kFp8Block), kb = int((a.k + kFp8Block - 1) / kFp8Block);
  const int tiles = 2 * nb;
  in_launches(tiles * ((a.k + 63) / 64), 256, [&](int64_t first, unsigned count) {
    hipLaunchKernelGGL(fp8_transpose_kernel, dim3(count), dim3(256), 0, stream, a.q, a.n, a.k, a.q_out, a.ldq, tiles,
                       first);
  });
  const dim3 grid(unsigned((int64_t(nb) * kb + 255) / 256 < 65536 ? (int64_t(nb) * kb + 255) / 256 : 65536));
  const int lds = int(a.ldq / kFp8Block);
  if (a.f32_scale)
    hipLaunchKernelGGL(scale_transpose_kernel<float>, grid, dim3(256), 0, stream, static_cast<const float*>(a.scale),
                       nb, kb, static_cast<float*>(a.scale_out), lds);
  else
    hipLaunchKernelGGL(scale_transpose_kernel<uint8_t>, grid, dim3(256), 0, stream,
                       static_cast<const uint8_t*>(a.scale), nb, kb, static_cast<uint8_t*>(a.scale_out), lds);
  return hipGetLastError();
}

}  // namespace convrot
