// FP8 quantisation: activations in blocks of 1 x 128, weights in blocks of
// 128 x 128, each with a power-of-two scale (E8M0) and E4M3 codes.
//
// The scale is the least power of two that brings the block's largest
// magnitude to 448 (E4M3's largest value) or below.  E4M3 keeps the same
// relative precision over its whole normal range, so a power of two loses
// nothing against max / 448, makes the division exact (each code is the
// nearest E4M3 value of an exact quotient, ties to even) and lets the matrix
// cores apply the scale themselves.
#include "fp8.h"
#include "kernels.h"

namespace convrot {
namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// ROW_HALF_MIRROR: lane i of each group of 8 reads lane 7 - i.
constexpr int kDppHalfMirror = 0x141;

// Activations.  A thread owns 16 consecutive features (bf16: two 16-byte
// loads, float32: four), 8 neighbouring threads one block, whose maximum
// meets in three DPP steps; no LDS.  Bound by HBM: it reads X once and
// writes one byte a value.  4096 x 5120 bfloat16 takes 11 us (5.7 TB/s),
// 32760 x 5120 78 us (6.5 TB/s, partly from the last-level cache).
template <bool BF16>
__global__ __launch_bounds__(256) void fp8_pack_kernel(const void* __restrict__ x, int64_t ldx,
                                                       int64_t m, int k, int kc,
                                                       uint8_t* __restrict__ q,
                                                       uint8_t* __restrict__ scale, int64_t lds) {
  const int64_t total = m * kc;  // kc: 16-feature chunks per row, whole blocks
  for (int64_t c0 = (int64_t)blockIdx.x * 256; c0 < total; c0 += (int64_t)gridDim.x * 256) {
    const int64_t c = c0 + threadIdx.x;
    const int64_t row = c / kc;
    const int f = int(c - row * kc) * 16;
    const bool in = c < total && f < k;  // k % 16 == 0: a chunk is inside or outside
    float v[16];
    if (in) {
      if constexpr (BF16) {
        const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + row * ldx + f);
        const u32x4 a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = bf16_lo(a[i]);
          v[2 * i + 1] = bf16_hi(a[i]);
          v[8 + 2 * i] = bf16_lo(b[i]);
          v[9 + 2 * i] = bf16_hi(b[i]);
        }
      } else {
        const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(x) + row * ldx + f);
        const f32x4 a = p[0], b = p[1], c4 = p[2], d = p[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = a[i];
          v[4 + i] = b[i];
          v[8 + i] = c4[i];
          v[12 + i] = d[i];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
    }
    unsigned a = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = max(a, abs_bits(v[i]));
    a = max(a, dpp_u32<kDppQuadSwap1>(a));
    a = max(a, dpp_u32<kDppQuadSwap2>(a));
    a = max(a, dpp_u32<kDppHalfMirror>(a));
    const unsigned s = fp8_scale_of(a);
    const float inv = fp8_inverse_scale(s);
    u32x4 codes;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      codes[i] = s == kFp8ScaleNan ? kFp8CodeNan
                                   : fp8_codes4(v[4 * i] * inv, v[4 * i + 1] * inv,
                                                v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    if (in) {
      *reinterpret_cast<u32x4*>(q + row * k + f) = codes;
      if ((threadIdx.x & 7) == 0) scale[(f / kFp8Block) * lds + row] = uint8_t(s);
    }
  }
}

// Weights: one workgroup per 128 x 128 block, which it reads twice, the second
// time mostly from the caches.  Offline.  13824 x 5120 takes 54 us in bfloat16
// (3.9 TB/s, each byte counted once) and 100 us in float32 (3.5).
template <bool BF16>
__global__ __launch_bounds__(256) void fp8_wquant_kernel(const void* __restrict__ w, int64_t ldw,
                                                         int64_t n, int k, int kb, int64_t first,
                                                         uint8_t* __restrict__ q,
                                                         uint8_t* __restrict__ scale) {
  __shared__ unsigned top[4];
  const int64_t block = first + blockIdx.x;
  const int64_t bn = block / kb;
  const int bk = int(block - bn * kb);
  auto at = [&](int64_t r, int c) -> float {
    if constexpr (BF16)
      return __uint_as_float(unsigned(static_cast<const uint16_t*>(w)[r * ldw + c]) << 16);
    else
      return static_cast<const float*>(w)[r * ldw + c];
  };
  // thread t: columns 4 (t % 32) .. +3 of rows t / 32 + 8 i
  const int c0 = bk * kFp8Block + int(threadIdx.x & 31) * 4;
  const int64_t r0 = bn * kFp8Block + (threadIdx.x >> 5);
  unsigned a = 0;
  for (int i = 0; i < 16; ++i) {
    const int64_t r = r0 + 8 * i;
    if (r < n && c0 < k)  // k % 16 == 0: four columns are inside or outside together
      for (int j = 0; j < 4; ++j) a = max(a, abs_bits(at(r, c0 + j)));
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) a = max(a, unsigned(__shfl_xor(int(a), d)));
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = a;
  __syncthreads();
  a = max(max(top[0], top[1]), max(top[2], top[3]));
  const unsigned s = fp8_scale_of(a);
  const float inv = fp8_inverse_scale(s);
  for (int i = 0; i < 16; ++i) {
    const int64_t r = r0 + 8 * i;
    if (r < n && c0 < k) {
      const unsigned codes =
          s == kFp8ScaleNan ? kFp8CodeNan
                            : fp8_codes4(at(r, c0) * inv, at(r, c0 + 1) * inv, at(r, c0 + 2) * inv,
                                         at(r, c0 + 3) * inv);
      *reinterpret_cast<unsigned*>(q + r * k + c0) = codes;
    }
  }
  if (threadIdx.x == 0) scale[bn * kb + bk] = uint8_t(s);
}

}  // namespace

hipError_t launch_fp8_pack(const void* x, bool bf16, int64_t ldx, int64_t m, int64_t k,
                           uint8_t* q, uint8_t* scale, int64_t lds, hipStream_t stream) {
  const int kc = int((k + kFp8Block - 1) / kFp8Block) * (kFp8Block / 16);
  const int64_t groups = (m * kc + 255) / 256;
  const dim3 grid(unsigned(groups < (1 << 20) ? groups : (1 << 20)));
  if (bf16)
    hipLaunchKernelGGL(fp8_pack_kernel<true>, grid, dim3(256), 0, stream, x, ldx, m, int(k), kc, q,
                       scale, lds);
  else
    hipLaunchKernelGGL(fp8_pack_kernel<false>, grid, dim3(256), 0, stream, x, ldx, m, int(k), kc,
                       q, scale, lds);
  return hipGetLastError();
}

hipError_t launch_fp8_wquant(const void* w, bool bf16, int64_t ldw, int64_t n, int64_t k,
                             uint8_t* q, uint8_t* scale, hipStream_t stream) {
  const int kb = int((k + kFp8Block - 1) / kFp8Block);
  in_launches((n + kFp8Block - 1) / kFp8Block * kb, 256, [&](int64_t first, unsigned count) {
    if (bf16)
      hipLaunchKernelGGL(fp8_wquant_kernel<true>, dim3(count), dim3(256), 0, stream, w, ldw, n, int(k), kb, first, q,
                         scale);
    else
      hipLaunchKernelGGL(fp8_wquant_kernel<false>, dim3(count), dim3(256), 0, stream, w, ldw, n, int(k), kb, first, q,
                         scale);
  });
  return hipGetLastError();
}

}  // namespace convrot
