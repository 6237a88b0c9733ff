// Rotary positions: every pair of features (a, b) of a head turns by the
// angle positions[token] * inv_freq[pair],
//   (a, b) -> (a c - b s, b c + a s),  c = factor cos, s = factor sin.
//
// The angle is formed in turns, in float64 (the product of a far position
// and a frequency needs more than 24 bits), its whole turns are taken off,
// and what is left goes to float32 sine and cosine: once per token and pair
// (into LDS), for all heads of all tensors.  Bound by HBM: every feature is
// read once and written once.
#include "common.h"
#include "kernels.h"

namespace convrot {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // per workgroup

// n / d for n d < 2^32 by one multiplication: m = ceil(2^32 / d) overshoots
// 2^32 / d by less than 1, so n m / 2^32 overshoots n / d by less than
// n / 2^32 < 1 / d.  (Here n < 2^18 items of a workgroup and d <= 4096.)
struct Divisor {
  unsigned m, d;
};
Divisor divisor(int d) { return {unsigned(((uint64_t(1) << 32) + d - 1) / d), unsigned(d)}; }
CR_DEVICE int quotient(int n, Divisor v) {
  return v.d == 1 ? n : int(__umulhi(unsigned(n), v.m));
}

struct Shape {
  int64_t first;  // workgroup of the launch's first one
  int tokens;     // per workgroup
  int pairs;      // rot / 2
  int units;      // work items per head: those that turn, then those that copy
  int turning;    // ... that turn
  int copy_lo;    // ... that copy features below the slice
  Divisor by_units, by_turning, by_pairs, by_heads[kMaxRopeTensors];
};

CR_DEVICE float load1(const void* p, bool bf16, int64_t at) {
  return bf16 ? __uint_as_float(unsigned(static_cast<const uint16_t*>(p)[at]) << 16)
              : static_cast<const float*>(p)[at];
}
CR_DEVICE void store1(void* p, bool bf16, int64_t at, float v) {
  if (bf16)
    static_cast<uint16_t*>(p)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
  else
    static_cast<float*>(p)[at] = v;
}

// Eight consecutive features; they need only the type's own alignment.
template <bool BF16>
CR_DEVICE void load8(float* v, const void* p, int64_t at) {
  if constexpr (BF16) {
    u32x4 w;
    __builtin_memcpy(&w, static_cast<const uint16_t*>(p) + at, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
    f32x4 w[2];
    __builtin_memcpy(w, static_cast<const float*>(p) + at, 32);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i / 4][i % 4];
  }
}
template <bool BF16>
CR_DEVICE void store8(void* p, int64_t at, const float* v) {
  if constexpr (BF16) {
    uint16_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
    __builtin_memcpy(static_cast<uint16_t*>(p) + at, w, 16);
  } else {
    __builtin_memcpy(static_cast<float*>(p) + at, v, 32);
  }
}

// A workgroup turns `tokens` tokens of every tensor.  VEC: a work item is 8
// pairs (half: 8 features of each half) or 4 (interleaved: 8 features in a
// row), or 8 features that are copied; the launcher checks that the slice and
// what lies beside it divide into such items.  Otherwise a work item is one
// pair, or one copied feature.
template <bool HALF, bool XB, bool YB, bool VEC>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeArgs a, const Shape s) {
  extern __shared__ __attribute__((aligned(16))) float2 cs[];  // [tokens][pairs]
  __shared__ int64_t place[kMaxTokens][2];                     // batch entry, token
  const int64_t total = a.batch * a.tokens;
  const int64_t t0 = (s.first + blockIdx.x) * s.tokens;
  const int nt = total - t0 < s.tokens ? int(total - t0) : s.tokens;
  for (int i = threadIdx.x; i < nt * s.pairs; i += kThreads) {
    const int tl = quotient(i, s.by_pairs), j = i - tl * s.pairs;
    const int64_t t = t0 + tl, b = t / a.tokens, tok = t - b * a.tokens;
    if (j == 0) {
      place[tl][0] = b;
      place[tl][1] = tok;
    }
    const int axis = a.axis ? a.axis[j] : 0;
    const bool known = unsigned(axis) < unsigned(a.axes);
    const int64_t at = b * a.pos_batch + tok * a.pos_token + (known ? axis : 0);
    const double pos = a.pos_type == kPosI32   ? double(static_cast<const int32_t*>(a.positions)[at])
                       : a.pos_type == kPosI64 ? double(static_cast<const int64_t*>(a.positions)[at])
                                               : double(static_cast<const float*>(a.positions)[at]);
    double turns = pos * (a.inv_freq[j] * 0.15915494309189533577);  // 1 / (2 pi)
    turns = known ? turns - rint(turns) : __builtin_nan("");
    float sn, c;
    sincospif(2.f * float(turns), &sn, &c);
    cs[i] = make_float2(c * a.factor, (a.inverse ? -sn : sn) * a.factor);
  }
  __syncthreads();
  for (int q = 0; q < a.count; ++q) {
    const RopeTensor& x = a.t[q];
    const int units = x.copy_rest ? s.units : s.turning;
    const Divisor by_units = x.copy_rest ? s.by_units : s.by_turning;
    const int n = nt * x.heads * units;
#pragma unroll 2
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int r = quotient(i, by_units), u = i - r * units;
      const int tl = quotient(r, s.by_heads[q]), h = r - tl * x.heads;
      const int64_t b = place[tl][0], tok = place[tl][1];
      const int64_t xi = b * x.xs[0] + tok * x.xs[1] + h * x.xs[2];
      const int64_t yi = b * x.ys[0] + tok * x.ys[1] + h * x.ys[2];
      const float2* t = cs + tl * s.pairs;
      if (u < s.turning) {
        if constexpr (!VEC) {
          const int f0 = a.start + (HALF ? u : 2 * u), f1 = f0 + (HALF ? s.pairs : 1);
          const float v = load1(x.x, XB, xi + f0), w = load1(x.x, XB, xi + f1);
          const float2 c = t[u];
          store1(x.y, YB, yi + f0, __builtin_fmaf(v, c.x, -(w * c.y)));
          store1(x.y, YB, yi + f1, __builtin_fmaf(w, c.x, v * c.y));
        } else if constexpr (HALF) {
          const int f0 = a.start + 8 * u, f1 = f0 + s.pairs;
          float v[8], w[8], vo[8], wo[8];
          load8<XB>(v, x.x, xi + f0);
          load8<XB>(w, x.x, xi + f1);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 c = t[8 * u + e];
            vo[e] = __builtin_fmaf(v[e], c.x, -(w[e] * c.y));
            wo[e] = __builtin_fmaf(w[e], c.x, v[e] * c.y);
          }
          store8<YB>(x.y, yi + f0, vo);
          store8<YB>(x.y, yi + f1, wo);
        } else {
          const int f = a.start + 8 * u;
          float v[8], o[8];
          load8<XB>(v, x.x, xi + f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c = t[4 * u + e];
            o[2 * e] = __builtin_fmaf(v[2 * e], c.x, -(v[2 * e + 1] * c.y));
            o[2 * e + 1] = __builtin_fmaf(v[2 * e + 1], c.x, v[2 * e] * c.y);
          }
          store8<YB>(x.y, yi + f, o);
        }
      } else {
        const int e = u - s.turning;
        if constexpr (VEC) {
          const int f = 8 * e + (e < s.copy_lo ? 0 : a.rot);
          float v[8];
          load8<XB>(v, x.x, xi + f);
          store8<YB>(x.y, yi + f, v);
        } else {
          const int f = e + (e < s.copy_lo ? 0 : a.rot);
          store1(x.y, YB, yi + f, load1(x.x, XB, xi + f));
        }
      }
    }
  }
}

template <bool HALF, bool XB, bool YB>
void launch_t(const RopeArgs& a, const Shape& s, bool vec, dim3 grid, size_t lds, hipStream_t stream) {
  if (vec)
    hipLaunchKernelGGL((rope_kernel<HALF, XB, YB, true>), grid, dim3(kThreads), lds, stream, a, s);
  else
    hipLaunchKernelGGL((rope_kernel<HALF, XB, YB, false>), grid, dim3(kThreads), lds, stream, a, s);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
  Shape s{};
  s.pairs = a.rot / 2;
  const int rest = a.d - a.rot, unit = a.half ? 16 : 8;  // features of a turning item
  // Items of 8 features where slice and head allow it: 372 against 396 us for
  // the last of the cases below, 15 against 36 for 2 x 2049 tokens of 40 heads
  // of 96.
  const bool vec = a.rot % unit == 0 && a.start % 8 == 0 && rest % 8 == 0;
  s.turning = vec ? a.rot / unit : s.pairs;
  s.units = s.turning + (vec ? rest / 8 : rest);
  s.copy_lo = vec ? a.start / 8 : a.start;
  s.by_units = divisor(s.units);
  s.by_turning = divisor(s.turning);
  s.by_pairs = divisor(s.pairs);
  int least = 1 << 30, most = 1;  // items of one token, in the smallest and the largest tensor
  for (int q = 0; q < a.count; ++q) {
    const int items = a.t[q].heads * s.units;
    least = items < least ? items : least;
    most = items > most ? items : most;
    s.by_heads[q] = divisor(a.t[q].heads);
  }
  // Enough tokens that the smallest tensor has an item for every thread, as
  // long as there are workgroups for every CU several times over, the items
  // stay few and the angles take at most 16 KB.  Measured with 1, 2, 4, 8 and
  // 16 tokens per workgroup (us, bfloat16): 65536 tokens of one head of 64
  // (which take 16) 45, 25, 16, 11, 10; 32768 of 8 heads of 64 (4) 29.7, 20.1,
  // 15.1, 13.3, 13.4; 32760 of 2 x 40 heads of 128, float32 to bfloat16 (1)
  // 372, 378, 385, 392, 405.
  const int64_t total = a.batch * a.tokens;
  s.tokens = 1;
  while (s.tokens < kMaxTokens && s.tokens * least < kThreads && total / (2 * s.tokens) >= 2048 &&
         int64_t(2) * s.tokens * most < 65536 && 2 * s.tokens * s.pairs <= 2048)
    s.tokens *= 2;
  const size_t lds = size_t(s.tokens) * s.pairs * sizeof(float) * 2;
  const int which = (a.half ? 4 : 0) | (a.x_bf16 ? 2 : 0) | (a.y_bf16 ? 1 : 0);
  in_launches((total + s.tokens - 1) / s.tokens, kThreads, [&](int64_t first, unsigned count) {
    const dim3 grid(count);
    s.first = first;
    switch (which) {
      case 0: launch_t<false, false, false>(a, s, vec, grid, lds, stream); break;
      case 1: launch_t<false, false, true>(a, s, vec, grid, lds, stream); break;
      case 2: launch_t<false, true, false>(a, s, vec, grid, lds, stream); break;
      case 3: launch_t<false, true, true>(a, s, vec, grid, lds, stream); break;
      case 4: launch_t<true, false, false>(a, s, vec, grid, lds, stream); break;
      case 5: launch_t<true, false, true>(a, s, vec, grid, lds, stream); break;
      case 6: launch_t<true, true, false>(a, s, vec, grid, lds, stream); break;
      default: launch_t<true, true, true>(a, s, vec, grid, lds, stream); break;
    }
  });
  return hipGetLastError();
}

}  // namespace convrot
