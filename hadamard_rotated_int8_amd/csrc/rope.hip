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

__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeArgs a, int tpg) {
  extern __shared__ float2 cs[];  // [tpg][pairs]
  const int pairs = a.rot / 2;
  const int64_t total = a.batch * a.tokens;
  const int64_t t0 = (int64_t)blockIdx.x * tpg;
  for (int i = threadIdx.x; i < tpg * pairs; i += kThreads) {
    const int64_t t = t0 + i / pairs;
    if (t >= total) break;
    const int j = i % pairs;
    const int64_t b = t / a.tokens, tok = t - b * a.tokens;
    const int64_t at = b * a.pos_batch + tok * a.pos_token + (a.axis ? a.axis[j] : 0);
    const double pos = a.pos_type == kPosI32   ? double(static_cast<const int32_t*>(a.positions)[at])
                       : a.pos_type == kPosI64 ? double(static_cast<const int64_t*>(a.positions)[at])
                                               : double(static_cast<const float*>(a.positions)[at]);
    double turns = pos * (a.inv_freq[j] * 0.15915494309189533577);
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * float(turns), &s, &c);
    cs[i] = make_float2(c * a.factor, (a.inverse ? -s : s) * a.factor);
  }
  __syncthreads();
  for (int q = 0; q < a.count; ++q) {
    const RopeTensor& x = a.t[q];
    // one work item per pair, and per feature outside the rotated part
    const int rest = a.d - a.rot;
    const int per_head = pairs + (x.copy_rest ? rest : 0);
    const int n = tpg * x.heads * per_head;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int e = i % per_head, h = i / per_head % x.heads, tl = i / per_head / x.heads;
      const int64_t t = t0 + tl;
      if (t >= total) break;
      const int64_t b = t / a.tokens, tok = t - b * a.tokens;
      const int64_t xi = b * x.xs[0] + tok * x.xs[1] + h * x.xs[2];
      const int64_t yi = b * x.ys[0] + tok * x.ys[1] + h * x.ys[2];
      if (e < pairs) {
        const int f0 = a.start + (a.half ? e : 2 * e), f1 = f0 + (a.half ? pairs : 1);
        const float u = load1(x.x, a.x_bf16, xi + f0), v = load1(x.x, a.x_bf16, xi + f1);
        const float2 r = cs[tl * pairs + e];
        store1(x.y, a.y_bf16, yi + f0, __builtin_fmaf(u, r.x, -(v * r.y)));
        store1(x.y, a.y_bf16, yi + f1, __builtin_fmaf(v, r.x, u * r.y));
      } else {
        const int f = e - pairs + (e - pairs < a.start ? 0 : a.rot);
        store1(x.y, a.y_bf16, yi + f, load1(x.x, a.x_bf16, xi + f));
      }
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
  const int pairs = a.rot / 2;
  int tpg = 1;
  const int64_t total = a.batch * a.tokens;
  const int64_t grid = (total + tpg - 1) / tpg;
  hipLaunchKernelGGL(rope_kernel, dim3(unsigned(grid)), dim3(kThreads),
                     size_t(tpg) * pairs * sizeof(float) * 2, stream, a, tpg);
  return hipGetLastError();
}

}  // namespace convrot
