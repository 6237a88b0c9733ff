// Group norm of channels-last features, with an optional SiLU behind it:
//   y = act((x - mean) / sqrt(var + eps) * weight + bias)
// mean and var over the positions of an image and the channels of a group.
//
// Bound by memory.  A group of up to 65536 values (32768 where its channels are
// no multiple of 8) stays in one workgroup's registers between its statistics
// and its result: one launch, x read once.
// Larger ones take three: statistics of runs of positions, their union, and
// the result, which goes through x from its end, where the first pass left it
// in the last-level cache.
//
// Sums are float32 in a fixed order.  In the first form the variance is taken
// of the differences from the mean, whose own mean takes off the mean's
// rounding; in the second all values are taken relative to the group's first
// one, sums of 4 or 8 rows at a time are turned into a mean and squared
// differences from it and those united pairwise, in 64 bits among workgroups.
// Either way a large common part of a group costs no digits.
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace convrot {
namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// Values of a thread that holds a group in registers, V channels at a time
// (with fewer than 8 the addresses take up as many registers again).
constexpr int held_values(int V) { return V == 8 ? 64 : 32; }
constexpr int kThreads = 512;  // of a workgroup of the large form
static_assert(kMaxGroupNormC <= kThreads * 8, "a thread has 8 channels");

template <bool BF16, int V>
CR_DEVICE void load_values(float* v, const void* p, int64_t at) {
  if constexpr (BF16) {
    uint16_t w[V];
    __builtin_memcpy(w, static_cast<const uint16_t*>(p) + at, 2 * V);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __uint_as_float(unsigned(w[i]) << 16);
  } else {
    __builtin_memcpy(v, static_cast<const float*>(p) + at, 4 * V);
  }
}
template <int V>
CR_DEVICE void store_values(const float* v, void* p, bool bf16, int64_t at) {
  if (bf16) {
    uint16_t w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
    __builtin_memcpy(static_cast<uint16_t*>(p) + at, w, 2 * V);
  } else {
    __builtin_memcpy(static_cast<float*>(p) + at, v, 4 * V);
  }
}
CR_DEVICE float load_one(const void* p, bool bf16, int64_t at) {
  return bf16 ? __uint_as_float(unsigned(static_cast<const uint16_t*>(p)[at]) << 16)
              : static_cast<const float*>(p)[at];
}
CR_DEVICE float vector_value(const VectorArgs& v, int c, float absent) {
  return v.p ? load_one(v.p, v.bf16, c) : absent;
}

// Every step adds two sums that both lanes of a pair hold: all lanes get the same bits.
CR_DEVICE float wave_total(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}
CR_DEVICE double wave_total(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// One group in one workgroup, V neighbouring channels at a time (V divides the
// group's channels).
template <bool BF16, int V>
__global__ __launch_bounds__(1024) void group_norm_held_kernel(const GroupNormArgs a) {
  constexpr int N = held_values(V) / V;
  __shared__ float2 part[2][16];
  const int64_t at = a.first + blockIdx.x;
  const int64_t batch = at / a.groups;
  const int group = int(at - batch * a.groups);
  const int each = a.c / a.groups, columns = each / V, waves = blockDim.x / 64;
  const int vectors = int(a.positions) * columns;
  const int64_t xbase = batch * a.xs[0] + group * each, ybase = batch * a.ys[0] + group * each;

  float v[N][V];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = threadIdx.x + i * blockDim.x, row = e / columns;
    if (e < vectors) {
      load_values<BF16, V>(v[i], a.x, xbase + row * a.xs[1] + (e - row * columns) * V);
#pragma unroll
      for (int j = 0; j < V; ++j) sum += v[i][j];
    }
  }
  auto group_sum = [&](float s, float q, int slot) {
    s = wave_total(s);
    q = wave_total(q);
    if ((threadIdx.x & 63) == 0) part[slot][threadIdx.x >> 6] = make_float2(s, q);
    __syncthreads();
    s = q = 0.f;
    for (int w = 0; w < waves; ++w) {
      s += part[slot][w].x;
      q += part[slot][w].y;
    }
    return make_float2(s, q);
  };
  const float count = 1.f / (float(a.positions) * float(each));
  const float mean = group_sum(sum, 0.f, 0).x * count;
  float rest = 0.f, square = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (threadIdx.x + i * blockDim.x < unsigned(vectors)) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[i][j] -= mean;
        rest += v[i][j];
        square = __builtin_fmaf(v[i][j], v[i][j], square);
      }
    }
  const float2 sums = group_sum(rest, square, 1);
  const float off = sums.x * count;  // of the mean
  const float var = sums.y * count - off * off;
  const float r = 1.f / sqrtf((var < 0.f ? 0.f : var) + a.eps);  // (a NaN stays one)
  int thread = threadIdx.x;
  asm volatile("" : "+v"(thread));  // (the places are formed again: kept, they would take too many registers)
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = thread + i * blockDim.x, row = e / columns, c = (e - row * columns) * V;
    if (e < vectors) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float w = vector_value(a.weight, group * each + c + j, 1.f), b = vector_value(a.bias, group * each + c + j, 0.f);
        const float n = __builtin_fmaf((v[i][j] - off) * r, w, b);
        v[i][j] = a.silu ? silu(n) : n;
      }
      store_values<V>(v[i], a.y, a.y_bf16, ybase + row * a.ys[1] + c);
    }
  }
}

// Thread t of the large form has channels 8 (t % columns) .. +7 of rows
// t / columns + i (kThreads / columns).  WHOLE: the channels are a multiple of 8.
struct Place {
  int c, left, row, step;  // first channel, how many there are, first row, rows at a time
  bool in;
};
CR_DEVICE Place place(int c) {
  const int columns = (c + 7) / 8, step = kThreads / columns;
  const int row = int(threadIdx.x) / columns, at = (int(threadIdx.x) - row * columns) * 8;
  return {at, c - at < 8 ? c - at : 8, row, step, row < step};
}
template <bool BF16, bool WHOLE>
CR_DEVICE void load_row(float* v, const void* p, int64_t at, int left) {
  if (WHOLE || left == 8) {
    load_values<BF16, 8>(v, p, at);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? load_one(p, BF16, at + i) : 0.f;
  }
}

// Mean (relative to the group's first value) and squared differences from it
// of each group over one run of positions.
template <bool BF16, bool WHOLE>
__global__ __launch_bounds__(kThreads) void group_norm_stats_kernel(const GroupNormArgs a) {
  constexpr int U = BF16 ? 8 : 4;  // rows at once
  __shared__ float means[kThreads * 8], squares[kThreads * 8];
  const int64_t run = a.first + blockIdx.x;
  const int64_t batch = run / a.runs;
  const int64_t p0 = a.positions * (run - batch * a.runs) / a.runs;
  const int64_t p1 = a.positions * (run - batch * a.runs + 1) / a.runs;
  const int each = a.c / a.groups;
  const Place me = place(a.c);
  float mean[8] = {}, sq[8] = {};
  if (me.in) {
    const int64_t base = batch * a.xs[0];
    float pivot[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) pivot[i] = load_one(a.x, BF16, base + (me.c + (i < me.left ? i : 0)) / each * each);
    float n = 0.f;
    for (int64_t r = p0 + me.row; r < p1; r += U * me.step) {
      float v[U][8];
      int rows = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = r + u * me.step;
        if (at < p1) ++rows;
        load_row<BF16, WHOLE>(v[u], a.x, base + (at < p1 ? at : r) * a.xs[1] + me.c, me.left);
      }
      const float nb = float(rows), inv = 1.f / nb;
      const float share = nb / (n + nb), both = n * share;
      n += nb;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float s = 0.f, q = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          v[u][i] -= pivot[i];
          s += u < rows ? v[u][i] : 0.f;
        }
        s *= inv;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float d = u < rows ? v[u][i] - s : 0.f;
          q = __builtin_fmaf(d, d, q);
        }
        const float d = s - mean[i];
        mean[i] = __builtin_fmaf(d, share, mean[i]);
        sq[i] += __builtin_fmaf(d * d, both, q);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    means[threadIdx.x * 8 + i] = mean[i];
    squares[threadIdx.x * 8 + i] = sq[i];
  }
  __syncthreads();
  // A group's channels of all rows, a wave to a group.
  const int columns = (a.c + 7) / 8, lane = threadIdx.x & 63;
  for (int g = threadIdx.x >> 6; g < a.groups; g += kThreads / 64) {
    const int entries = each * me.step;
    float s = 0.f;
    for (int e = lane; e < entries; e += 64) {
      const int row = e / each, c = g * each + e - row * each;
      const int64_t rows = p1 - p0 > row ? (p1 - p0 - row + me.step - 1) / me.step : 0;
      s += float(rows) * means[(row * columns + c / 8) * 8 + c % 8];
    }
    const float m = wave_total(s) / (float(p1 - p0) * float(each));
    s = 0.f;
    for (int e = lane; e < entries; e += 64) {
      const int row = e / each, c = g * each + e - row * each, at = (row * columns + c / 8) * 8 + c % 8;
      const int64_t rows = p1 - p0 > row ? (p1 - p0 - row + me.step - 1) / me.step : 0;
      const float d = means[at] - m;
      s += squares[at] + float(rows) * d * d;
    }
    s = wave_total(s);
    if (lane == 0) reinterpret_cast<float2*>(a.part)[run * a.groups + g] = make_float2(m, s);
  }
}

// The runs of a group, united; a wave to a group of an image.
template <bool BF16>
__global__ __launch_bounds__(64) void group_norm_unite_kernel(const GroupNormArgs a) {
  const int64_t at = a.first + blockIdx.x, batch = at / a.groups;
  const int group = int(at - batch * a.groups), each = a.c / a.groups;
  const float2* part = reinterpret_cast<const float2*>(a.part) + batch * a.runs * a.groups + group;
  auto rows = [&](int64_t i) { return double(a.positions * (i + 1) / a.runs - a.positions * i / a.runs); };
  double s = 0;
  for (int i = threadIdx.x; i < a.runs; i += 64) s += rows(i) * double(part[int64_t(i) * a.groups].x);
  const double mean = wave_total(s) / double(a.positions);
  s = 0;
  for (int i = threadIdx.x; i < a.runs; i += 64) {
    const float2 p = part[int64_t(i) * a.groups];
    const double d = double(p.x) - mean;
    s += double(p.y) + rows(i) * each * d * d;
  }
  const double var = wave_total(s) / (double(a.positions) * each);
  if (threadIdx.x == 0) {
    const float r = float(1.0 / sqrt(var + double(a.eps)));
    reinterpret_cast<f32x4*>(a.stats)[at] = f32x4{load_one(a.x, BF16, batch * a.xs[0] + group * each), float(mean), r, 0.f};
  }
}

template <bool BF16, bool WHOLE>
__global__ __launch_bounds__(kThreads) void group_norm_apply_kernel(const GroupNormArgs a) {
  constexpr int U = 4;
  // (from the end of x)
  const int64_t run = a.batch * a.runs - 1 - (a.first + blockIdx.x);
  const int64_t batch = run / a.runs;
  const int64_t p0 = a.positions * (run - batch * a.runs) / a.runs;
  const int64_t p1 = a.positions * (run - batch * a.runs + 1) / a.runs;
  const int each = a.c / a.groups;
  const Place me = place(a.c);
  if (!me.in) return;
  float pivot[8], mean[8], scale[8], bias[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = me.c + (i < me.left ? i : 0);
    const f32x4 s = reinterpret_cast<const f32x4*>(a.stats)[batch * a.groups + c / each];
    pivot[i] = s[0];
    mean[i] = s[1];
    scale[i] = s[2] * vector_value(a.weight, c, 1.f);
    bias[i] = vector_value(a.bias, c, 0.f);
  }
  for (int64_t r = p0 + me.row; r < p1; r += U * me.step) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = r + u * me.step < p1 ? r + u * me.step : r;
      load_row<BF16, WHOLE>(v[u], a.x, batch * a.xs[0] + at * a.xs[1] + me.c, me.left);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = r + u * me.step;
      if (at >= p1) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = __builtin_fmaf(v[u][i] - pivot[i] - mean[i], scale[i], bias[i]);
        v[u][i] = a.silu ? silu(n) : n;
      }
      const int64_t to = batch * a.ys[0] + at * a.ys[1] + me.c;
      if (WHOLE || me.left == 8) {
        store_values<8>(v[u], a.y, a.y_bf16, to);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < me.left) store_values<1>(v[u] + i, a.y, a.y_bf16, to + i);
      }
    }
  }
}

template <bool BF16, int V>
void launch_held(GroupNormArgs a, hipStream_t stream) {
  const int64_t vectors = a.positions * (a.c / a.groups / V);
  const int64_t waves = (vectors + 63) / 64;
  const int threads = 64 * int(waves < 16 ? waves : 16);
  in_launches(a.batch * a.groups, threads, [&](int64_t first, unsigned count) {
    a.first = first;
    hipLaunchKernelGGL((group_norm_held_kernel<BF16, V>), dim3(count), dim3(threads), 0, stream, a);
  });
}

template <bool BF16>
void launch_large(GroupNormArgs a, hipStream_t stream) {
  auto go = [&](auto whole) {
    constexpr bool kWhole = decltype(whole)::value;
    in_launches(a.batch * a.runs, kThreads, [&](int64_t first, unsigned count) {
      a.first = first;
      hipLaunchKernelGGL((group_norm_stats_kernel<BF16, kWhole>), dim3(count), dim3(kThreads), 0, stream, a);
    });
    in_launches(a.batch * a.groups, 64, [&](int64_t first, unsigned count) {
      a.first = first;
      hipLaunchKernelGGL(group_norm_unite_kernel<BF16>, dim3(count), dim3(64), 0, stream, a);
    });
    in_launches(a.batch * a.runs, kThreads, [&](int64_t first, unsigned count) {
      a.first = first;
      hipLaunchKernelGGL((group_norm_apply_kernel<BF16, kWhole>), dim3(count), dim3(kThreads), 0, stream, a);
    });
  };
  if (a.c % 8 == 0)
    go(std::true_type{});
  else
    go(std::false_type{});
}

}  // namespace

int64_t plan_group_norm(int64_t batch, int64_t positions, int c, int groups) {
  const int each = c / groups;
  if (positions * each <= 1024 * held_values(each % 8 == 0 ? 8 : 1)) return 0;
  // Two workgroups for each CU, of whole steps of 8 rows.
  const int64_t rows = 8 * (kThreads / ((c + 7) / 8));
  int64_t runs = (2 * int64_t(device_cu_count()) + batch - 1) / batch;
  if (runs > (positions + rows - 1) / rows) runs = (positions + rows - 1) / rows;
  return runs;
}

hipError_t launch_group_norm(const GroupNormArgs& a, hipStream_t stream) {
  const int each = a.c / a.groups;
  if (a.runs > 0) {
    a.x_bf16 ? launch_large<true>(a, stream) : launch_large<false>(a, stream);
  } else if (a.x_bf16) {
    each % 8 == 0 ? launch_held<true, 8>(a, stream)
    : each % 2 == 0 ? launch_held<true, 2>(a, stream) : launch_held<true, 1>(a, stream);
  } else {
    each % 8 == 0 ? launch_held<false, 8>(a, stream)
    : each % 2 == 0 ? launch_held<false, 2>(a, stream) : launch_held<false, 1>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace convrot
