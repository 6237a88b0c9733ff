// Group norm of channels-last features, with an optional SiLU behind it:
//   y = act((x - mean) / sqrt(var + eps) * weight + bias)
// mean and var over the positions of an image and the channels of a group.
//
// Bound by memory.  A group of up to 65536 values (32768 where its channels are
// no multiple of 8) stays in one workgroup's registers between its statistics
// and its result: one launch, x read once.  2 x 64 positions of 1280 channels in
// 32 groups: 4.7 us, a launch and two trips to memory.
// Larger ones take three launches: statistics of runs of positions, their
// union, and the result, which goes through x from its end, where the first
// pass left it in the last-level cache.  1048576 positions of 128 channels take
// 158 us: 65 to read them once (4.1 TB/s; a library's reductions read at 3.5 to
// 4.0), 87 to read them and write y (6.2 TB/s, some of it from the last-level
// cache), 4.6 between.  Workgroups that unite the runs for themselves in the
// third launch spend more than the second one takes (190 us in all, 175 then).
//
// Sums are float32 in a fixed order.  In the first form the variance is taken
// of the differences from the mean, whose own mean takes off the mean's
// rounding.  In the second a thread takes each channel's values relative to the
// first one that it reads, turns 4 rows at a time into a mean and squared
// differences from it and unites those pairwise; the threads' means and the
// workgroups' sums are united in 64 bits (16384 x 512: 0.6 us of 26), and the
// result takes the mean off in two parts of 32.
// Either way neither a large common part of a group nor single values far from
// the others cost digits (a value relative to one that is far away is rounded
// to that one's spacing; only the thread that read it first is).
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
template <int V>
CR_DEVICE void silu_all(float* v, bool bf16) {
  if (bf16) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = silu_rough(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = silu(v[i]);
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
  extern __shared__ float affine[];  // the group's weights, its biases
  const int64_t at = a.first + blockIdx.x;
  const int64_t batch = at / a.groups;
  const int group = int(at - batch * a.groups);
  const int each = a.c / a.groups, columns = each / V, waves = blockDim.x / 64;
  const int vectors = int(a.positions) * columns;
  const int64_t xbase = batch * a.xs[0] + group * each, ybase = batch * a.ys[0] + group * each;

  float v[N][V];
  float sum = 0.f;
  // (on its way beside x)
  for (int c = threadIdx.x; c < each; c += blockDim.x) {
    affine[c] = vector_value(a.weight, group * each + c, 1.f);
    affine[each + c] = vector_value(a.bias, group * each + c, 0.f);
  }
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
      for (int j = 0; j < V; ++j)
        v[i][j] = __builtin_fmaf((v[i][j] - off) * r, affine[c + j], affine[each + c + j]);
      if (a.silu) silu_all<V>(v[i], a.y_bf16);
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
// Rows at a time, and those that a thread has under way: a block of kRows steps.
constexpr int kRows = 4;
constexpr __host__ __device__ int row_step(int c) { return kThreads / ((c + 7) / 8); }
// Run r of an image has the blocks r, r + runs, ...: how many rows that is.
struct RunRows {
  int64_t block, blocks, base, extra, last, missing;
  CR_DEVICE explicit RunRows(const GroupNormArgs& a) {
    block = kRows * row_step(a.c);
    blocks = (a.positions + block - 1) / block;
    base = blocks / a.runs;
    extra = blocks - base * a.runs;  // runs with a block more
    last = extra > 0 ? extra - 1 : a.runs - 1;  // whose last block is the image's last one
    missing = blocks * block - a.positions;
  }
  CR_DEVICE int64_t of(int64_t run) const { return (base + (run < extra)) * block - (run == last ? missing : 0); }
};
CR_DEVICE Place place(int c) {
  const int columns = (c + 7) / 8, step = row_step(c);
  const int row = int(threadIdx.x) / columns, at = (int(threadIdx.x) - row * columns) * 8;
  return {at, c - at < 8 ? c - at : 8, row, step, row < step};
}
template <bool BF16>
struct Raw {  // eight values as they lie in memory
  uint32_t w[BF16 ? 4 : 8];
};
template <bool BF16, bool WHOLE>
CR_DEVICE Raw<BF16> load_row(const void* p, int64_t at, int left) {
  constexpr int kSize = BF16 ? 2 : 4;
  Raw<BF16> r = {};
  const uint8_t* from = static_cast<const uint8_t*>(p) + at * kSize;
  if (WHOLE || left == 8) {
    __builtin_memcpy(r.w, from, 8 * kSize);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= left) continue;
      if constexpr (BF16)
        r.w[i / 2] |= unsigned(static_cast<const uint16_t*>(p)[at + i]) << (16 * (i & 1));
      else
        r.w[i] = static_cast<const uint32_t*>(p)[at + i];
    }
  }
  return r;
}
template <bool BF16>
CR_DEVICE float value_of(const Raw<BF16>& r, int i) {
  if constexpr (BF16)
    return i & 1 ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]);
  else
    return __uint_as_float(r.w[i]);
}

// Mean and squared differences from it of each group over one run.  (Neighbouring blocks go to different runs, and
// all workgroups are on one stretch of x: 262144 positions of 256 channels 86
// us, 90 with each run in one piece.)
template <bool BF16, bool WHOLE>
__global__ __launch_bounds__(kThreads, 4) void group_norm_stats_kernel(const GroupNormArgs a) {
  __shared__ double means[kThreads * 8], met[2][kThreads / 64];
  __shared__ float squares[kThreads * 8];
  const int64_t at = a.first + blockIdx.x;
  const int64_t batch = at / a.runs, run = at - batch * a.runs;
  const int each = a.c / a.groups;
  const Place me = place(a.c);
  const int64_t block = kRows * me.step, stride = block * a.runs;
  float pivot[8] = {}, mean[8] = {}, sq[8] = {};
  if (me.in) {
    const int64_t base = batch * a.xs[0];
    // The next rows are on their way while these are summed.
    Raw<BF16> held[kRows];
    auto load = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t row = r + u * me.step;
        held[u] = load_row<BF16, WHOLE>(a.x, base + (row < a.positions ? row : a.positions - 1) * a.xs[1] + me.c, me.left);
      }
    };
    float n = 0.f;
    auto add = [&](auto whole, int rows, int64_t next) __attribute__((always_inline)) {
      constexpr bool kAll = decltype(whole)::value;  // (rows is kRows)
      float v[kRows][8];
#pragma unroll
      for (int u = 0; u < kRows; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = value_of<BF16>(held[u], i);
      load(next);
      const float nb = float(rows), inv = 1.f / nb;
      const float share = nb / (n + nb), both = n * share;
      n += nb;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float s = 0.f, q = 0.f;
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          v[u][i] -= pivot[i];
          s += kAll || u < rows ? v[u][i] : 0.f;
        }
        s *= inv;
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const float d = kAll || u < rows ? v[u][i] - s : 0.f;
          q = __builtin_fmaf(d, d, q);
        }
        const float d = s - mean[i];
        mean[i] = __builtin_fmaf(d, share, mean[i]);
        sq[i] += __builtin_fmaf(d * d, both, q);
      }
    };
    int64_t r = run * block + me.row;
    load(r);
#pragma unroll
    for (int i = 0; i < 8; ++i) pivot[i] = value_of<BF16>(held[0], i);
    for (; r + (kRows - 1) * me.step < a.positions; r += stride) add(std::true_type{}, kRows, r + stride);
    if (r < a.positions) add(std::false_type{}, int((a.positions - r + me.step - 1) / me.step), r);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    means[threadIdx.x * 8 + i] = double(pivot[i]) + double(mean[i]);
    squares[threadIdx.x * 8 + i] = sq[i];
  }
  __syncthreads();
  // A group's channels of all rows: a wave to a group, or with fewer groups than
  // waves as many as there are for each (486708 positions of 24 channels in one
  // group, float32: 33 us; with one wave 41).
  constexpr int kWaves = kThreads / 64;
  const int columns = (a.c + 7) / 8, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t rows = RunRows(a).of(run);
  const double some = double(rows / me.step);  // ... of a step's row, and one more of the first ones
  const int more = int(rows % me.step);
  const double share = 1 / (double(rows) * each);
  auto reduce = [&](auto one) __attribute__((always_inline)) {
    constexpr bool kOne = decltype(one)::value;
    const int team = kOne ? 1 : kWaves / a.groups, teams = kWaves / team;  // waves of a group, groups at once
    for (int g0 = 0; g0 < a.groups; g0 += teams) {  // (once, where a team has more than one wave)
      const int g = g0 + wave / team, member = wave % team;
      const int entries = wave / team < teams && g < a.groups ? each * me.step : 0;
      auto total = [&](auto s, int slot) __attribute__((always_inline)) {
        s = wave_total(s);
        if constexpr (kOne) return s;
        if (lane == 0) met[slot][wave] = s;
        __syncthreads();
        s = 0;
        for (int w = wave - member; w < wave - member + team && w < kWaves; ++w) s += decltype(s)(met[slot][w]);
        return s;
      };
      double s = 0;
      for (int e = lane + 64 * member; e < entries; e += 64 * team) {
        const int row = e / each, c = g * each + e - row * each;
        s += (row < more ? some + 1 : some) * means[(row * columns + c / 8) * 8 + c % 8];
      }
      const double m = total(s, 0) * share;
      float q = 0.f;
      for (int e = lane + 64 * member; e < entries; e += 64 * team) {
        const int row = e / each, c = g * each + e - row * each, i = (row * columns + c / 8) * 8 + c % 8;
        const float d = float(means[i] - m);
        q += squares[i] + float(row < more ? some + 1 : some) * d * d;
      }
      q = total(q, 1);
      if (lane == 0 && member == 0 && entries > 0)
        reinterpret_cast<double2*>(a.part)[(batch * a.groups + g) * a.runs + run] = make_double2(m, q);
    }
  };
  if (a.groups > kWaves / 2)
    reduce(std::true_type{});
  else
    reduce(std::false_type{});
}

// The runs of a group, united; a workgroup to a group of an image.
constexpr int kUniters = 256;
__global__ __launch_bounds__(kUniters) void group_norm_unite_kernel(const GroupNormArgs a) {
  __shared__ double sums[2][kUniters / 64];
  const int64_t at = a.first + blockIdx.x;
  const int each = a.c / a.groups;
  const double2* part = reinterpret_cast<const double2*>(a.part) + at * a.runs;
  const RunRows rows(a);
  auto total = [&](double s, int slot) {
    s = wave_total(s);
    if ((threadIdx.x & 63) == 0) sums[slot][threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0;
#pragma unroll
    for (int w = 0; w < kUniters / 64; ++w) s += sums[slot][w];
    return s;
  };
  double s = 0;
  for (int i = threadIdx.x; i < a.runs; i += kUniters) s += double(rows.of(i)) * part[i].x;
  const double mean = total(s, 0) / double(a.positions);
  s = 0;
  for (int i = threadIdx.x; i < a.runs; i += kUniters) {
    const double2 p = part[i];
    const double d = p.x - mean;
    s += p.y + double(rows.of(i)) * each * d * d;
  }
  const double var = total(s, 1) / (double(a.positions) * each);
  if (threadIdx.x == 0) {
    a.stats[4 * at] = float(mean);
    a.stats[4 * at + 1] = float(mean - double(float(mean)));
    a.stats[4 * at + 2] = float(1.0 / sqrt(var + double(a.eps)));
  }
}

template <bool BF16, bool WHOLE>
__global__ __launch_bounds__(kThreads) void group_norm_apply_kernel(const GroupNormArgs a) {
  // (from the end of x)
  const int64_t at = a.batch * a.runs - 1 - (a.first + blockIdx.x);
  const int64_t batch = at / a.runs, run = at - batch * a.runs;
  const int each = a.c / a.groups;
  const Place me = place(a.c);
  if (!me.in) return;
  const int64_t block = kRows * me.step, blocks = (a.positions + block - 1) / block;
  int64_t b = run + (blocks - 1 - run) / a.runs * a.runs;
  // (the first rows before the statistics, the next ones before these are done)
  Raw<BF16> held[kRows];
  auto load = [&](int64_t b) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int64_t row = b * block + me.row + u * me.step;
      held[u] = load_row<BF16, WHOLE>(a.x, batch * a.xs[0] + (row < a.positions ? row : a.positions - 1) * a.xs[1] + me.c,
                                      me.left);
    }
  };
  load(b);
  float mean[8], rest[8], scale[8], bias[8];  // (the mean is the two's sum)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = me.c + (i < me.left ? i : 0);
    const f32x4 s = reinterpret_cast<const f32x4*>(a.stats)[batch * a.groups + c / each];
    mean[i] = s[0];
    rest[i] = s[1];
    scale[i] = s[2] * vector_value(a.weight, c, 1.f);
    bias[i] = vector_value(a.bias, c, 0.f);
  }
  // (The three ways apart: with the choice at each row 2 x 16384 x 320 takes 29.6 us instead of 28.8.)
  auto finish = [&](auto act) __attribute__((always_inline)) {
    for (; b >= 0; b -= a.runs) {
      const int64_t r = b * block + me.row;
      Raw<BF16> x[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) x[u] = held[u];
      if (b >= a.runs) load(b - a.runs);
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int64_t row = r + u * me.step;
        if (row >= a.positions) break;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = act(__builtin_fmaf(value_of<BF16>(x[u], i) - mean[i] - rest[i], scale[i], bias[i]));
        const int64_t to = batch * a.ys[0] + row * a.ys[1] + me.c;
        if (WHOLE || me.left == 8) {
          store_values<8>(v, a.y, a.y_bf16, to);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < me.left) store_values<1>(v + i, a.y, a.y_bf16, to + i);
        }
      }
    }
  };
  if (!a.silu)
    finish([](float n) { return n; });
  else if (a.y_bf16)
    finish([](float n) { return silu_rough(n); });
  else
    finish([](float n) { return silu(n); });
}

template <bool BF16, int V>
void launch_held(GroupNormArgs a, hipStream_t stream) {
  const int64_t vectors = a.positions * (a.c / a.groups / V);
  const int64_t waves = (vectors + 63) / 64;
  const int threads = 64 * int(waves < 16 ? waves : 16);
  in_launches(a.batch * a.groups, threads, [&](int64_t first, unsigned count) {
    a.first = first;
    hipLaunchKernelGGL((group_norm_held_kernel<BF16, V>), dim3(count), dim3(threads),
                       2 * (a.c / a.groups) * sizeof(float), stream, a);
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
    in_launches(a.batch * a.groups, kUniters, [&](int64_t first, unsigned count) {
      a.first = first;
      hipLaunchKernelGGL(group_norm_unite_kernel, dim3(count), dim3(kUniters), 0, stream, a);
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
  // A run for each CU, with a block of rows at least.  1048576 positions of 128
  // channels, 16384 of 512, 2 x 16384 of 320: 166, 26 and 29 us (158 since the
  // result's rows come ahead); with two 169, 31 and 35; with four 172, 31 and 40.  Two blocks at least: 3 x 1927 of
  // 336 in float32 22.5 us instead of 20.2.
  const int64_t rows = kRows * row_step(c);
  int64_t runs = (int64_t(device_cu_count()) + batch - 1) / batch;
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
