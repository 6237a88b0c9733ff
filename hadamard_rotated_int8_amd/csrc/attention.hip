// Attention of m queries to l keys, softmax(scale Q K^T) V, on CDNA4 matrix
// cores: one pass over the keys with a running maximum and sum.
//
// A wave holds the transposed scores S^T = K Q^T of 32 queries: a lane then
// has 16 keys of one query in registers, its maximum takes one exchange with
// the other half of the wave, and the 8 values it holds of 16 keys are as they
// stand the second operand of O^T = V^T P^T (both operands of a product may
// name its 16 terms in any order, as long as it is the same).  V^T is read
// from LDS with the transposing read, so K and V lie there as they come.
#include "common.h"
#include "kernels.h"

namespace convrot {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr int kKeys = 64;  // keys of a tile
constexpr int kWaves = 4;
constexpr float kLog2e = 1.44269504f;
constexpr float kMinusInf = -__builtin_inff();

// The 16-byte chunk c of row r of a tile lies at slot c ^ swizzle(r).  A
// fragment of K is one chunk of 32 rows, read 16 lanes at a time (rows that
// differ in their last 4 bits), one of V 4 chunks of 4 rows: both then touch
// every bank once.
template <int kPitch>
CR_DEVICE int key_swizzle(int row) {
  return kPitch == 128 ? (row >> 1) & 7 : row & 15;
}
template <int kPitch>
CR_DEVICE int value_swizzle(int row) {
  return kPitch == 128 ? (row & 2) << 1 : (row & 3) << 2;
}

CR_DEVICE float other_half(float v) {  // lane ^ 32
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// D: the head's features rounded up to 32.  QB: blocks of 32 queries of a wave.
template <int D, int QB>
__global__ __launch_bounds__(kWaves * 64) void attention_kernel(const AttentionArgs p) {
  constexpr int kPitch = D <= 64 ? 128 : D <= 128 ? 256 : 512;  // bytes of a row in LDS
  constexpr int kChunks = kPitch / 16;
  constexpr int kRowsPiece = 1024 / kPitch;   // rows that one load instruction of a wave brings
  constexpr int kTile = kKeys * kPitch;       // bytes of K, or of V
  constexpr int kPieces = kTile / 1024 / kWaves;
  constexpr int kRows = kWaves * QB * 32;     // queries of a workgroup
  __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * kTile];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 31, fh = lane >> 5;
  // Neighbouring workgroups of an XCD share a head's keys.
  int slot = int(p.first) + xcd_slot(blockIdx.x, gridDim.x);
  const int split = slot % p.splits;
  slot /= p.splits;
  const int tile = slot % p.tiles;
  slot /= p.tiles;
  const int head = slot % p.kv_heads, batch = slot / p.kv_heads;
  const int64_t rows = p.m * p.ratio;  // a key head's queries, (token, query head)
  const int64_t row0 = int64_t(tile) * kRows + wave * QB * 32;

  int64_t keys = p.l;
  if (p.lengths) {
    const int n = p.lengths[batch];
    keys = n < 0 ? 0 : n < keys ? n : keys;
  }
  const int64_t all = (keys + kKeys - 1) / kKeys;  // tiles of keys
  const int first = int(all * split / p.splits), last = int(all * (split + 1) / p.splits);
  const uint16_t* kbase = p.k + batch * p.ks[0] + head * p.ks[2];
  const uint16_t* vbase = p.v + batch * p.vs[0] + head * p.vs[2];
  const uint8_t* mask = p.mask ? p.mask + batch * p.mask_stride : nullptr;
  const int dbytes = p.d * 2;

  // The keys of tile t that take part, one bit for each.
  auto tile_mask = [&](int t) -> uint64_t {
    const int64_t left = keys - int64_t(t) * kKeys;
    if (left <= 0) return 0;
    if (!mask) return left >= kKeys ? ~uint64_t(0) : (uint64_t(1) << left) - 1;
    return __ballot(lane < left && mask[int64_t(t) * kKeys + lane] != 0);
  };
  // Rows of K and V of tile t into LDS area `to`; absent keys and features
  // read as zero (a NaN of a hidden V must not meet a weight of zero).
  auto issue = [&](int t, int to, uint64_t seen) {
    const __amdgpu_buffer_rsrc_t kr = buffer_rsrc(kbase + int64_t(t) * kKeys * p.ks[1], 0x7FFFFFFF);
    const __amdgpu_buffer_rsrc_t vr = buffer_rsrc(vbase + int64_t(t) * kKeys * p.vs[1], 0x7FFFFFFF);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int q = wave + kWaves * i;
      const int row = q * kRowsPiece + lane / kChunks, at = lane % kChunks;
      const bool in = (seen >> row) & 1;
      const int kc = (at ^ key_swizzle<kPitch>(row)) * 16, vc = (at ^ value_swizzle<kPitch>(row)) * 16;
      uint8_t* dst = smem + to * 2 * kTile + q * 1024;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(kr, (lds_void*)dst, 16,
                                               in && kc < dbytes ? unsigned(row * int(p.ks[1]) * 2 + kc) : kOutOfRange,
                                               0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(vr, (lds_void*)(dst + kTile), 16,
                                               in && vc < dbytes ? unsigned(row * int(p.vs[1]) * 2 + vc) : kOutOfRange,
                                               0, 0, 0);
    }
  };

  // Q: lane l holds query l % 32, features 16 t + 8 (l / 32) .. +7.
  bf16x8 qf[QB][D / 16];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const int64_t r = row0 + 32 * b + fr;
    const int64_t token = r / p.ratio, j = r - token * p.ratio;
    const uint16_t* src = p.q + batch * p.qs[0] + token * p.qs[1] + (head * p.ratio + j) * p.qs[2];
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      const int f = 16 * t + 8 * fh;
      qf[b][t] = r < rows && f < p.d ? *reinterpret_cast<const bf16x8*>(src + f) : bf16x8{};
    }
  }

  f32x16 o[QB][D / 32] = {};
  float top[QB], total[QB];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    top[b] = kMinusInf;
    total[b] = 0.f;
  }
  const float c = p.scale * kLog2e;

  uint64_t seen = first < last ? tile_mask(first) : 0;
  if (first < last) issue(first, 0, seen);
  for (int t = first; t < last; ++t) {
    const uint8_t* kt = smem + ((t - first) & 1) * 2 * kTile;
    const uint8_t* vt = kt + kTile;
    const uint64_t next = t + 1 < last ? tile_mask(t + 1) : 0;
    waitvm<0>();  // this tile has landed, and every wave has read the one before it
    barrier();
    if (t + 1 < last) issue(t + 1, (t + 1 - first) & 1, next);
#pragma unroll
    for (int g = 0; g < kKeys / 32; ++g) {
      const unsigned bits = unsigned(seen >> (32 * g));
      f32x16 s[QB] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const int row = 32 * g + fr;
        const bf16x8 kf =
            *reinterpret_cast<const bf16x8*>(kt + row * kPitch + (((2 * k + fh) ^ key_swizzle<kPitch>(row)) << 4));
#pragma unroll
        for (int b = 0; b < QB; ++b) s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[b][k], s[b], 0, 0, 0);
      }
      bf16x8 pf[QB][2];
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        // Register e: key 8 (e / 4) + 4 (lane / 32) + e % 4 of the 32.
        if (bits != ~0u) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (!((bits >> (8 * (e / 4) + 4 * fh + e % 4)) & 1)) s[b][e] = kMinusInf;
        }
        float most = s[b][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) most = fmaxf(most, s[b][e]);
        most = fmaxf(most, other_half(most));
        const float now = fmaxf(top[b], most);
        const float base = now == kMinusInf ? 0.f : now;
        const float shrink = __builtin_amdgcn_exp2f((top[b] - base) * c);
        top[b] = now;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const __bf16 w = (__bf16)__builtin_amdgcn_exp2f((s[b][e] - base) * c);
          pf[b][e / 8][e % 8] = w;
          sum += float(w);
        }
        total[b] = total[b] * shrink + sum;
#pragma unroll
        for (int n = 0; n < D / 32; ++n) o[b][n] *= shrink;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < D / 32; ++n) {
          i16x4 part[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = 32 * g + 16 * h + 8 * i + 4 * fh + ((lane & 15) >> 2);
            const int chunk = 4 * n + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
            part[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_i16x4*)(vt + row * kPitch + ((chunk ^ value_swizzle<kPitch>(row)) << 4) + (lane & 1) * 8));
          }
          const bf16x8 vf = __builtin_bit_cast(
              bf16x8, i16x8{part[0][0], part[0][1], part[0][2], part[0][3], part[1][0], part[1][1], part[1][2],
                            part[1][3]});
#pragma unroll
          for (int b = 0; b < QB; ++b) o[b][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[b][h], o[b][n], 0, 0, 0);
        }
    }
    seen = next;
  }

  // Register e of block n: feature 32 n + 8 (e / 4) + 4 (lane / 32) + e % 4 of query lane % 32.
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const float sum = total[b] + other_half(total[b]);
    const int64_t r = row0 + 32 * b + fr;
    if (r >= rows) continue;
    const int64_t token = r / p.ratio, j = r - token * p.ratio;
    if (p.splits > 1) {
      const int64_t at = ((int64_t(split) * p.batch + batch) * p.kv_heads + head) * rows + r;
      float* dst = p.part + at * p.d;
      if (fh == 0) {
        p.stats[2 * at] = top[b] * c;
        p.stats[2 * at + 1] = sum;
      }
#pragma unroll
      for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int f = 32 * n + 8 * q + 4 * fh;
          if (f < p.d)
            *reinterpret_cast<f32x4*>(dst + f) =
                f32x4{o[b][n][4 * q], o[b][n][4 * q + 1], o[b][n][4 * q + 2], o[b][n][4 * q + 3]};
        }
      continue;
    }
    uint16_t* dst = p.out + batch * p.os[0] + token * p.os[1] + (head * p.ratio + j) * p.os[2];
    const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = 32 * n + 8 * q + 4 * fh;
        if (at < p.d)
          *reinterpret_cast<u32x2*>(dst + at) =
              u32x2{bf16_pair(o[b][n][4 * q] * f, o[b][n][4 * q + 1] * f),
                    bf16_pair(o[b][n][4 * q + 2] * f, o[b][n][4 * q + 3] * f)};
      }
  }
}

// The parts of a split, joined: thread = 4 features of a row.
__global__ __launch_bounds__(256) void attention_join_kernel(const AttentionArgs p, int64_t first) {
  const int quads = p.d / 4;
  const int64_t rows = p.m * p.ratio, count = p.batch * p.kv_heads * rows;
  const int64_t i = (first + blockIdx.x) * 256 + threadIdx.x;
  const int64_t r = i / quads;
  const int f = int(i - r * quads) * 4;
  if (r >= count) return;
  float top = kMinusInf;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, p.stats[2 * (s * count + r)]);
  const float base = top == kMinusInf ? 0.f : top;
  f32x4 v = {};
  float sum = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float w = __builtin_amdgcn_exp2f(p.stats[2 * (s * count + r)] - base);
    sum += w * p.stats[2 * (s * count + r) + 1];
    v += w * *reinterpret_cast<const f32x4*>(p.part + (s * count + r) * p.d + f);
  }
  v *= sum == 0.f ? 0.f : 1.f / sum;
  const int64_t pair = r / rows, in = r - pair * rows, token = in / p.ratio;
  const int64_t batch = pair / p.kv_heads, head = (pair - batch * p.kv_heads) * p.ratio + in - token * p.ratio;
  *reinterpret_cast<u32x2*>(p.out + batch * p.os[0] + token * p.os[1] + head * p.os[2] + f) =
      u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
}

template <int D, int QB>
hipError_t launch_t(const AttentionArgs& a, hipStream_t stream) {
  AttentionArgs p = a;
  in_launches(a.batch * a.kv_heads * a.tiles * a.splits, kWaves * 64, [&](int64_t first, unsigned count) {
    p.first = first;
    hipLaunchKernelGGL((attention_kernel<D, QB>), dim3(count), dim3(kWaves * 64), 0, stream, p);
  });
  if (a.splits > 1) {
    const int64_t values = a.batch * a.kv_heads * a.m * a.ratio * (a.d / 4);
    in_launches((values + 255) / 256, 256, [&](int64_t first, unsigned count) {
      hipLaunchKernelGGL(attention_join_kernel, dim3(count), dim3(256), 0, stream, p, first);
    });
  }
  return hipGetLastError();
}

}  // namespace

AttentionPlan plan_attention(int64_t batch, int64_t kv_heads, int64_t rows, int64_t l, int d) {
  constexpr int kTileRows = kWaves * 32;
  AttentionPlan plan{};
  plan.tiles = (rows + kTileRows - 1) / kTileRows;
  plan.splits = 1;
  const int64_t blocks = batch * kv_heads * plan.tiles, cus = device_cu_count();
  const int64_t key_tiles = (l + kKeys - 1) / kKeys;
  if (blocks > 0 && blocks < cus) {
    int64_t want = cus / blocks;
    if (want > key_tiles / 2) want = key_tiles / 2;
    if (want > 1) plan.splits = int(want);
  }
  return plan;
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t stream) {
  if (a.d <= 64) return launch_t<64, 1>(a, stream);
  if (a.d <= 96) return launch_t<96, 1>(a, stream);
  if (a.d <= 128) return launch_t<128, 1>(a, stream);
  if (a.d <= 160) return launch_t<160, 1>(a, stream);
  return launch_t<256, 1>(a, stream);
}

}  // namespace convrot
