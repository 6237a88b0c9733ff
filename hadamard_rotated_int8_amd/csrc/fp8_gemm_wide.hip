// FP8 linear for outputs with many tiles: a persistent kernel with 256 x 256
// tiles, power-of-two scales and bfloat16 output (the formula and the
// instruction are fp8_gemm.hip's).
//
// One workgroup of 4 waves per CU, one wave per SIMD with the whole register
// file: each wave owns 128 x 128 of the tile, 16 blocks of 32 x 32 in 256
// accumulator registers, so that a 64-wide slice of K is 16 instructions of
// 64 cycles for 16 KB read from LDS (at 128 bytes a cycle half of the four
// waves' matrix time; 128 x 64 a wave would be three quarters, and the loads
// into LDS come on top).
//   * K advances by half-blocks of 64 features through a ring of 4 LDS stages
//     (32 KB each, both operands).  Direct-to-LDS loads run 4 half-blocks
//     ahead: as soon as every wave holds a half-block's fragments in
//     registers its stage is refilled.
//   * Fragments are read one half-block ahead, between the instructions: an
//     X fragment as soon as its last instruction is issued, W fragments into
//     a second set.  One barrier per half-block.
//   * The scale bytes of a block's 256 rows are one load per wave (each wave
//     has a copy of its own), read as bytes one half-block ahead; the weight
//     scales of a tile are fetched a tile ahead.
//   * The load stream does not stop at a tile's end: the next tile's first
//     four half-blocks arrive while this tile is stored.
//   * LDS rows are 64 bytes; 16-byte chunk c of row r sits at slot
//     c ^ ((r >> 2) & 3), so 16 lanes that read 16 consecutive rows touch 16
//     different groups of 4 banks.
//   * Bytes past K and rows past M or n read as zero, in both operands (a
//     NaN code of another row must not meet even a zero).
#include <mutex>

#include "fp8_gemm.h"

namespace convrot {
namespace {

constexpr int kTile = 256;
constexpr int kHalf = 64;                      // features per half-block
constexpr int kStage = 2 * kTile * kHalf;      // bytes: X rows, then W rows
constexpr int kStages = 4;
constexpr int kPieces = kStage / 1024 / 4;     // loads per wave and half-block (16 rows each)
constexpr int kScales = kStages * kStage;      // LDS offset of the scale ring: 2 blocks x 4 waves x 256 rows
constexpr int kWScales = kScales + 2 * 4 * 256;
constexpr int kMinBlocks = 3;
constexpr int64_t kMaxLdy = 1 << 21;           // a tile's rows of Y lie in 31 bits
// Weight scales of a tile: 2 rows of kb bytes, for this tile and the next.
constexpr int kMaxBlocks = 1041;               // CONVROT_MAX_K / 128, rounded up
constexpr int kLds = kWScales + 2 * 2 * kMaxBlocks;
static_assert(kLds <= 160 * 1024, "LDS");

CR_DEVICE int chunk_slot(int row) { return (row >> 2) & 3; }

template <bool GELU>
__global__ __launch_bounds__(256, 1) void fp8_gemm_wide_kernel(const Fp8Params p, int total) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLds];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int G = gridDim.x, slot = xcd_slot(blockIdx.x, G);
  const int ntiles = (total - slot + G - 1) / G;  // >= 1
  const int K = p.K, kb = p.kb;

  // ---------------------------------------------------------------- loading
  struct Operands {  // of one tile
    __amdgpu_buffer_rsrc_t x, w;
    const uint8_t* sx;  // the tile's first row in block 0 of the scales
    int srows;          // scale bytes per block, padded
  };
  auto operands = [&](int it) {
    Operands o;
    if (it >= ntiles) {  // past the end: nothing is fetched
      o.x = o.w = buffer_rsrc(nullptr, 0);
      o.sx = nullptr;
      o.srows = 0;
      return o;
    }
    const Fp8Tile t = fp8_tile<kTile, kTile>(p, slot + it * G);
    const Fp8Params::Seg& sg = p.seg[t.seg];
    const int rows = p.M - t.m0 < kTile ? p.M - t.m0 : kTile;
    const int cols = sg.n - t.n0 < kTile ? sg.n - t.n0 : kTile;
    o.x = buffer_rsrc(p.qx + (int64_t)t.m0 * K, rows * K);
    o.w = buffer_rsrc(sg.qw + (int64_t)t.n0 * K, cols * K);
    o.sx = p.sx + t.m0;
    o.srows = (rows + 3) & ~3;
    return o;
  };
  // Piece q of a stage: rows 16 q .. +15; lane l fills slot l % 4 of row
  // l / 4 with global chunk (l % 4) ^ chunk_slot(row).
  const int chunk = (lane & 3) ^ ((lane >> 4) & 3);
  const unsigned lane_off = unsigned((lane >> 2) * K + chunk * 16);
  Operands cur = operands(0), next = operands(1);
  int ls = 0, lstage = 0, lring = 0;  // the half-block being loaded, its stage and its scales' place
  unsigned voff = 0;
  auto begin_half = [&]() { voff = ls * kHalf + chunk * 16 < K ? lane_off : kOutOfRange; };
  auto piece = [&](int i) {
    const bool is_x = i < kPieces / 2;
    const int q = wave + 4 * (is_x ? i : i - kPieces / 2);
    uint8_t* dst = smem + lstage * kStage + (is_x ? 0 : kTile * kHalf) + q * 1024;
    const __amdgpu_buffer_rsrc_t rs = is_x ? cur.x : cur.w;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)dst, 16, voff, q * 16 * K + ls * kHalf, 0, 0);
  };
  auto scale_piece = [&]() {  // (ls even) the rows' scales of block ls / 2
    uint8_t* dst = smem + kScales + lring * 1024 + wave * 256;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_rsrc(cur.sx + (ls >> 1) * p.lds, cur.srows),
                                             (lds_void*)dst, 4, lane * 4, 0, 0, 0);
  };
  auto end_half = [&](bool second) {  // (a tile ends with a block's second half)
    lstage = (lstage + 1) & 3;
    ++ls;
    if (second) lring ^= 1;
    if (second && ls == 2 * kb) {
      ls = 0;
      cur = next;
    }
  };
  // The weight scales of tile `it`: entry e = (row e / kb, block e % kb).
  auto wscale_at = [&](int it, int e) -> unsigned {
    const Fp8Tile t = fp8_tile<kTile, kTile>(p, slot + it * G);
    const Fp8Params::Seg& sg = p.seg[t.seg];
    const int r = t.n0 / kFp8Block + (e >= kb ? 1 : 0), b = e >= kb ? e - kb : e;
    return r * kFp8Block < sg.n ? static_cast<const uint8_t*>(sg.sw)[(int64_t)r * kb + b] : 127u;
  };
  uint8_t* wsc = smem + kWScales;

  // -------------------------------------------------------------- fragments
  const int fr = lane & 31, fh = lane >> 5;
  const int fb0 = fr * kHalf + ((fh ^ chunk_slot(fr)) << 4);
  const int fb1 = fr * kHalf + (((2 + fh) ^ chunk_slot(fr)) << 4);
  v8i xf[4], wf[2][4];
  auto frag = [&](const uint8_t* rows) -> v8i {
    const v4i a = *reinterpret_cast<const v4i*>(rows + fb0);
    const v4i b = *reinterpret_cast<const v4i*>(rows + fb1);
    return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  };
  auto read_x = [&](const uint8_t* st, int i) { xf[i] = frag(st + (wm * 128 + i * 32) * kHalf); };
  auto read_w = [&](const uint8_t* st, int set, int j) {
    wf[set][j] = frag(st + kTile * kHalf + (wn * 128 + j * 32) * kHalf);
  };
  int sx[4], sw, nsx[4], nsw;
  auto read_scales = [&](int ring, int it, int b) {
    const uint8_t* s = smem + kScales + ring * 1024 + wave * 256 + wm * 128 + fr;
#pragma unroll
    for (int i = 0; i < 4; ++i) nsx[i] = s[32 * i];
    nsw = wsc[((it & 1) * 2 + wn) * kb + b];
  };
  f32x16 acc[4][4];

  // --------------------------------------------------------------- prologue
#pragma unroll 1
  for (int e = threadIdx.x; e < 2 * kb; e += 256) wsc[e] = uint8_t(wscale_at(0, e));
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    begin_half();
#pragma unroll
    for (int i = 0; i < kPieces; ++i) piece(i);
    if (h % 2 == 0) scale_piece();
    end_half(h % 2 == 1);
  }
  waitvm<3 * kPieces + 1>();  // half-block 0 and its scales
  wait_lgkm0();
  barrier();
  int stage = 0, ring = 0;  // of the block being computed: its first stage, its scales
  // A tile's first fragments and scales (its first half-block has landed).
  auto prime = [&](int it) __attribute__((always_inline)) {
    const uint8_t* st = smem + stage * kStage;
#pragma unroll
    for (int i = 0; i < 4; ++i) read_x(st, i);
#pragma unroll
    for (int j = 0; j < 4; ++j) read_w(st, 0, j);
    read_scales(ring, it, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) sx[i] = nsx[i];
    sw = nsw;
  };
  // A use of the accumulators: without one the compiler sinks a tile's first
  // and last instructions to whatever comes after the next branch.
  auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));
  };

  // One half-block; T: the block's first or second.  FIRST, LAST: the tile's
  // (PIN: of its first or last block; the last reads no fragments ahead: they would have to live through the
  // tile's end).  nb: the block whose scales the second half reads ahead.
  auto half = [&](auto first_t, auto last_t, auto pin_t, auto t_t, int it, int nb) __attribute__((always_inline)) {
    constexpr bool FIRST = decltype(first_t)::value;
    constexpr bool LAST = decltype(last_t)::value;
    constexpr bool PIN = decltype(pin_t)::value;
    constexpr int T = decltype(t_t)::value;
    const uint8_t* nx = smem + ((stage + T + 1) & 3) * kStage;
#pragma unroll
    for (int idx = 0; idx < 16; ++idx) {
      const int i = idx / 4, j = idx % 4;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          wf[T][j], xf[i], FIRST ? f32x16{} : acc[i][j], 0, 0, 0, sw, 0, sx[i]);
      __builtin_amdgcn_sched_barrier(0);
      if (idx == 1) {
        // The next half-block has landed once only the loads of the two after
        // it may be in flight (one of them brings a block's scales); this
        // one's fragments are all in registers.
        waitvm<2 * kPieces + 1>();
        wait_lgkm0();
        barrier();
        begin_half();
      }
      if (!LAST) {
        if (idx % 4 == 3) read_x(nx, i);
        if (idx >= 2 && idx % 2 == 0 && idx < 10) read_w(nx, 1 - T, idx / 2 - 1);
        if (T == 1 && idx == 10) read_scales(ring ^ 1, it, nb);
      }
      if (idx >= 2) {
        constexpr int slots = 14;
#pragma unroll
        for (int d = 0; d < kPieces; ++d)
          if (idx == 2 + (2 * d + 1) * slots / (2 * kPieces)) piece(d);
        if (T == 0 && idx == 14) scale_piece();
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (PIN) pin();
    end_half(T == 1);
    if (T == 1) {
      stage = (stage + 2) & 3;
      ring ^= 1;
      if (!LAST) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sx[i] = nsx[i];
        sw = nsw;
      }
    }
  };
  using Yes = std::true_type;
  using No = std::false_type;
  using T0 = std::integral_constant<int, 0>;
  using T1 = std::integral_constant<int, 1>;

  for (int it = 0; it < ntiles; ++it) {
    const Fp8Tile t = fp8_tile<kTile, kTile>(p, slot + it * G);
    const bool more = it + 1 < ntiles;
    next = operands(it + 1);
    // The next tile's weight scales: fetched here, laid down after the first block.
    const int e0 = threadIdx.x;
    unsigned ws0 = 127;
    if (more && e0 < 2 * kb) ws0 = wscale_at(it + 1, e0);
    prime(it);
    half(Yes{}, No{}, No{}, T0{}, it, 0);
    half(No{}, No{}, Yes{}, T1{}, it, 1);
    if (more) {
      uint8_t* d = wsc + ((it + 1) & 1) * 2 * kb;
      if (e0 < 2 * kb) d[e0] = uint8_t(ws0);
#pragma unroll 1
      for (int e = e0 + 256; e < 2 * kb; e += 256) d[e] = uint8_t(wscale_at(it + 1, e));
    }
    for (int b = 1; b < kb - 1; ++b) {
      half(No{}, No{}, No{}, T0{}, it, 0);
      half(No{}, No{}, No{}, T1{}, it, b + 1);
    }
    half(No{}, No{}, No{}, T0{}, it, 0);
    half(No{}, Yes{}, Yes{}, T1{}, it, 0);

    // Store.  Register e of block (i, j): column 8 (e / 4) + 4 (lane / 32) +
    // e % 4, row lane % 32.  Two quads of bfloat16 pairs trade half-waves, so
    // that a lane holds 8 consecutive columns.
    // (Lane numbers are re-formed here rather than kept through the K loop.)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int fr = lane & 31, fh = lane >> 5;
    const Fp8Params::Seg& sg = p.seg[t.seg];
    const int cols = sg.n - t.n0;
    const int ldy = int(sg.ldy);
    uint16_t* y = static_cast<uint16_t*>(sg.y);
    const __amdgpu_buffer_rsrc_t br =
        buffer_rsrc(sg.bias ? sg.bias + t.n0 : nullptr, sg.bias ? (cols < kTile ? cols : kTile) * 4 : 0);
    // A resource over the tile's rows (those past M are outside it); the lane's
    // offset is fixed, row blocks go into the scalar and column blocks into
    // the immediate offset.  (ldy < kMaxLdy: see fp8_wide_wanted.)
    const int rows = p.M - t.m0 < kTile ? p.M - t.m0 : kTile;
    const bool whole = cols >= kTile && (ldy & 7) == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
    const __amdgpu_buffer_rsrc_t yr = buffer_rsrc(
        y + (int64_t)t.m0 * ldy + t.n0, ((rows - 1) * ldy + (cols < kTile ? cols : kTile)) * 2);
    const unsigned yoff = unsigned((wm * 128 + fr) * ldy + wn * 128 + 8 * fh) * 2;
    auto store = [&](auto whole_t) __attribute__((always_inline)) {
      constexpr bool WHOLE = decltype(whole_t)::value;  // every column exists, rows 16-byte aligned
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4 bias[4];
        const int c0 = wn * 128 + j * 32;  // the block's first column in the tile
#pragma unroll
        for (int q = 0; q < 4; ++q)
          bias[q] = __builtin_bit_cast(
              f32x4, __builtin_amdgcn_raw_buffer_load_b128(br, unsigned(c0 + 8 * q + 4 * fh) * 4, 0, 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // One block at a time leaves the accumulators' half of the register
          // file (and, opaque, is not formed for both branches at once).
          f32x16 sum = acc[i][j];
          asm volatile("" : "+v"(sum));
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            u32x2 w[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const int q = 2 * q2 + s;
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[e] = sum[4 * q + e] + bias[q][e];
                if constexpr (GELU) v[e] = gelu_erf(v[e]);
              }
              w[s] = u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
            }
            const auto a = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
            const auto b = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
            // a, b: columns 8 g .. +3 and +4 .. +7 of the block, g = 2 q2 + lane / 32
            const u32x4 out = {a[0], b[0], a[1], b[1]};
            const int c = c0 + 16 * q2 + 8 * fh;
            if constexpr (WHOLE) {
              __builtin_amdgcn_raw_buffer_store_b128(out, yr, yoff + j * 64 + q2 * 32, i * 64 * ldy, 0);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                __builtin_amdgcn_raw_buffer_store_b16(
                    uint16_t(out[e / 2] >> (16 * (e & 1))), yr,
                    c + e < cols ? yoff + j * 64 + q2 * 32 + e * 2 : kOutOfRange, i * 64 * ldy, 0);
            }
          }
        }
      }
    };
    if (whole)
      store(Yes{});
    else
      store(No{});
  }
  waitvm<0>();  // no load into LDS may be in flight at the end
}

}  // namespace

bool fp8_wide_wanted(const Fp8GemmArgs& a) {
  if (a.f32_scale || !a.y_bf16 || (a.k + kFp8Block - 1) / kFp8Block < kMinBlocks) return false;
  int64_t tiles = 0;
  for (int i = 0; i < a.count; ++i) {
    if (a.w[i].ldy >= kMaxLdy) return false;
    tiles += ((a.m + kTile - 1) / kTile) * ((a.w[i].n + kTile - 1) / kTile);
  }
  return tiles >= device_cu_count();
}

hipError_t launch_fp8_gemm_wide(const Fp8GemmArgs& a, hipStream_t stream) {
  const Fp8Params p = fp8_params<kTile, kTile>(a);
  const int total = p.tiles_m * p.tiles_n;
  const int cus = device_cu_count();
  const dim3 grid(total < cus ? total : cus);
  if (a.gelu)
    hipLaunchKernelGGL(fp8_gemm_wide_kernel<true>, grid, dim3(256), 0, stream, p, total);
  else
    hipLaunchKernelGGL(fp8_gemm_wide_kernel<false>, grid, dim3(256), 0, stream, p, total);
  return hipGetLastError();
}

}  // namespace convrot
