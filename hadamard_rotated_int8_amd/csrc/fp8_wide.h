// FP8 products for bfloat16 outputs with many tiles: a persistent kernel with
// 256 x 256 tiles for power-of-two scales and 256 x 128 for float32 weight
// scales (the formula is fp8_gemm.hip's).  fp8_gemm_wide.hip makes the linear
// of it, fp8_gated.hip the gated pair of projections.
//
// With power-of-two scales:
//
// One workgroup of 4 waves per CU, one wave per SIMD with the whole register
// file: each wave owns 128 x 128 of the tile, 64 blocks of 16 x 16 in 256
// accumulator registers.  A block of 128 features is one
// v_mfma_scale_f32_16x16x128_f8f6f4 per 16 x 16 block (64 of them, 32 cycles
// each) for 32 KB read from LDS, half of what LDS can deliver to four waves
// in that time.  Under full load the chip is bound by power, and this form
// gives 4.2 PFLOP/s in a loop on registers where v_mfma_scale_f32_32x32x64
// gives 3.9 (random codes; 5.0 on zeros for both).
//   * Work goes in half-blocks: 32 instructions, 4 rows of 16 x 16 blocks.
//     During a half-block the fragments of the next block's same rows are
//     read: an X fragment into the registers of the one just used up, W
//     fragments into a second set.
//   * LDS is a ring of 4 half-stages of 32 KB: half-stage 2 v + h holds the
//     64 rows of each wave's X and W that half h of block v - 1 reads.  Its
//     direct-to-LDS loads are issued three half-blocks before, into the slot
//     that every wave has read by then.  One barrier per half-block.
//   * The scale bytes of a block's 256 rows are one load per wave (each wave
//     has a copy of its own); the weight scales of a tile are fetched a tile
//     ahead.
//   * Neither the loads nor the reads stop at a tile's end: the next tile's
//     first half-stages arrive, and its first fragments are read, before this
//     tile is stored, and its first three half-blocks wait for no store.
//   * A tile's bias and weight scales come into LDS a tile ahead.
//   * LDS rows are 128 bytes; 16-byte chunk c of row r sits at slot c ^ (r & 7).
//     A 16-byte read is served 16 lanes at a time, lanes 0-3, 12-15, 20-23 and
//     24-27 first; of a fragment these hold rows 0-3 and 12-15 of one chunk
//     and rows 4-11 of the next, in 16 different groups of 4 banks.  (With
//     bit 3 of the row in the slot as well, which suits 16 rows of one chunk,
//     46 % of the LDS' busy cycles were conflicts.)
//   * Bytes past K and rows past M or n read as zero, in both operands (a
//     NaN code of another row must not meet even a zero).
//   * A tile is stored 16 rows x 64 columns at a time through LDS, as whole
//     128-byte lines, non-temporal (Y should not push operands out of L2).
//
// float32 weight scales are applied by one fused multiply-add per output and
// block, between the matrix instructions, which therefore start from zero and
// write vector registers; those hold the accumulators of 128 x 64 per wave,
// and the operands are in the accumulation half.  A block takes 1024 cycles
// of matrix instructions for 96 KB read from LDS and 48 KB loaded into it
// (1152 cycles at 128 bytes each), so LDS binds it as well as the
// multiply-adds: without the reads the loop is 20 % faster, without the
// multiply-adds 16 %.  4096 x 4096 -> 12288 takes 238 to 252 us with its pack,
// 1 % of it the wait states before each instruction.
//
// GATED: the tile's columns are 128 (64) rows of the gate's weights and the
// same rows of the up projection's, so that a tile gives 128 (64) columns of
// act(gate) * up.  Of each wave's columns the first half of a half-stage pair
// is the gate's and the second the up projection's: nothing changes but where
// W comes from, which of two weight scales an instruction takes, and that the
// two sums of an output meet in the lane that has both.
#pragma once

#include <type_traits>

#include "fp8_gemm.h"

namespace convrot {
namespace {

enum { kPlain = 0, kGated = 1, kGatedKept = 2 };  // kGatedKept: both projections are outputs too

constexpr int kBM = 256;
constexpr int kMinBlocks = 3;
constexpr int64_t kMaxLdy = 1 << 21;           // a tile's rows of Y lie in 31 bits

// Tiles of 256 x 256, or 256 x 128 with float32 weight scales: FN 16-column
// blocks per wave.
template <bool F32, int MODE = kPlain>
struct WideCfg {
  static constexpr int BN = F32 ? 128 : 256;               // rows of W
  static constexpr int OUTS = MODE == kPlain ? BN : BN / 2;  // columns of Y
  static constexpr int FN = BN / 32;
  static constexpr int XHALF = 128 * kBK;                  // bytes of X in a half-stage: 64 rows per wave
  static constexpr int HALF = XHALF + BN / 2 * kBK;        // ... and of W
  static constexpr int XP = XHALF / 1024 / 4;              // loads per wave and half-stage (8 rows each)
  static constexpr int WP = BN / 2 * kBK / 1024 / 4;
  static constexpr int PIECES = XP + WP;
  static constexpr int SCALES = 4 * HALF;                  // LDS offsets: 4 blocks x 4 waves x 256 rows
  static constexpr int WSCALES = SCALES + 4 * 4 * 256;     // 2 tiles x scale rows x blocks
  static constexpr int WROWS = F32 && MODE == kPlain ? 1 : 2;  // scale rows of a tile
  static constexpr int WSIZE = F32 ? 4 : 1;
  static constexpr int BIAS = (WSCALES + 2 * WROWS * kMaxBlocks * WSIZE + 1023) / 1024 * 1024;
  static constexpr int OUT = BIAS + 2048;                  // 4 KB per wave
  static constexpr int LDS = OUT + 4 * 4096;
  // A wave's stores of a whole tile (an edge tile has more).
  static constexpr int STORES = MODE == kPlain ? 4 * FN : MODE == kGated ? 2 * FN : 6 * FN;
  static constexpr int LOADED = 2 * PIECES + 1;            // loads in flight behind a half-stage that is read
  // ... and with a tile's stores behind them, or as many as a wait can name.
  static constexpr int STORED = LOADED + STORES < kVmMax ? LOADED + STORES : kVmMax;
  static_assert(LDS <= 160 * 1024, "LDS");
};

CR_DEVICE int swz128(int row) { return row & 7; }

// One 16 x 16 x 128 product onto (FIRST: into) its accumulators.  As inline
// assembly, since all 256 accumulation registers hold the tile: the sum has to
// stay in its registers, and the compiler, free to choose others, spills.  It
// also keeps the instructions where they are written (the compiler would sink
// a tile's last ones past the next branch).  The compiler does not see that it
// is a matrix instruction.  FRESH: an operand may have been written by the
// vector instruction before (scale bytes are widened where they are first
// used), which takes 2 wait states.  mfma_settle comes before results are
// read.  tests/test_matrix_registers.py checks the built code for both: that
// the compiler puts no copy right before an instruction without the wait, and
// nothing that touches a result too early behind one.
template <bool FIRST, bool FRESH>
CR_DEVICE void mfma(f32x4& c, v8i w, v8i x, int sw, int sx) {
  if constexpr (FIRST && FRESH)
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, 0, %3, %4 op_sel_hi:[0,0,0]"
                 : "=a"(c)
                 : "v"(w), "v"(x), "v"(sw), "v"(sx));
  else if constexpr (FIRST)
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, 0, %3, %4 op_sel_hi:[0,0,0]"
                 : "=a"(c)
                 : "v"(w), "v"(x), "v"(sw), "v"(sx));
  else if constexpr (FRESH)
    asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
                 : "+a"(c)
                 : "v"(w), "v"(x), "v"(sw), "v"(sx));
  else
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0]"
                 : "+a"(c)
                 : "v"(w), "v"(x), "v"(sw), "v"(sx));
}
// A product by itself, from zero, for float32 weight scales: those are applied
// by vector instructions, which reach only half of the registers.  The
// accumulators are kept there and the operands in the other half.  The
// compiler may copy any operand there right before the instruction (it does so
// with W fragments that it carries round the K loop), so the 2 wait states
// come before every one.  It does not wait for c; kPartLead instructions later
// it is there.
CR_DEVICE void mfma_part(f32x4& c, v8i w, v8i x, int one, int sx) {
  asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, 0, %3, %4 op_sel_hi:[0,0,0]"
               : "=&v"(c)
               : "a"(w), "a"(x), "v"(one), "v"(sx));
}
constexpr int kPartLead = 3;  // 96 cycles; 11 wait states of 4 are needed
CR_DEVICE void mfma_settle() { asm volatile("s_nop 15\n\ts_nop 3" ::: "memory"); }  // 8 passes: 18 states

template <bool GELU, bool F32, int MODE>
CR_DEVICE void fp8_wide(const Fp8Params& p, int total) {
  using C = WideCfg<F32, MODE>;
  constexpr int FN = C::FN, BN = C::BN, OUTS = C::OUTS;
  constexpr bool GATED = MODE != kPlain;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int G = gridDim.x, slot = xcd_slot(blockIdx.x, G);
  const int ntiles = (total - slot + G - 1) / G;  // >= 1
  // Blocks come in pairs, one for each set of W fragments: an odd number of
  // them gets one of zeros.
  const int K = p.K, kb = p.kb, nb = (kb + 1) & ~1;  // nb >= 4

  // ---------------------------------------------------------------- loading
  struct Operands {  // of one tile
    __amdgpu_buffer_rsrc_t x, w, u;  // (u: the up projection's weights)
    const uint8_t* sx;  // the tile's first row in block 0 of the scales
    int srows;          // scale bytes per block, padded
  };
  // The bias of tile `it` (zeros without one and past n): 64 floats per wave.
  auto load_bias = [&](int it) {
    const Fp8Tile t = fp8_tile<kBM, OUTS>(p, slot + it * G);
    const int which = GATED ? wave * 64 / OUTS : 0;  // (gated: the up projection's behind the gate's)
    const Fp8Params::Seg& sg = p.seg[GATED ? which & 1 : t.seg];
    const int cols = sg.n - t.n0 < OUTS ? sg.n - t.n0 : OUTS;
    const __amdgpu_buffer_rsrc_t rs =
        buffer_rsrc(sg.bias + (sg.bias ? t.n0 : 0), sg.bias && which < 2 ? cols * 4 : 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(smem + C::BIAS + (it & 1) * 1024 + wave * 256), 4,
                                             (wave * 64 - which * OUTS + lane) * 4, 0, 0, 0);
  };
  auto operands = [&](int it) {
    if (it >= ntiles)  // past the end: nothing is fetched
      return Operands{buffer_rsrc(nullptr, 0), buffer_rsrc(nullptr, 0), buffer_rsrc(nullptr, 0), p.sx, 0};
    const Fp8Tile t = fp8_tile<kBM, OUTS>(p, slot + it * G);
    const Fp8Params::Seg& sg = p.seg[t.seg];
    const int rows = p.M - t.m0 < kBM ? p.M - t.m0 : kBM;
    const int cols = sg.n - t.n0 < OUTS ? sg.n - t.n0 : OUTS;
    return Operands{buffer_rsrc(p.qx + (int64_t)t.m0 * K, rows * K),
                    buffer_rsrc(sg.qw + (int64_t)t.n0 * K, cols * K),
                    buffer_rsrc(GATED ? p.seg[1].qw + (int64_t)t.n0 * K : nullptr, GATED ? cols * K : 0),
                    p.sx + t.m0, (rows + 3) & ~3};
  };
  // Piece q of an operand in half-stage h: LDS rows 8 q .. +7.  Of X (q < 16)
  // these are rows 64 h + 8 q .. of the first wave's 128 (q < 8) or of the
  // second's; of W likewise, with BN / 2 columns per wave.  Lane l fills slot
  // l % 8 of row l / 8 with global chunk (l % 8) ^ swz128(row).
  const int chunk = (lane & 7) ^ (lane >> 3);
  const unsigned lane_off = unsigned((lane >> 3) * K + chunk * 16);
  Operands cur = operands(0), next = operands(1);
  // The half-stage being loaded: its block, half and slot, and its scales' place.
  int lb = 0, lhalf = 0, lslot = 0, lring = 0;
  unsigned voff = 0;
  __amdgpu_buffer_rsrc_t wsrc = cur.w;
  auto begin_load = [&](bool second) {
    voff = lb * kBK + chunk * 16 < K ? lane_off : kOutOfRange;
    if (GATED) wsrc = second ? cur.u : cur.w;
  };
  auto piece = [&](int i) {
    const bool is_x = i < C::XP;
    const int q = wave + 4 * (is_x ? i : i - C::XP);
    constexpr int WQ = BN / 32;  // W pieces of one wave
    const int row = is_x    ? lhalf * 64 + (q & 7) * 8 + (q >> 3) * 128
                    : GATED ? (q % WQ) * 8 + (q / WQ) * (BN / 4)
                            : lhalf * (BN / 4) + (q % WQ) * 8 + (q / WQ) * (BN / 2);
    uint8_t* dst = smem + lslot * C::HALF + (is_x ? 0 : C::XHALF) + q * 1024;
    const __amdgpu_buffer_rsrc_t rs = is_x ? cur.x : GATED ? wsrc : cur.w;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)dst, 16, voff, row * K + lb * kBK, 0, 0);
  };
  auto scale_piece = [&]() {  // (first halves) the rows' scales of the block
    uint8_t* dst = smem + C::SCALES + lring * 1024 + wave * 256;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_rsrc(cur.sx + lb * p.lds, lb < kb ? cur.srows : 0),
                                             (lds_void*)dst, 4, lane * 4, 0, 0, 0);
  };
  auto end_load = [&](bool second) {
    lslot = (lslot + 1) & 3;
    lhalf ^= 1;
    if (second) {
      lring = (lring + 1) & 3;
      if (++lb == nb) {
        lb = 0;
        cur = next;
      }
    }
  };
  // The weight scales of tile `it`: entry e = (row e / nb, block e % nb); one
  // where there is no weight.
  using WScale = typename std::conditional<F32, float, uint8_t>::type;
  auto wscale_at = [&](int it, int e) -> WScale {
    const Fp8Tile t = fp8_tile<kBM, OUTS>(p, slot + it * G);
    const Fp8Params::Seg& sg = p.seg[GATED ? (e >= nb ? 1 : 0) : t.seg];
    const int r = t.n0 / kFp8Block + (!GATED && e >= nb ? 1 : 0), b = e >= nb ? e - nb : e;
    return r * kFp8Block < sg.n && b < kb ? static_cast<const WScale*>(sg.sw)[(int64_t)r * kb + b]
                                          : WScale(F32 ? 1 : 127);
  };
  WScale* wsc = reinterpret_cast<WScale*>(smem + C::WSCALES);
  const int entries = C::WROWS * nb;                        // of a tile
  const int wrow = F32 || GATED ? 0 : wn;                   // the wave's scale row (gated: the gate's)

  // -------------------------------------------------------------- fragments
  // Lane l holds row l % 16 of a 16-row block, chunks l / 16 and 4 + l / 16.
  const int fr = lane & 15, fg = lane >> 4;
  const int fb0 = fr * kBK + ((fg ^ swz128(fr)) << 4);
  const int fb1 = fr * kBK + (((4 + fg) ^ swz128(fr)) << 4);
  // W fragments 0 .. 3 alternate between two sets; 4 .. 7 come first in a
  // block's last row and last in the next one's first, and need only one.
  // (With float32 scales there are only 4, in two sets.)
  v8i xf[8], wf[2][4], wl[4];
  int sx[8];
  typename std::conditional<F32, float, int>::type sw = 0, nsw = 0, psw = 0;  // of the gate, or of all columns
  typename std::conditional<F32, float, int>::type su = 0, nsu = 0, psu = 0;  // of the up projection
  auto frag = [&](const uint8_t* rows) -> v8i {
    const v4i a = *reinterpret_cast<const v4i*>(rows + fb0);
    const v4i b = *reinterpret_cast<const v4i*>(rows + fb1);
    return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  };
  // Fragment i (0 .. 7) and its rows' scales, from its half-stage.
  auto read_x = [&](const uint8_t* st, int ring, int i) {
    xf[i] = frag(st + (wm * 64 + (i & 3) * 16) * kBK);
    sx[i] = smem[C::SCALES + ring * 1024 + wave * 256 + wm * 128 + i * 16 + fr];
  };
  auto read_w = [&](const uint8_t* st, int set, int j) {
    (j < 4 ? wf[set][j & 3] : wl[j & 3]) = frag(st + C::XHALF + (wn * (BN / 4) + (j % (FN / 2)) * 16) * kBK);
  };
  f32x4 acc[8][FN];
  int one = 127;  // (opaque: not formed again right before an instruction that reads it)
  asm volatile("" : "+v"(one));

  // --------------------------------------------------------------- prologue
#pragma unroll 1
  for (int e = threadIdx.x; e < entries; e += 256) wsc[e] = wscale_at(0, e);
  auto load_all = [&](bool second) {
    begin_load(second);
    if (!second) scale_piece();
#pragma unroll
    for (int i = 0; i < C::PIECES; ++i) piece(i);
    end_load(second);
  };
  load_bias(0);
  load_all(false);
  load_all(true);
  load_all(false);
  load_all(true);
  waitvm<C::LOADED>();  // half-stages 0 and 1
  wait_lgkm0();
  barrier();
  // The first fragments, and the loads that wait for their slot.
#pragma unroll
  for (int i = 0; i < 8; ++i) read_x(smem + (i / 4) * C::HALF, 0, i);
#pragma unroll
  for (int j = 0; j < FN; ++j) read_w(smem + (j / (FN / 2)) * C::HALF, 0, j);
  sw = wsc[wrow * nb];
  if constexpr (GATED) su = wsc[nb];
  wait_lgkm0();
  barrier();
  load_all(false);

  int st = 0, ring = 0;  // of the block being computed: the slot of its first half, its scales
  // float32 weight scales: the block sums of the last instructions, and sum n
  // of half h onto its accumulators.
  f32x4 part[4];
  auto add_part = [&](int h, int n, bool first, float fg, float fu) __attribute__((always_inline)) {
    f32x4& c = acc[4 * h + n / FN][n % FN];
    const float f = GATED && n % FN >= FN / 2 ? fu : fg;
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = first ? part[n & 3][e] * f : __builtin_fmaf(part[n & 3][e], f, c[e]);
    asm volatile("" : "+v"(c));  // (here, not where the compiler would collect them)
  };
  // Half H of a block, with W set S, while the fragments of the next block
  // (block nblk of tile nit) are read.  EARLY: one of the tile's first three,
  // which read half-stages loaded before the last tile's stores.
  // FIRST: the tile's first block.  PREV: the half-block before it left block
  // sums to add (0: none, 1: of the tile's first block, 2: of another).
  auto half = [&](auto first_t, auto prev_t, auto s_t, auto h_t, auto early_t, int it, int nit,
                  int nblk) __attribute__((always_inline)) {
    constexpr int PREV = decltype(prev_t)::value;
    constexpr bool FIRST = decltype(first_t)::value;
    constexpr bool EARLY = decltype(early_t)::value;
    constexpr int S = decltype(s_t)::value, H = decltype(h_t)::value;
    const uint8_t* nx = smem + ((st + 2 + H) & 3) * C::HALF;
    const int nring = (ring + 1) & 3;
    constexpr int NI = 4 * FN;  // instructions
    for_each_index(std::make_integer_sequence<int, NI>{}, [&](auto idx_t) __attribute__((always_inline)) {
      constexpr int idx = decltype(idx_t)::value;
      if constexpr (F32) {
        constexpr int i = 4 * H + idx / FN, j = idx % FN;
        mfma_part(part[idx & 3], wf[S][j], xf[i], one, sx[i]);
      } else {
        constexpr int i = 4 * H + idx / 8, j = i == 7 ? (idx + 4) % 8 : idx % 8;
        mfma<FIRST, idx % (GATED ? 4 : 8) == 0>(acc[i][j], j < 4 ? wf[S][j & 3] : wl[j & 3], xf[i],
                                                GATED && j >= 4 ? su : sw, sx[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (idx == 3) {
        // The half-stage read here has landed once only the loads of the two
        // after it (one of them brings a block's scales) and stores behind them
        // may be in flight; every wave has read the one before it.
        if (EARLY && it > 0)
          waitvm<C::STORED>();
        else
          waitvm<C::LOADED>();
        wait_lgkm0();
        barrier();
        begin_load(H == 0);
      }
      if (idx % FN == FN - 1) read_x(nx, nring, 4 * H + idx / FN);
      if constexpr (F32) {
        if (idx == 5 || idx == 9) read_w(nx, 1 - S, 2 * H + (idx - 5) / 4);
      } else {
        if (H == 0 && idx % 8 == 4) read_w(nx, 1 - S, idx / 8);
        if (H == 1 && idx >= 24 && idx < 28) read_w(nx, 0, (idx + 4) % 8);
      }
      if (H == 1 && idx == 10) nsw = wsc[((nit & 1) * C::WROWS + wrow) * nb + nblk];
      if (GATED && H == 1 && idx == 11) nsu = wsc[((nit & 1) * C::WROWS + 1) * nb + nblk];
      if (idx > 3) {
        constexpr int slots = NI - 4;
#pragma unroll
        for (int d = 0; d < C::PIECES; ++d)
          if (idx == 4 + (2 * d + 1) * slots / (2 * C::PIECES)) piece(d);
        if (H == 1 && idx == NI - 2) scale_piece();
      }
      if constexpr (F32) {
        if (idx >= kPartLead)
          add_part(H, idx - kPartLead, FIRST, sw, su);
        else if (PREV != 0)
          add_part(1 - H, NI - kPartLead + idx, PREV == 1, H == 0 ? psw : sw, H == 0 ? psu : su);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    end_load(H == 0);
    if (H == 1) {
      st = (st + 2) & 3;
      ring = nring;
      psw = sw;
      sw = nsw;
      if constexpr (GATED) {
        psu = su;
        su = nsu;
      }
    }
  };
  using Yes = std::true_type;
  using No = std::false_type;
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;

  for (int it = 0; it < ntiles; ++it) {
    const Fp8Tile t = fp8_tile<kBM, OUTS>(p, slot + it * G);
    const bool more = it + 1 < ntiles;
    next = operands(it + 1);
    // The next tile's weight scales: fetched here, laid down after the first pair.
    const int e0 = threadIdx.x;
    WScale ws0 = 0;
    if (more && e0 < entries) ws0 = wscale_at(it + 1, e0);
    half(Yes{}, I0{}, I0{}, I0{}, Yes{}, it, it, 1);
    if (more) load_bias(it + 1);  // (behind a barrier: every wave has stored the tile before)
    half(Yes{}, I1{}, I0{}, I1{}, Yes{}, it, it, 1);
    half(No{}, I1{}, I1{}, I0{}, Yes{}, it, it, 2);
    half(No{}, I2{}, I1{}, I1{}, No{}, it, it, 2);
    if (more) {
      WScale* d = wsc + ((it + 1) & 1) * entries;
      if (e0 < entries) d[e0] = ws0;
#pragma unroll 1
      for (int e = e0 + 256; e < entries; e += 256) d[e] = wscale_at(it + 1, e);
    }
    for (int b = 2; b < nb; b += 2) {
      const bool end = b + 2 == nb;  // (past the last tile: scales that nobody uses)
      half(No{}, I2{}, I0{}, I0{}, No{}, it, it, b + 1);
      half(No{}, I2{}, I0{}, I1{}, No{}, it, it, b + 1);
      half(No{}, I2{}, I1{}, I0{}, No{}, it, it, b + 2);
      half(No{}, I2{}, I1{}, I1{}, No{}, it, end ? it + 1 : it, end ? 0 : b + 2);
      if constexpr (F32) {
        // Kept in the half of the registers where the instructions take them;
        // the compiler would carry half of them round the loop in the other,
        // at 40 copies more.  (All have arrived; fragment 7 has not.)
#pragma unroll
        for (int i = 0; i < 7; ++i) asm volatile("" : "+a"(xf[i]));
      }
    }
    mfma_settle();
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (F32) {
#pragma unroll
      for (int n = 4 * FN - kPartLead; n < 4 * FN; ++n) {
        asm volatile("" : "+v"(part[n & 3]));  // (not read before here)
        add_part(1, n, false, psw, psu);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+a"(acc[i][j]));  // (not read before here)
    }

    // Store.  Register e of block (i, j): column 16 j + 4 (lane / 16) + e, row
    // 16 i + lane % 16.  Step s: 16 rows x 64 columns go through the wave's LDS
    // area (one of two of 2 KB: 128-byte rows, chunk c of row r at slot
    // c ^ (r & 7)) and leave as whole 128-byte lines, 8 rows to a store, one
    // step later, under the next one's conversions.  (The area is the wave's
    // own: its LDS accesses stay in order.)
    // (Lane numbers are re-formed here rather than kept through the K loop.)
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int fr = lane & 15, fg = lane >> 4;
    const Fp8Params::Seg& sg = p.seg[t.seg];
    const int cols = sg.n - t.n0;
    // A resource over the tile's rows (those past M are outside it); row
    // blocks go into the scalar offset.  (ldy < kMaxLdy: see fp8_wide_wanted.)
    const int rows = p.M - t.m0 < kBM ? p.M - t.m0 : kBM;
    constexpr bool SHORT = F32 && GATED;             // 32 columns of a wave, not 64
    const int sr = SHORT ? lane >> 2 : lane >> 3;    // the lane's row and first column when it stores
    const int sc = (SHORT ? lane & 3 : lane & 7) * 8;
    struct Out {
      __amdgpu_buffer_rsrc_t r;
      unsigned off;
      int ld;
      bool whole;
    };
    auto output = [&](void* at, int64_t ld64) {
      uint16_t* y = static_cast<uint16_t*>(at);
      const int ld = int(ld64);
      return Out{buffer_rsrc(y + (int64_t)t.m0 * ld + t.n0, ((rows - 1) * ld + (cols < OUTS ? cols : OUTS)) * 2),
                 unsigned((wm * 128 + sr) * ld + wn * (OUTS / 2) + sc) * 2, ld,
                 cols >= OUTS && (ld & 7) == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0};
    };
    const Out yo = output(sg.y, sg.ldy);
    uint8_t* out = smem + C::OUT + wave * 4096;
    const uint8_t* bs = smem + C::BIAS + (it & 1) * 1024;
    auto finish = [&](f32x4 v, f32x4 bias) __attribute__((always_inline)) {
      v += bias;
      if constexpr (GELU) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = gelu_erf(v[e]);
      }
      return u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    };
    // act(gate) * up of the biased sums.
    auto gate4 = [&](f32x4 g, f32x4 u) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = (p.act == kActGelu ? gelu_erf(g[e]) : silu_rough(g[e])) * u[e];
      return g;
    };
    // 8 columns of a row, `row` and `col` from the wave's first.
    auto store = [&](auto whole_t, const Out& o, u32x4 w, int col, int row) __attribute__((always_inline)) {
      const int soff = row * o.ld * 2;
      if constexpr (decltype(whole_t)::value) {
        __builtin_amdgcn_raw_buffer_store_b128(w, o.r, o.off + col * 2, soff, kNonTemporal);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          __builtin_amdgcn_raw_buffer_store_b16(
              uint16_t(w[e / 2] >> (16 * (e & 1))), o.r,
              wn * (OUTS / 2) + col + sc + e < cols ? o.off + (col + e) * 2 : kOutOfRange, soff, 0);
      }
    };
    if constexpr (SHORT) {
      // As below, with 4 chunks of gate and 4 of up sums to a row, and one
      // store of 16 rows x 32 columns for each output.
      const f32x4* bg = reinterpret_cast<const f32x4*>(bs + (wn * (OUTS / 2) + sc) * 4);
      const f32x4* bu = reinterpret_cast<const f32x4*>(bs + (OUTS + wn * (OUTS / 2) + sc) * 4);
      const f32x4 bg0 = bg[0], bg1 = bg[1], bu0 = bu[0], bu1 = bu[1];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<f32x4*>(out + fr * 256 + (((4 * j + fg) ^ fr) << 4)) = acc[i][j];
        __builtin_amdgcn_sched_barrier(0);
        const int c = 2 * (lane & 3);
        auto sums = [&](int chunk) {
          return *reinterpret_cast<const f32x4*>(out + sr * 256 + ((chunk ^ sr) << 4));
        };
        const f32x4 g0 = sums(c) + bg0, g1 = sums(c + 1) + bg1, u0 = sums(8 + c) + bu0, u1 = sums(9 + c) + bu1;
        auto send = [&](const Out& o, f32x4 a, f32x4 b) __attribute__((always_inline)) {
          const u32x4 w = {bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3]), bf16_pair(b[0], b[1]), bf16_pair(b[2], b[3])};
          if (o.whole)
            store(Yes{}, o, w, 0, 16 * i);
          else
            store(No{}, o, w, 0, 16 * i);
        };
        send(yo, gate4(g0, u0), gate4(g1, u1));
        if constexpr (MODE == kGatedKept) {
          send(output(p.kept[0], p.ldk), g0, g1);
          send(output(p.kept[1], p.ldk), u0, u1);
        }
      }
    } else if constexpr (GATED) {
      // Step s is one output's 16 rows x 64 columns: the product's, then,
      // where they are kept, the gate's and the up projection's.
      constexpr int KINDS = MODE == kGatedKept ? 3 : 1;
      f32x4 bg[4], bu[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bg[j] = *reinterpret_cast<const f32x4*>(bs + (wn * (OUTS / 2) + 16 * j + 4 * fg) * 4);
        bu[j] = *reinterpret_cast<const f32x4*>(bs + (OUTS + wn * (OUTS / 2) + 16 * j + 4 * fg) * 4);
      }
      const Out ko[2] = {output(p.kept[0], p.ldk), output(p.kept[1], p.ldk)};
      auto store_all = [&](auto whole_t) __attribute__((always_inline)) {
        for_each_index(std::make_integer_sequence<int, 8 * KINDS + 1>{}, [&](auto s_t) __attribute__((always_inline)) {
          constexpr int s = decltype(s_t)::value;
          __builtin_amdgcn_sched_barrier(0);
          u32x4 w[2] = {};
          if (s > 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              w[k] = *reinterpret_cast<const u32x4*>(out + ((s - 1) & 1) * 2048 + (8 * k + sr) * 128 +
                                                     (((lane & 7) ^ sr) << 4));
          }
          if constexpr (s < 8 * KINDS) {
            constexpr int i = s / KINDS, kind = s % KINDS;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f32x4 g = {}, u = {};
              if (kind != 2) {
                g = acc[i][j];
                asm volatile("" : "+v"(g));  // (leaves the accumulators' half of the registers here, not earlier)
                g += bg[j];
              }
              if (kind != 1) {
                u = acc[i][4 + j];
                asm volatile("" : "+v"(u));
                u += bu[j];
              }
              const f32x4 v = kind == 0 ? gate4(g, u) : kind == 1 ? g : u;
              *reinterpret_cast<u32x2*>(out + (s & 1) * 2048 + fr * 128 + (((2 * j + (fg >> 1)) ^ (fr & 7)) << 4) +
                                        (fg & 1) * 8) = u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
            }
          }
          if (s > 0) {
            constexpr int kind = (s + KINDS - 1) % KINDS;
#pragma unroll
            for (int k = 0; k < 2; ++k)
              store(whole_t, kind == 0 ? yo : ko[kind == 1 ? 0 : 1], w[k], 0, 16 * ((s - 1) / KINDS) + 8 * k);
          }
        });
      };
      if (yo.whole && (KINDS == 1 || (ko[0].whole && ko[1].whole)))
        store_all(Yes{});
      else
        store_all(No{});
    } else if constexpr (F32) {
      // The sums themselves go through LDS (256-byte rows, chunk c of row r at
      // slot c ^ r), one step at a time, and are finished behind it: the
      // accumulators leave the epilogue few registers.
      const f32x4 bias0 = *reinterpret_cast<const f32x4*>(bs + (wn * (BN / 2) + sc) * 4);
      const f32x4 bias1 = *reinterpret_cast<const f32x4*>(bs + (wn * (BN / 2) + sc + 4) * 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<f32x4*>(out + fr * 256 + (((4 * j + fg) ^ fr) << 4)) = acc[i][j];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = 8 * k + sr, c = 2 * (lane & 7);
          const u32x2 lo = finish(*reinterpret_cast<const f32x4*>(out + r * 256 + ((c ^ r) << 4)), bias0);
          const u32x2 hi = finish(*reinterpret_cast<const f32x4*>(out + r * 256 + (((c + 1) ^ r) << 4)), bias1);
          const u32x4 w = {lo[0], lo[1], hi[0], hi[1]};
          if (yo.whole)
            store(Yes{}, yo, w, 0, 16 * i + 8 * k);
          else
            store(No{}, yo, w, 0, 16 * i + 8 * k);
        }
      }
    } else {
      f32x4 bias[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j)
        bias[j] = *reinterpret_cast<const f32x4*>(bs + (wn * (BN / 2) + 16 * j + 4 * fg) * 4);
      auto store_all = [&](auto whole_t) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s <= 16; ++s) {
          __builtin_amdgcn_sched_barrier(0);
          u32x4 w[2] = {};
          if (s > 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              w[k] = *reinterpret_cast<const u32x4*>(out + ((s - 1) & 1) * 2048 + (8 * k + sr) * 128 +
                                                     (((lane & 7) ^ sr) << 4));
          }
          if (s < 16) {
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              const int j = (4 * (s & 1) + jj) % FN;
              f32x4 v = acc[s >> 1][j];
              asm volatile("" : "+v"(v));  // (leaves the accumulators' half of the registers here, not earlier)
              *reinterpret_cast<u32x2*>(out + (s & 1) * 2048 + fr * 128 +
                                        (((2 * jj + (fg >> 1)) ^ (fr & 7)) << 4) + (fg & 1) * 8) =
                  finish(v, bias[j]);
            }
          }
          if (s > 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              store(whole_t, yo, w[k], ((s - 1) & 1) * 64, 16 * ((s - 1) >> 1) + 8 * k);
          }
        }
      };
      if (yo.whole)
        store_all(Yes{});
      else
        store_all(No{});
    }
  }
  waitvm<0>();  // no load into LDS may be in flight at the end
}

}  // namespace
}  // namespace convrot
