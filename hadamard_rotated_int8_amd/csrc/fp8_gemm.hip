// FP8 linear on CDNA4 matrix cores: E4M3 codes, a scale for each block of 128
// features.
//
//   Y[r, o] = act( sum_b sx[r, b] sw[o / 128, b] sum_{i in b} qx[r, i] qw[o, i] + bias[o] )
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies the products of a lane's 32
// features by 2^(ea + eb) as it adds them, so power-of-two (E8M0) scales cost
// no vector work: a block is two such instructions with the same scale bytes.
// float32 weight scales (checkpoints that hold max / 448) cannot go through
// the instruction: the block's sum starts from zero with the activation's
// scale applied by the matrix core, and is added to the running sum with one
// fused multiply-add per value.
//
// The FP8 instructions line up the products of 8 consecutive features by the
// largest sum e of two factors' exponents (-6 for a subnormal or a zero) and
// cut each to a multiple of 2^(e - 13); those 8, and the groups' sums onto the
// accumulator, they add to 24 bits (measured: the largest product keeps all of
// its bits, the 7 others lose less than a unit each, and a 1 survives a
// running sum of 2^23).  The result is off by 1.5e-5 of its size for normal
// data and 4e-5 where features differ much (with and without scales, the same
// for every K), and by at most 7 2^-13 of the groups' largest products where
// these cancel.  That is inside a bfloat16 output's rounding (2^-8) unless the
// output is small by cancellation, but not inside what a float32 output
// promises.  Outputs in float32 therefore convert the codes to
// bfloat16 (exact) with their scales as they leave LDS and use the bfloat16
// instruction, which adds in full float32, at half the matrix rate.
//
// The weights are the instruction's first operand: a lane then holds 4
// consecutive columns of one output row per accumulator quad and stores them
// as one vector.  Which 32 features of a 64-wide slice a lane holds does not
// matter as long as both operands agree (the sum runs over all of them and
// the scale is the block's).
#include "fp8_gemm.h"

namespace convrot {
namespace {

CR_DEVICE int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

CR_DEVICE f32x16 mfma_bf16(const Bf16Frag& a, const Bf16Frag& b, f32x16 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

// One workgroup per output tile.  KG groups of WM x WN waves share the blocks
// of features in turn, each with a ring of stages of its own, and their sums
// meet in LDS at the end, in the groups' order; a wave owns FM x FN blocks of
// 32 x 32.  Operands reach LDS by direct-to-LDS loads of whole 128-byte lines
// (16-byte chunk c of stage row r at slot c ^ swz(r), so 16 lanes that read 16
// consecutive rows touch 16 different groups of 4 banks), STAGES - 1 stages
// ahead of the products.  Rows past M or n and bytes past K read as zero
// (range check of the buffer resource).  The activation's scale bytes of a
// step's block lie side by side and come along as one load (every wave makes
// its own copy, so that all have the same number of loads to wait for); the
// weights' scales of the whole tile are laid out in LDS as 32-bit values first.
// EXACT: bfloat16 instructions, for float32 outputs (the others are bfloat16).
//
// GATED: of the BN rows of W in a tile every 32 are 16 of the gate's and the
// same 16 of the up projection's.  A lane then holds both sums of 8 of its 16
// columns of a 32 x 32 block, and the tile gives BN / 2 columns of
// act(gate) * up.
template <int FM, int FN, int WM, int WN, int KG, int STAGES, bool F32SCALE, bool EXACT, bool GATED>
__global__ __launch_bounds__(WM* WN* KG * 64) void fp8_gemm_kernel(const Fp8Params p) {
  constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN, WAVES = WM * WN;
  constexpr int XB = BM * kBK, WB = BN * kBK;
  constexpr int STAGE = XB + WB + WAVES * 256;  // + the rows' scales, a copy for each wave
  constexpr int PIECES = (XB + WB) / 1024;  // 1 KB: 8 rows
  constexpr int OUTS = GATED ? BN / 2 : BN;  // columns of Y
  // Weight scale rows of a tile (gated: the gate's, the up projection's).
  constexpr int NBW = GATED ? 2 : BN > kFp8Block ? BN / kFp8Block : 1;
  static_assert(!GATED || OUTS <= kFp8Block, "one scale row each");
  constexpr int LOADS = PIECES / WAVES + 1;  // of a wave and stage
  // The fragments come before the next loads, or after them where four waves
  // to a SIMD have others to hide behind: 333 x 4112 -> 4096 float32 (eight
  // waves) 23.3 us against 25.6, 256 x 5120 -> 13824 (sixteen) 33.3 and 28.7.
  constexpr bool LOADS_FIRST = KG * WAVES >= 16;
  static_assert(STAGES >= 2 && (STAGES - 2) * LOADS <= kVmMax, "vmcnt range");
  static_assert(KG == 1 || (KG - 1) * BM * BN * 4 <= KG * STAGES * STAGE, "the groups' sums fit");
  static_assert(KG * STAGES * STAGE + BN * 4 + NBW * (kMaxBlocks + KG) * 4 <= 160 * 1024, "LDS");
  static_assert(BM <= 256 && PIECES % WAVES == 0, "one load of scales, the others split evenly");
  static_assert(kFp8Block % (32 * FN) == 0 || (32 * FN) % kFp8Block == 0, "blocks in one scale row");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  float* bias = reinterpret_cast<float*>(smem + KG * STAGES * STAGE);  // [BN]
  unsigned* wscale = reinterpret_cast<unsigned*>(bias + BN);              // [NBW][kbp]

  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wid / WAVES, wave = wid % WAVES;
  uint8_t* ring = smem + group * STAGES * STAGE;
  const int wm = wave / WN, wn = wave % WN;
  const int K = p.K, kb = p.kb, kbp = kb + KG - 1;  // (the last turn's blocks)
  const Fp8Tile tile = fp8_tile<BM, OUTS>(p, p.first + xcd_slot(blockIdx.x, gridDim.x));
  const Fp8Params::Seg& sg = p.seg[GATED ? 0 : tile.seg];
  const int m0 = tile.m0, n0 = tile.n0;
  const int rows = p.M - m0 < BM ? p.M - m0 : BM;
  const int cols = sg.n - n0 < OUTS ? sg.n - n0 : OUTS;
  const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(p.qx + (int64_t)m0 * K, rows * K);
  static_assert(!GATED || (XB / 1024 % 4 == 0 && (WAVES < 4 || WAVES % 4 == 0)), "whose a piece is");
  const uint8_t* uw = GATED ? p.seg[1].qw : sg.qw;
  const __amdgpu_buffer_rsrc_t ur = buffer_rsrc(uw + (int64_t)n0 * K, cols * K);
  const __amdgpu_buffer_rsrc_t wr =
      buffer_rsrc((GATED && WAVES >= 4 && (wave & 2) ? uw : sg.qw) + (int64_t)n0 * K, cols * K);

  // Past the last block everything is out of range: the loads keep their
  // number, for the waits.
  auto issue = [&](int turn, int slot) {
    uint8_t* st = ring + slot * STAGE;
    const int step = turn * KG + group;
    const int k0 = step * kBK;
    // (An ordinary loop: behind one over constants the compiler asks for the
    // fifth and sixth fragment only after the wait for the third and fourth, which
    // shows where the weights lie in the caches: 48 x 5120 -> 13824 float32 17.2 us
    // instead of 16.6, 256 x 4096 -> 4096 13.9 and 13.5.
    // tests/test_fragment_reads.py has the built code.)
#pragma unroll
    for (int i = 0; i < PIECES / WAVES; ++i) {
      const int q = wave + WAVES * i;
      const bool is_x = q < XB / 1024;
      const int row = (is_x ? q : q - XB / 1024) * 8 + lane / 8;
      const int kc = k0 + ((lane & 7) ^ swz(row)) * 16;
      const int from = GATED && !is_x ? (row >> 5) * 16 + (row & 15) : row;  // of the operand
      const unsigned off = kc < K ? unsigned(from * K + kc) : kOutOfRange;
      // (Pieces 4 n + 2 and 4 n + 3 are the up projection's: known here, or the same for all of a wave's.)
      const bool up = GATED && WAVES < 4 && ((WAVES * i) & 2);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_x ? xr : up ? ur : wr, (lds_void*)(st + q * 1024), 16, off, 0, 0, 0);
    }
    // (the scales' rows are padded to a multiple of 4)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        buffer_rsrc(p.sx + step * p.lds + m0, step < kb ? (rows + 3) & ~3 : 0),
        (lds_void*)(st + XB + WB + wave * 256), 4, lane * 4, 0, 0, 0);
  };

  // (before the first wait: the loads' way is long)
#pragma unroll
  for (int t = 0; t < STAGES - 1; ++t) issue(t, t);
  {  // the tile's weight scales (rows past n, blocks past K: one) and bias
    const int first_row = n0 / kFp8Block, nrows = (sg.n + kFp8Block - 1) / kFp8Block;
    for (int i = threadIdx.x; i < NBW * kbp; i += KG * WAVES * 64) {
      const int r = first_row + (GATED ? 0 : i / kbp), b = i % kbp;
      const void* sw = GATED && i >= kbp ? p.seg[1].sw : sg.sw;
      const int64_t at = (int64_t)r * kb + b;
      unsigned v = F32SCALE ? __float_as_uint(1.f) : 127u;
      if (r < nrows && b < kb)
        v = F32SCALE ? static_cast<const unsigned*>(sw)[at] : static_cast<const uint8_t*>(sw)[at];
      wscale[i] = v;
    }
    for (int i = threadIdx.x; i < BN; i += KG * WAVES * 64) {
      const int c = i % OUTS;
      const float* b = GATED && i >= OUTS ? p.seg[1].bias : sg.bias;
      bias[i] = b && c < cols ? b[n0 + c] : 0.f;
    }
  }

  const int fr = lane & 31, fh = lane >> 5;
  f32x16 acc[FM][FN] = {};
  auto frag = [&](const uint8_t* base, int row, int t2) -> v8i {
    const v4i a = *reinterpret_cast<const v4i*>(base + row * kBK + (((4 * t2 + fh) ^ swz(row)) << 4));
    const v4i b = *reinterpret_cast<const v4i*>(base + row * kBK + (((4 * t2 + 2 + fh) ^ swz(row)) << 4));
    return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  };
  for (int turn = 0, slot = 0; turn * KG < kb; ++turn) {
    const int step = turn * KG + group;
    // This step's stage has landed once only those behind it may be in
    // flight; every wave has read the one before it, which is refilled.
    waitvm<(STAGES - 2) * LOADS>();
    wait_lgkm0();
    barrier();
    if constexpr (LOADS_FIRST) issue(turn + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1);
    const uint8_t* st = ring + slot * STAGE;
    // All of the step's fragments are requested before the first is used.
    int sx[FM];
    unsigned sw[FN], su[FN];  // (su: the up projection's float32 scale)
    v8i xf[2][FM], wf[2][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) sx[i] = st[XB + WB + wave * 256 + wm * FM * 32 + i * 32 + fr];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      // Of a gated block the first operand's rows 16 .. 31, lanes like rows, are the up projection's.
      sw[j] = wscale[(GATED ? (!F32SCALE && (lane & 16) ? 1 : 0) : (wn * FN * 32 + j * 32) / kFp8Block) * kbp + step];
      if (GATED && F32SCALE) su[j] = wscale[kbp + step];
    }
    auto block_scale = [&](int j, int e) {  // float32, of element e of block j
      return __uint_as_float(GATED && e >= 8 ? su[j] : sw[j]);
    };
#pragma unroll
    for (int t2 = 0; t2 < 2; ++t2) {
#pragma unroll
      for (int i = 0; i < FM; ++i) xf[t2][i] = frag(st, wm * FM * 32 + i * 32 + fr, t2);
#pragma unroll
      for (int j = 0; j < FN; ++j) wf[t2][j] = frag(st + XB, wn * FN * 32 + j * 32 + fr, t2);
    }
    if constexpr (!LOADS_FIRST) issue(turn + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1);
    slot = slot + 1 == STAGES ? 0 : slot + 1;
    if constexpr (EXACT) {
      // Power-of-two scales ride on the conversion; a float32 weight scale is
      // applied to the block's sum.
      f32x16 part[FM][FN];
      if constexpr (F32SCALE) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) part[i][j] = f32x16{};
      }
#pragma unroll
      for (int t2 = 0; t2 < 2; ++t2) {
        Bf16Frag xb[FM], wb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) xb[i] = to_bf16(xf[t2][i], e8m0_value(sx[i]));
#pragma unroll
        for (int j = 0; j < FN; ++j) wb[j] = to_bf16(wf[t2][j], F32SCALE ? 1.f : e8m0_value(sw[j]));
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            f32x16& c = F32SCALE ? part[i][j] : acc[i][j];
            c = mfma_bf16(wb[j], xb[i], c);
          }
      }
      if constexpr (F32SCALE) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              acc[i][j][e] = __builtin_fmaf(part[i][j][e], block_scale(j, e), acc[i][j][e]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          f32x16 c = F32SCALE ? f32x16{} : acc[i][j];
          const int s = F32SCALE ? 127 : int(sw[j]);
#pragma unroll
          for (int t2 = 0; t2 < 2; ++t2)
            c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wf[t2][j], xf[t2][i], c, 0, 0, 0, s, 0, sx[i]);
          if constexpr (F32SCALE) {
#pragma unroll
            for (int e = 0; e < 16; ++e) c[e] = __builtin_fmaf(c[e], block_scale(j, e), acc[i][j][e]);
          }
          acc[i][j] = c;
        }
    }
  }
  waitvm<0>();  // no load into LDS may be in flight at the end
  if constexpr (KG > 1) {  // the groups' sums, in their order
    wait_lgkm0();
    barrier();
    f32x4* sums = reinterpret_cast<f32x4*>(smem);
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sums[(((group - 1) * WAVES + wave) * FM * FN * 4 + (i * FN + j) * 4 + q) * 64 + lane] =
                f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    }
    wait_lgkm0();
    barrier();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < KG; ++g)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 v = sums[(((g - 1) * WAVES + wave) * FM * FN * 4 + (i * FN + j) * 4 + q) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
          }
  }
  // Register e of block (i, j): column 8 (e / 4) + 4 (lane / 32) + e % 4, row lane % 32.
  const GatedOut out = gated_out(p);
  const int64_t ldy = sg.ldy;
  const bool vec = (ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(sg.y) & (p.y_bf16 ? 7 : 15)) == 0;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int m = m0 + wm * FM * 32 + i * 32 + fr;
    if constexpr (GATED) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int c = (wn * FN + j) * 16 + 8 * q + 4 * fh, n = n0 + c;
          float g[4], u[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            g[e] = acc[i][j][4 * q + e] + bias[c + e];
            u[e] = acc[i][j][8 + 4 * q + e] + bias[OUTS + c + e];
          }
          if (m < p.M && n < sg.n) store_gated4<!EXACT>(out, m, n, g, u);
        }
    } else {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = n0 + wn * FN * 32 + j * 32 + 8 * q + 4 * fh;
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = acc[i][j][4 * q + e] + bias[n - n0 + e];
            if (p.gelu) v[e] = gelu_erf(v[e]);
          }
          if (m < p.M && n < sg.n)
            store4(sg.y, (int64_t)m * ldy + n, v, sg.n - n, p.y_bf16, vec && sg.n - n >= 4);
        }
    }
  }
}

template <int FM, int FN, int WM, int WN, int KG, int STAGES, bool F32SCALE, bool EXACT, bool GATED>
hipError_t launch_g(const Fp8GemmArgs& a, hipStream_t stream) {
  constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
  constexpr int NBW = GATED ? 2 : BN > kFp8Block ? BN / kFp8Block : 1;
  Fp8Params p = fp8_params<BM, BN>(a);
  const size_t lds = KG * STAGES * ((BM + BN) * kBK + WM * WN * 256) + BN * 4 + size_t(NBW) * (p.kb + KG - 1) * 4;
  constexpr int kThreads = WM * WN * KG * 64;
  in_launches(int64_t(p.tiles_m) * p.tiles_n, kThreads, [&](int64_t first, unsigned count) {
    p.first = int(first);
    hipLaunchKernelGGL((fp8_gemm_kernel<FM, FN, WM, WN, KG, STAGES, F32SCALE, EXACT, GATED>), dim3(count),
                       dim3(kThreads), lds, stream, p);
  });
  return hipGetLastError();
}

enum { kLinears = 1, kPairs = 2 };  // what a shape is for

template <int FM, int FN, int WM, int WN, int KG, int STAGES, bool F32SCALE, bool EXACT, int FOR>
hipError_t launch_t(const Fp8GemmArgs& a, hipStream_t stream) {
  if constexpr (FOR == kLinears)
    return launch_g<FM, FN, WM, WN, KG, STAGES, F32SCALE, EXACT, false>(a, stream);
  else if constexpr (FOR == kPairs)
    return launch_g<FM, FN, WM, WN, KG, STAGES, F32SCALE, EXACT, true>(a, stream);
  else
    return a.gated ? launch_g<FM, FN, WM, WN, KG, STAGES, F32SCALE, EXACT, true>(a, stream)
                   : launch_g<FM, FN, WM, WN, KG, STAGES, F32SCALE, EXACT, false>(a, stream);
}

template <int FM, int FN, int WM, int WN, int KG, int STAGES, bool EXACT, int FOR = kLinears | kPairs>
hipError_t launch_type(const Fp8GemmArgs& a, hipStream_t stream) {
  return a.f32_scale ? launch_t<FM, FN, WM, WN, KG, STAGES, true, EXACT, FOR>(a, stream)
                     : launch_t<FM, FN, WM, WN, KG, STAGES, false, EXACT, FOR>(a, stream);
}

template <int FM, int FN, int WM, int WN, int KG, int STAGES>
hipError_t launch_modes(const Fp8GemmArgs& a, hipStream_t stream) {
  return a.y_bf16 ? launch_type<FM, FN, WM, WN, KG, STAGES, false>(a, stream)
                  : launch_type<FM, FN, WM, WN, KG, STAGES, true>(a, stream);
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t stream) {
  if (fp8_wide_wanted(a)) return a.gated ? launch_fp8_gated_wide(a, stream) : launch_fp8_gemm_wide(a, stream);
  // What bounds few tiles is the latency of a step's loads, barrier and
  // fragments, some 0.3 us however little they bring, and that a CU has only
  // so many loads under way: so tiles as small as the CUs still take one of
  // each, with the blocks of features shared among groups of waves.  Beyond
  // one tile of 128 x 128 for each CU, and for up to 64 rows beyond one of
  // 64 x 64, two workgroups to a CU cover each other's waits instead.
  // Measured (us, in a graph; bfloat16 outputs | float32 outputs), tiles of
  //                        32x32     32x64 64x64 64x64 | 32x32     32x64 64x64 64x64
  //   in groups             4    8    4     2     1    |  4    8    4     2     1
  //   33 x  4096 ->  4096   7.3  7.6  8.2   9.6  11.8  |  8.5  7.8  9.6  13.4  17.8
  //   16 x 13824 ->  5120  15.2 18.3 17.7  23.1  32.2  | 18.6 18.4 21.7  36.3  50.0
  //   64 x 13824 ->  5120  27.1 33.9 19.3  25.8  32.5  | 34.4 34.4 23.4  36.1  50.0
  //   64 x  5120 -> 13824  29.1 32.4 20.6  15.3  16.8  | 33.2 32.6 22.9  17.8  22.6
  //   64 x  5120 -> 20480  35.9 40.2 29.8  28.2  25.4  | 40.7 40.6 33.0  32.2  29.6
  // and
  //                        64x64 64x128 128x128 128x64 128x128 | the same
  //   in groups             1     1      1       2      2
  //   300 x  4096 ->  4096 16.2  25.3   24.5    14.4   19.0    | 25.0 26.5 35.1 20.6 29.3
  //   512 x  4096 ->  4096 17.6  25.2   30.3    15.4   20.2    | 26.5 27.9 40.1 22.0 30.2
  //   200 x 13824 ->  5120 37.0  67.1   85.3    35.2   52.2    | 69.3 72.7  117 52.2 82.5
  //   256 x  5120 -> 13824 38.6  32.6   41.0    34.2   28.3    | 54.0 44.4 53.7 45.2 39.3
  //  1000 x  4096 ->  4096 29.7  27.0   32.3    27.5   22.9    | 44.7 38.0 42.7 39.2 35.4
  //  2048 x  4096 ->  4096 53.4  53.7   38.2    52.0   42.5    | 82.3 69.3 61.7 76.3 67.1
  //    64 x  4096 -> 100000 103   129    122     123    130    |  106  114  120  133  129
  // (Eight groups need a stage less, which costs more than they gain where
  // the products are quick, with bfloat16 outputs.)
  auto tiles = [&](int64_t bm, int64_t bn) {
    int64_t t = 0;  // (a gated pair's columns of W come 16 and 16)
    for (int i = 0; i < a.count; ++i) t += (a.w[i].n + bn - 1) / bn;
    if (a.gated) t = (a.w[0].n + bn / 2 - 1) / (bn / 2);
    return t * ((a.m + bm - 1) / bm);
  };
  const int64_t cus = device_cu_count();
  if (tiles(32, 32) <= cus) {
    if (a.y_bf16) return launch_type<1, 1, 1, 1, 4, 3, false>(a, stream);
    return launch_type<1, 1, 1, 1, 8, 2, true>(a, stream);
  }
  if (tiles(32, 64) <= cus) return launch_modes<1, 1, 1, 2, 4, 3>(a, stream);
  if (tiles(64, 64) <= cus) return launch_modes<1, 1, 2, 2, 2, 3>(a, stream);
  if (a.m <= 64) return launch_modes<1, 1, 2, 2, 1, 3>(a, stream);
  if (tiles(128, 64) <= cus) return launch_modes<2, 1, 2, 2, 2, 3>(a, stream);
  if (tiles(128, 128) <= cus) {
    if (!a.y_bf16) return launch_type<1, 2, 4, 2, 2, 2, true>(a, stream);
    // A pair with bfloat16 outputs has one group of waves and four stages,
    // whose loads are longer under way: weights from memory, 128 x 5120 ->
    // 13824, 256 x 5120 -> 8192, 333 x 4112 -> 4104: 43, 39 and 35 us, in two
    // groups 47, 44 and 38.  (float32 outputs wait for the matrix cores: 512 x
    // 5120 -> 4096 54 and 51.)
    if (a.gated) return launch_type<2, 1, 2, 4, 1, 4, false, kPairs>(a, stream);
    return launch_type<1, 2, 4, 2, 2, 2, false, kLinears>(a, stream);
  }
  return launch_modes<2, 2, 2, 2, 1, 2>(a, stream);
}

}  // namespace convrot
