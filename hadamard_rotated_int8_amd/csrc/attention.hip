// Attention of m queries to l keys, softmax(scale Q K^T) V, on CDNA4 matrix
// cores: one pass over the keys with a running maximum and sum.
//
// A wave holds the transposed scores S^T = K Q^T of 32 queries: a lane then
// has 16 keys of one query in registers, its maximum takes one exchange with
// the other half of the wave, and the 8 values it holds of 16 keys are as they
// stand the second operand of O^T = V^T P^T (both operands of a product may
// name its 16 terms in any order, as long as it is the same).  V^T is read
// from LDS with the transposing read, so K and V lie there as they come.
//
// With many keys power binds it, and how products and vector instructions share
// the cycles that it leaves: 4095 x 32760, 40 heads of 128, takes 2500 to 2650
// us, 1.04 to 1.1 PFLOP/s (a large library product 1.36), at 1.72 of 2.4 GHz,
// with the matrix cores busy in 58 % of the cycles, vector instructions issued
// in 54 % and waves waiting in 25 % of theirs.  With few keys the workgroups'
// starts and ends come to as much: 32760 x 512 440 us, 0.78 PFLOP/s, matrix
// cores busy in 39 %; 3 x 1023 x 333, 32 heads of 80 on 8, with a mask, 29 us,
// five tiles of keys to a workgroup.  One query over 512 keys, 40 heads: 10.6 us,
// the steps' and loads' latency.
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
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
typedef __attribute__((address_space(3))) uint8_t lds_byte;

constexpr float kLog2e = 1.44269504f;
constexpr float kSlack = 8.f;  // powers of two that a weight may exceed 1 by
constexpr float kMinusInf = -__builtin_inff();
constexpr float kLowest = -3.40282347e38f;

// Bytes of a key's or value's row in LDS.
constexpr int row_pitch(int d) { return d <= 64 ? 128 : d <= 128 ? 256 : 512; }

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

// 16 bytes for each lane from `base` + place + soff to LDS, lane by lane from
// `to` on; zeros where place lies outside the first `bytes`.  As inline
// assembly, since the compiler drains every direct-to-LDS load that it knows
// of before it lets a transposing read pass, and the loads for later tiles are
// to stay in flight.  It has no register to write; the waits that its data
// need are waitvm's, before a barrier.  (Nothing else in these kernels uses m0.)
CR_DEVICE void load_to_lds(const void* base, unsigned bytes, unsigned place, int soff, unsigned to) {
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  const u32x4 resource = {unsigned(at), unsigned(at >> 32) & 0xFFFFu, bytes, unsigned(kBufferWord3)};
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(to), "v"(place), "s"(resource), "s"(soff)
               : "memory");
}

// One product onto (FIRST: from `start` into) its accumulators.  As inline
// assembly, so that sums stay in their registers: the compiler, free to choose
// others, gives the output's sums two sets round the loop and spills.  It does
// not see that these are matrix instructions: an operand that a vector
// instruction may have written right before takes 2 wait states, results are
// touched 18 later (mfma_settle, or two more products).
// tests/test_attention_hazards.py checks the built code for both.  ACC: Q and
// the output's sums are in the accumulation half of the registers, where a wave
// has all of them.
template <bool FIRST, bool ACC>
CR_DEVICE void scores_mfma(f32x16& s, bf16x8 k, bf16x8 q, const f32x16& start) {
  if constexpr (FIRST && ACC)
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %3" : "=&v"(s) : "v"(k), "a"(q), "v"(start));
  else if constexpr (FIRST)
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %3" : "=&v"(s) : "v"(k), "v"(q), "v"(start));
  else if constexpr (ACC)
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(s) : "v"(k), "a"(q));
  else
    asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(s) : "v"(k), "v"(q));
}
template <bool ACC>
CR_DEVICE void output_mfma(f32x16& o, bf16x8 v, bf16x8 p) {
  if constexpr (ACC)
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(o) : "v"(v), "v"(p));
  else
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(o) : "v"(v), "v"(p));
}
template <bool ACC>
CR_DEVICE void mfma_settle(f32x16& o) {
  if constexpr (ACC)
    asm volatile("" : "+a"(o));
  else
    asm volatile("" : "+v"(o));
}

CR_DEVICE float other_half(float v) {  // lane ^ 32
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// Bit i: byte i of the four is not 0.
CR_DEVICE unsigned byte_bits(unsigned w) {
  const unsigned t = (((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | w) >> 7 & 0x01010101u;
  return t * 0x01020408u >> 24;
}

// Waves of a workgroup; two tiles of 32 keys for each fill LDS.
constexpr int attention_waves(int d, bool few) { return few && d > 128 ? 2 : 4; }

// D: the head's features rounded up to 32.  MASK: keys are hidden one by one,
// not only from a length on.
//
// A wave has 32 queries.  Keys go in blocks of 32; step t multiplies Q with
// block t + 1 and the weights of block t - 1 with its values, D / 8
// instructions of 32 cycles, one of each in turn, and turns the scores of block
// t into weights between them.  K's and V's fragments are read 4 ahead, across
// steps.
//
// The weights are powers of two relative to a base that follows the maximum
// only when that has risen by more than kSlack powers of two, which no other
// block after the first few does: float32 sums and bfloat16 weights have the
// same relative precision at 256 as at 1.  So a step takes the base as it is,
// finds the maximum beside it, and if that has risen too far does its weights
// again at the end.
//
// Tiles of kKeys keys lie in a ring of areas in LDS; a wave goes through a tile
// in two steps.  FEW: of a workgroup's waves each takes its own block of every
// tile, in one step, for the same 32 queries, and their sums meet in LDS.
template <int D, bool FEW, bool MASK>
__global__ __launch_bounds__(attention_waves(D, FEW) * 64, D <= 128 && !FEW ? 2 : 1) void attention_kernel(
    const AttentionArgs p) {
  constexpr int kWaves = attention_waves(D, FEW);
  constexpr int kPitch = row_pitch(D);        // bytes of a row in LDS
  constexpr int kChunks = kPitch / 16;
  constexpr int kRowsPiece = 1024 / kPitch;   // rows that one load instruction of a wave brings
  constexpr int kKeys = FEW ? 32 * kWaves : 64;
  constexpr int kTile = kKeys * kPitch;       // bytes of K, or of V
  constexpr int kPieces = kTile / 1024 / kWaves;
  constexpr int kRows = FEW ? 32 : kWaves * 32;  // queries of a workgroup
  constexpr bool kAcc = D > 128 || FEW;       // (see scores_mfma)
  constexpr int kRing = 2 * kTile * 3 <= 48 * 1024 ? 3 : 2;
  constexpr int KF = D / 16, NF = D / 32;     // fragments of 32 keys of K; blocks of 32 features of V
  constexpr int kSlots = 2 * KF;              // matrix instructions of a step
  constexpr int kAhead = KF % 4 == 0 ? 4 : KF / 2;  // fragments read ahead (the next step takes the same registers)
  constexpr int kLag = FEW ? 2 : 1;           // tiles that an area's V is behind its K
  static_assert(kRing * 2 * kTile <= 160 * 1024 && (!FEW || kWaves * 32 * (D + 4) * 4 <= kRing * 2 * kTile), "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kRing * 2 * kTile];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 31, fh = lane >> 5;
  // Neighbouring workgroups of an XCD share a head's keys.
  // The keys of tiles from p.whole on (a multiple of the XCDs) are split.
  int slot, split = 0, splits = 1;
  if (p.splits == 1 || int(blockIdx.x) < p.whole) {
    slot = int(p.first) + xcd_slot(blockIdx.x, p.splits == 1 ? gridDim.x : p.whole);
  } else {
    splits = p.splits;
    slot = xcd_slot(blockIdx.x - p.whole, gridDim.x - p.whole);
    split = slot % splits;
    slot = p.whole + slot / splits;
  }
  // The first of the tile's rows among the parts of its split.
  const int64_t part0 = (int64_t(split) * (p.batch * p.kv_heads * p.tiles - p.whole) + slot - p.whole) * (FEW ? 32 : kWaves * 32);
  const int tile = slot % p.tiles;
  slot /= p.tiles;
  const int head = slot % p.kv_heads, batch = slot / p.kv_heads;
  const int64_t rows = p.m * p.ratio;  // a key head's queries, (token, query head)
  const int64_t row0 = int64_t(tile) * kRows + (FEW ? 0 : wave * 32);
  const int own = FEW ? wave * 32 : 0;  // first row of a tile that the wave reads

  int keys = int(p.l);
  if (p.lengths) {
    const int n = p.lengths[batch];
    keys = n < 0 ? 0 : n < keys ? n : keys;
  }
  const int64_t all = (int64_t(keys) + kKeys - 1) / kKeys;  // tiles of keys
  const int first = int(all * split / splits);
  int last = int(all * (split + 1) / splits);
  const uint16_t* kbase = p.k + batch * p.ks[0] + head * p.ks[2];
  const uint16_t* vbase = p.v + batch * p.vs[0] + head * p.vs[2];
  const int dbytes = p.d * 2;

  // MASK: a bit for each key of 64 blocks of 32 from block `window` on, a word in
  // each lane; read anew where a tile's step needs words behind them.  (2 x 4096
  // x 77, 10 heads of 64: 12.4 us with a mask, 11.4 without; 4096 x 4096, 16 of
  // 128, no two blocks hiding the same keys: 147 and 140.  As scalar loads from
  // words that another kernel made 18.7 and 203, and 3.8 for that.)
  unsigned seen = 0;
  int window = first * (kKeys / 32);
  auto mask_words = [&](int block) __attribute__((always_inline)) {
    const uint8_t* row = p.mask + batch * p.mask_stride;
    const unsigned at = unsigned(block + lane) * 32;
    unsigned bits = 0;
    if (p.l >= 32) {  // (32 keys up to the last one and what is in front of `at` shifted out)
      const unsigned end = unsigned(p.l) - 32, from = at < end ? at : end;
      unsigned w[8];
      __builtin_memcpy(w, row + from, 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) bits |= byte_bits(w[i]) << (4 * i);
      bits = at - from < 32 ? bits >> (at - from) : 0u;
    } else {  // (a byte to a lane)
      bits = unsigned(__ballot(lane < p.l && row[lane < p.l ? lane : 0] != 0));
    }
    return bits;
  };
  auto move_window = [&](int t) __attribute__((always_inline)) {  // for tile t and those that its step loads
    if (MASK && (t + kRing + 1) * (kKeys / 32) - window > 64) {
      window = t * (kKeys / 32);
      seen = mask_words(window);
    }
  };
  if (MASK && first < last) {
    seen = mask_words(window);
    // Without a key that is seen there is nothing to do (a NaN or infinity of a
    // query times the zeros of hidden keys would be a NaN).
    const unsigned blocks = last * (kKeys / 32), end = unsigned(last) * kKeys < unsigned(keys) ? last * kKeys : keys;
    auto none = [&](unsigned bits, int block) {
      const unsigned at = unsigned(block + lane) * 32, left = at < end ? end - at : 0;
      return __ballot((left < 32 ? bits & ((1u << left) - 1) : bits) != 0) == 0;
    };
    if (none(seen, window)) {
      unsigned b = window + 64;
      while (b < blocks && none(mask_words(b), b)) b += 64;
      if (b >= blocks) last = first;
    }
  }
  auto block_word = [&](int t, int row) __attribute__((always_inline)) {
    return unsigned(__builtin_amdgcn_readlane(seen, t * (kKeys / 32) + row / 32 - window));
  };

  // The keys of block `row` / 32 of tile t that take part, one bit for each;
  // none behind the last.
  auto block_bits = [&](int t, int row) -> unsigned {
    const int left = t >= last ? 0 : keys - t * kKeys - row;
    unsigned bits = unsigned((uint64_t(1) << (left < 0 ? 0 : left < 32 ? left : 32)) - 1);
    if (MASK) bits &= block_word(t, row);
    return bits;
  };
  // Rows of K (of tile t) and V (of the tile kLag before) into LDS area `to`, in
  // pieces of 1 KB; hidden and absent ones read as zero: a score is then what
  // its accumulator starts from, and a NaN of a hidden value does not meet its
  // weight of zero.  (Rows behind the last key lie outside the resource: a
  // token's stride is 0 or holds the row.)  A wave's piece i is kStep i rows
  // behind its first; where those are no multiples of 16, K's chunks change places.
  constexpr int kStep = kWaves * kRowsPiece;
  constexpr int kPlaces = kStep >= 16 ? 1 : 16 / kStep;
  static_assert(kStep % 4 == 0 && (kStep % 64 == 0 || 64 % kStep == 0), "places");
  const int prow = wave * kRowsPiece + lane / kChunks;
  unsigned kplace[kPlaces], vplace;
#pragma unroll
  for (int i = 0; i < kPlaces; ++i) {
    const int c = (lane % kChunks ^ key_swizzle<kPitch>(prow + i * kStep)) * 16;
    kplace[i] = c < dbytes ? unsigned(prow * int(p.ks[1]) * 2 + c) : kOutOfRange;
  }
  {
    const int c = (lane % kChunks ^ value_swizzle<kPitch>(prow)) * 16;
    vplace = c < dbytes ? unsigned(prow * int(p.vs[1]) * 2 + c) : kOutOfRange;
  }
  struct {
    const uint16_t *k, *v;
    unsigned kbytes, vbytes;
    unsigned to;
    uint64_t kseen[kKeys / 64], vseen[kKeys / 64];  // (with a mask)
  } load;
  auto bytes_of = [&](int t, int64_t stride) -> unsigned {  // of tile t's rows, up to the last key
    const int left = t < first || t >= last ? 0 : keys - t * kKeys;
    return left <= 0 ? 0 : (left < kKeys ? unsigned(left) - 1 : kKeys - 1) * unsigned(stride) * 2 + dbytes;
  };
  auto begin_load = [&](int t, int to) __attribute__((always_inline)) {
    load.k = kbase + int64_t(t) * kKeys * p.ks[1];
    load.v = vbase + int64_t(t - kLag) * kKeys * p.vs[1];
    load.kbytes = bytes_of(t, p.ks[1]);
    load.vbytes = bytes_of(t - kLag, p.vs[1]);
    load.to = unsigned(reinterpret_cast<uintptr_t>((lds_byte*)smem)) + to * 2 * kTile + wave * 1024;
    if constexpr (MASK) {  // (whatever it says of tiles that are not there)
#pragma unroll
      for (int w = 0; w < kKeys / 64; ++w) {
        load.kseen[w] = block_word(t, 64 * w) | uint64_t(block_word(t, 64 * w + 32)) << 32;
        load.vseen[w] = block_word(t - kLag, 64 * w) | uint64_t(block_word(t - kLag, 64 * w + 32)) << 32;
      }
    }
  };
  auto piece = [&](int j) __attribute__((always_inline)) {  // K's, then V's
    const bool v = j >= kPieces;
    const int i = v ? j - kPieces : j;
    unsigned at = v ? vplace : kplace[i % kPlaces];
    if constexpr (MASK) {
      // (the wave's rows of the piece are neighbours: its first one's bit, then the lane's)
      const uint64_t rows = (v ? load.vseen : load.kseen)[i * kStep / 64];
      const unsigned hidden = unsigned(~rows >> ((wave * kRowsPiece + i * kStep) % 64));
      at |= hidden << (31 - lane / kChunks) & kOutOfRange;
    }
    load_to_lds(v ? load.v : load.k, v ? load.vbytes : load.kbytes, at, i * kStep * int(v ? p.vs[1] : p.ks[1]) * 2,
                load.to + (v ? kTile : 0) + i * kWaves * 1024);
  };

  // Q: lane l holds query l % 32, features 16 t + 8 (l / 32) .. +7.
  bf16x8 qf[KF];
  {
    const int64_t r = row0 + fr;
    const int64_t token = p.ratio == 1 ? r : int64_t(unsigned(r) / unsigned(p.ratio));  // (rows are below 2^31)
    const int64_t j = r - token * p.ratio;
    const uint16_t* src = p.q + batch * p.qs[0] + token * p.qs[1] + (head * p.ratio + j) * p.qs[2];
#pragma unroll
    for (int t = 0; t < KF; ++t) {
      const int f = 16 * t + 8 * fh;
      qf[t] = r < rows && f < p.d ? *reinterpret_cast<const bf16x8*>(src + f) : bf16x8{};
    }
  }
  if constexpr (kAcc) {  // (into the accumulation half, where the products take them)
#pragma unroll
    for (int t = 0; t < KF; ++t) asm volatile("" : "+a"(qf[t]));
  }
  // Tile u's area holds K of tile u and V of tile u - kLag: what the steps that
  // make the scores of tile u read.
  constexpr int kLoads = 2 * kPieces;
  if (first < last) {
#pragma unroll
    for (int u = 0; u < kRing; ++u) {
      begin_load(first + u, u);
#pragma unroll
      for (int j = 0; j < kLoads; ++j) piece(j);
    }
  }

  // (slack finite: a row that has seen no key yet has a limit of minus infinity plus it)
  const float c = p.scale * kLog2e, slack = fminf(kSlack / c, -kLowest);
  f32x16 o[NF] = {}, s[2];
  u32x4 pf[2][2] = {};
  bf16x8 kf[kAhead], vf[kAhead];
  float top = kMinusInf, limit = kMinusInf, total = 0.f, base = 0.f;

  const int kat = (own + fr) * kPitch + ((fh ^ key_swizzle<kPitch>(fr)) << 4);
  const int vrow = 4 * fh + ((lane & 15) >> 2);
  const int vat = (own + vrow) * kPitch +
                  (((2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ value_swizzle<kPitch>(vrow)) << 4) + (lane & 1) * 8;
  // Fragments of the area at `at`; `row`: the first of 32 rows.
  auto read_k = [&](int at, int row, int k) __attribute__((always_inline)) {
    kf[k % kAhead] = *(const lds_bf16x8*)((const lds_byte*)smem + ((kat + at) ^ (k << 5)) + row * kPitch);
  };
  auto read_v = [&](int at, int row, int j) __attribute__((always_inline)) {  // block j % NF of keys 16 (j / NF) ..
    i16x4 part[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      part[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_i16x4*)((lds_byte*)smem + ((vat + at) ^ ((j % NF) << 6)) + kTile + (row + 16 * (j / NF) + 8 * i) * kPitch));
    vf[j % kAhead] = __builtin_bit_cast(bf16x8, i16x8{part[0][0], part[0][1], part[0][2], part[0][3], part[1][0],
                                                      part[1][1], part[1][2], part[1][3]});
  };
  // Score e of block t to a weight, two at a time.
  float most = 0.f, sum = 0.f, held = 0.f;
  auto weigh = [&](int x, int e) __attribute__((always_inline)) {
    const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x][e], c, -base));
    sum = e == 0 ? w : sum + w;
    if (e % 2 == 0) {
      held = w;
    } else {
      const bf16x2 both = {(__bf16)held, (__bf16)w};
      const unsigned word = __builtin_bit_cast(unsigned, both);
      asm volatile("" ::"v"(word), "v"(sum));  // (formed here, not where the compiler would collect them)
      pf[x][e / 8][e % 8 / 2] = word;
    }
  };
  // What the scores of a block start from: zero, minus infinity where the key is hidden.
  // Register e: key 8 (e / 4) + 4 (lane / 32) + e % 4 of the 32.
  f32x16 start = {};
  unsigned starts = ~0u;
  auto hide = [&](unsigned bits) __attribute__((always_inline)) {
    if (bits != starts) {
      starts = bits;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int at = 8 * (e / 4) + e % 4;  // (for either half of the wave a bit, as its lanes' select)
        const uint64_t both = unsigned(__builtin_amdgcn_sbfe(int(bits), at, 1)) |
                              uint64_t(unsigned(__builtin_amdgcn_sbfe(int(bits), at + 4, 1))) << 32;
        float v;
        asm("v_cndmask_b32_e64 %0, %1, 0, %2" : "=v"(v) : "v"(kMinusInf), "s"(both));
        start[e] = v;
      }
    }
  };
  // A block's maximum so far, with score e; at the end over both halves of the wave.
  auto maximum = [&](int x, int e) __attribute__((always_inline)) {
    most = e == 0 ? s[x][0] : fmaxf(most, s[x][e]);
    if (e == 15) most = fmaxf(most, other_half(most));
  };
  auto score = [&](f32x16& to, auto first_t, int f) __attribute__((always_inline)) {
    scores_mfma<decltype(first_t)::value, kAcc>(to, kf[f % kAhead], qf[f], start);
    // The first product reads `start` after it has been issued, for 11 wait
    // states that the compiler does not know of: the registers stay taken.
    if (f == KF - 1) asm volatile("" ::"v"(start));
  };
  auto output = [&](int x, int f) __attribute__((always_inline)) {
    output_mfma<kAcc>(o[f % NF], vf[f % kAhead], __builtin_bit_cast(bf16x8, pf[x][f / NF]));
  };
  auto settled = [&]() __attribute__((always_inline)) {  // before the output's sums are read
    asm volatile("s_nop 15\n\ts_nop 3" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < NF; ++n) mfma_settle<kAcc>(o[n]);
  };

  // The step with the scores and weights of set X, on rows ROW .. of the area at
  // `at`: the next block's K (`bits`: which of its keys are seen) and the last
  // one's values; the next step's rows start at NROW of the area at `nat`.
  // CROSS: that is another area, which has landed once only the loads behind
  // it may be in flight, and this one, which every wave has then read, is
  // given up to the loads that begin() names: at slot kSync, two behind the
  // last reads.  The loads go one by one into the kSpan slots from there on,
  // the next step's among them: the memory path takes 16 cycles of a CU for
  // each, and a wave whose loads stand in line issues nothing else (4096 x
  // 8192, 64 heads of 128: 1110 us with the loads all at once, 1020 so).
  constexpr int kSync = 2 * (KF - kAhead) + 2;
  constexpr int kRest = kSlots - kSync - 1;            // a step's slots behind kSync
  constexpr int kMost = FEW ? kSlots - 1 : kSlots + kRest;  // (up to the next kSync, or its step)
  constexpr int kSpan = 2 * kLoads < kMost ? 2 * kLoads : kMost;
  // QK, PV: which of the products there are (the first and the last step lack one).
  auto step = [&](auto x_t, auto qk_t, auto pv_t, auto row_t, auto cross_t, int at, int nat, unsigned bits,
                  auto&& begin) __attribute__((always_inline)) {
    constexpr int X = decltype(x_t)::value, Y = 1 - X, ROW = decltype(row_t)::value, NROW = FEW ? 0 : 32 - ROW;
    constexpr bool QK = decltype(qk_t)::value, PV = decltype(pv_t)::value, CROSS = decltype(cross_t)::value;
    if (QK) hide(bits);
    for_each_index(std::make_integer_sequence<int, kSlots>{}, [&](auto i_t) __attribute__((always_inline)) {
      constexpr int i = decltype(i_t)::value, f = i / 2;
      constexpr bool K = i % 2 == 0;
      if constexpr (K && QK)
        score(s[Y], std::integral_constant<bool, f == 0>{}, f);
      else if constexpr (!K && PV)
        output(Y, f);
      if (i < 2) __builtin_amdgcn_sched_barrier(0);  // (block t's last scores take that long)
      // The fragment kAhead ahead, of this step's rows or the next one's.
      if constexpr (f + kAhead < KF) {
        if constexpr (K && QK)
          read_k(at, ROW, f + kAhead);
        else if constexpr (!K && PV)
          read_v(at, ROW, f + kAhead);
      }
      if constexpr (CROSS && i == kSync) {
        wait_lgkm0();
        waitvm<(kRing - 2) * kLoads>();
        barrier();
        begin();
      }
      if constexpr (QK || (FEW && i <= kSync)) {
        constexpr int n = CROSS && i > kSync ? i - kSync - 1 : CROSS && !FEW ? kSpan : i + kRest;  // slots since kSync
        if constexpr (n < kSpan)
          for_each_index(std::make_integer_sequence<int, kLoads>{}, [&](auto j_t) __attribute__((always_inline)) {
            constexpr int j = decltype(j_t)::value;
            if constexpr (j * kSpan / kLoads == n) piece(j);
          });
      }
      auto next = [&](auto j_t) __attribute__((always_inline)) {  // what slot j frees the registers for
        constexpr int j = decltype(j_t)::value, jf = j / 2 + kAhead - KF;
        if constexpr (jf >= 0) {
          if constexpr (j % 2 == 0 && QK)
            read_k(nat, NROW, jf);
          else if constexpr (j % 2 == 1)
            read_v(nat, NROW, jf);
        }
      };
      if constexpr (!CROSS || i > kSync) next(i_t);
      if constexpr (CROSS && i == kSync)
        for_each_index(std::make_integer_sequence<int, kSync + 1>{}, next);
      constexpr int lo = 16 * i / kSlots, hi = 16 * (i + 1) / kSlots;
#pragma unroll
      for (int e = lo; e < hi; ++e) weigh(X, e);
      constexpr int span = 3 * kSlots / 4;  // (the maximum within three quarters of the step)
      constexpr int mlo = i < span ? 16 * i / span : 16, mhi = i < span ? 16 * (i + 1) / span : 16;
#pragma unroll
      for (int e = mlo; e < mhi; ++e) maximum(X, e);
      __builtin_amdgcn_sched_barrier(0);
    });
    if (__ballot(most > limit) != 0) {
      settled();
      const float now = fmaxf(top, most);
      base = now == kMinusInf ? 0.f : now * c;
      const float shrink = __builtin_amdgcn_exp2f(__builtin_fmaf(top, c, -base));
      top = now;
      limit = now + slack;
      total *= shrink;
      if (PV) {
#pragma unroll
        for (int n = 0; n < NF; ++n) o[n] *= shrink;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) weigh(X, e);
    }
    total += sum;
  };

  // (opaque, so that addresses are formed where they are used and not kept for every area)
  auto area = [&](int u) __attribute__((always_inline)) {
    int at = (u - first) % kRing * 2 * kTile;
    asm volatile("" : "+s"(at));
    return at;
  };
  using Yes = std::true_type;
  using No = std::false_type;
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I32 = std::integral_constant<int, 32>;
  // The last block's values, on rows ROW .. of the area at `at`.
  auto finish = [&](int x, int at, int row) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < KF; ++f) {
      output(x, f);
      if (f + kAhead < KF) read_v(at, row, f + kAhead);
    }
    settled();
  };

  if (first < last) {
    int at = area(first), to = area(first + 1);
    waitvm<(kRing - 1) * kLoads>();
    barrier();
#pragma unroll
    for (int k = 0; k < kAhead; ++k) read_k(at, 0, k);
    hide(block_bits(first, own));
    for_each_index(std::make_integer_sequence<int, KF>{}, [&](auto f_t) __attribute__((always_inline)) {
      constexpr int f = decltype(f_t)::value;
      score(s[0], std::integral_constant<bool, f == 0>{}, f);
      if constexpr (f + kAhead < KF)
        read_k(at, 0, f + kAhead);
      else if constexpr (!FEW)
        read_k(at, 32, f + kAhead - KF);
    });
    asm volatile("s_nop 15\n\ts_nop 3" : "+v"(s[0]));
    // (Neither loop tests first: round one the compiler keeps two sets of the output's sums.)
    if constexpr (FEW) {
      wait_lgkm0();
      waitvm<(kRing - 2) * kLoads>();
      barrier();
      begin_load(first + kRing, 0);
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        if (j * kSpan / kLoads < kRest) piece(j);  // (the others in the first step)
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        read_k(to, 0, k);
        read_v(to, 0, k);
      }
      // Step t makes the scores of tile t + 1, so it reads that one's area.
      int u = first + 1;
      auto go = [&](auto x_t) __attribute__((always_inline)) {
        at = to;
        to = area(u + 1);
        move_window(u);
        step(x_t, Yes{}, Yes{}, I0{}, Yes{}, at, to, block_bits(u, own),
             [&]() __attribute__((always_inline)) { begin_load(u + kRing, (u - first) % kRing); });
        ++u;
      };
      if (u + 1 < last) do {
        go(I0{});
        go(I1{});
      } while (u + 1 < last);
      auto end = [&](auto x_t) __attribute__((always_inline)) {
        at = to;
        to = area(u + 1);
        step(x_t, No{}, Yes{}, I0{}, Yes{}, at, to, 0u, []() {});
        finish(decltype(x_t)::value, to, 0);
      };
      if (u < last) {
        go(I0{});
        end(I1{});
      } else {
        end(I0{});
      }
    } else {
      step(I0{}, Yes{}, No{}, I32{}, Yes{}, at, to, block_bits(first, 32),
           [&]() __attribute__((always_inline)) { begin_load(first + kRing, 0); });
      int u = first + 1;
      if (u < last) do {
        at = to;
        to = area(u + 1);
        move_window(u);
        step(I1{}, Yes{}, Yes{}, I0{}, No{}, at, at, block_bits(u, 0), []() {});
        step(I0{}, Yes{}, Yes{}, I32{}, Yes{}, at, to, block_bits(u, 32),
             [&]() __attribute__((always_inline)) { begin_load(u + kRing, (u - first) % kRing); });
      } while (++u < last);
      step(I1{}, No{}, Yes{}, I0{}, No{}, to, to, 0u, []() {});
      finish(1, to, 32);
    }
    waitvm<0>();  // no load into LDS may be in flight where the outputs go through it
    wait_lgkm0();
    barrier();
  }

  // Register e of block n: feature 32 n + 8 (e / 4) + 4 (lane / 32) + e % 4 of query lane % 32.
  auto out_row = [&](int64_t r) __attribute__((always_inline)) {
    const int64_t token = p.ratio == 1 ? r : int64_t(unsigned(r) / unsigned(p.ratio));
    return p.out + batch * p.os[0] + token * p.os[1] + (head * p.ratio + r - token * p.ratio) * p.os[2];
  };
  int me = lane;
  asm volatile("" : "+v"(me));  // (places are formed again: kept, they would be registers too many)
  const int query = me & 31, half = me >> 5;
  const float all_sum = total + other_half(total);
  // What a part's sums are relative to.  Minus infinity: there were no keys.  The
  // lowest number: keys that are seen, but all their scores minus infinity; where
  // that is so of a whole row, 0 / 0 is what its softmax is.
  const float relative = first == last ? kMinusInf : top == kMinusInf ? kLowest : base;
  if constexpr (FEW) {
    // The waves' sums, in their order, by all threads.
    constexpr int kRow = D + 4;  // (a row's distance in floats: 16 bytes off the banks of the one before)
    float* sums = reinterpret_cast<float*>(smem) + wave * 32 * kRow;
#pragma unroll
    for (int n = 0; n < NF; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(sums + query * kRow + 32 * n + 8 * q + 4 * half) =
            f32x4{o[n][4 * q], o[n][4 * q + 1], o[n][4 * q + 2], o[n][4 * q + 3]};
    if (half == 0) {
      sums[query * kRow + D] = relative;
      sums[query * kRow + D + 1] = all_sum;
    }
    __syncthreads();
    const int chunks = p.d / 8;
    for (int i = threadIdx.x; i < 32 * chunks; i += kWaves * 64) {
      const int row = i / chunks, f = (i - row * chunks) * 8;
      if (row0 + row >= rows) break;
      const float* at = reinterpret_cast<const float*>(smem) + row * kRow;
      float most = kMinusInf;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) most = fmaxf(most, at[w * 32 * kRow + D]);
      f32x4 lo = {}, hi = {};
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float* src = at + w * 32 * kRow;
        const float weight = __builtin_amdgcn_exp2f(src[D] - (most == kMinusInf ? 0.f : most));
        sum += weight * src[D + 1];
        lo += weight * *reinterpret_cast<const f32x4*>(src + f);
        hi += weight * *reinterpret_cast<const f32x4*>(src + f + 4);
      }
      if (splits > 1) {
        float* dst = p.part + (part0 + row) * p.d + f;
        *reinterpret_cast<f32x4*>(dst) = lo;
        *reinterpret_cast<f32x4*>(dst + 4) = hi;
        if (f == 0) {
          p.stats[2 * (part0 + row)] = most;
          p.stats[2 * (part0 + row) + 1] = sum;
        }
      } else {
        const float g = most == kMinusInf ? 0.f : 1.f / sum;
        *reinterpret_cast<u32x4*>(out_row(row0 + row) + f) =
            u32x4{bf16_pair(lo[0] * g, lo[1] * g), bf16_pair(lo[2] * g, lo[3] * g), bf16_pair(hi[0] * g, hi[1] * g),
                  bf16_pair(hi[2] * g, hi[3] * g)};
      }
    }
  } else if (splits > 1) {
    if (row0 + query >= rows) return;
    const int64_t r = wave * 32 + query;
    float* dst = p.part + (part0 + r) * p.d;
    if (half == 0) {
      p.stats[2 * (part0 + r)] = relative;
      p.stats[2 * (part0 + r) + 1] = all_sum;
    }
#pragma unroll
    for (int n = 0; n < NF; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int f = 32 * n + 8 * q + 4 * half;
        if (f < p.d)
          *reinterpret_cast<f32x4*>(dst + f) = f32x4{o[n][4 * q], o[n][4 * q + 1], o[n][4 * q + 2], o[n][4 * q + 3]};
      }
  } else {
    // Whole rows out of the wave's own part of LDS (whose accesses stay in order).
    uint8_t* mine = smem + wave * 32 * kPitch;
    const float g = relative == kMinusInf ? 0.f : 1.f / all_sum;
#pragma unroll
    for (int n = 0; n < NF; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<u32x2*>(mine + query * kPitch + (((4 * n + q) ^ key_swizzle<kPitch>(query)) << 4) + 8 * half) =
            u32x2{bf16_pair(o[n][4 * q] * g, o[n][4 * q + 1] * g), bf16_pair(o[n][4 * q + 2] * g, o[n][4 * q + 3] * g)};
#pragma unroll
    for (int i = 0; i < 32 / (64 / kChunks); ++i) {
      const int row = i * (64 / kChunks) + me / kChunks, chunk = me % kChunks;
      const u32x4 v = *reinterpret_cast<const u32x4*>(mine + row * kPitch + ((chunk ^ key_swizzle<kPitch>(row)) << 4));
      if (row0 + row < rows && chunk * 16 < dbytes) *reinterpret_cast<u32x4*>(out_row(row0 + row) + chunk * 8) = v;
    }
  }
}

// The parts of the tiles whose keys are split, joined: thread = 4 features of a row.
__global__ __launch_bounds__(256) void attention_join_kernel(const AttentionArgs p, int64_t first) {
  const int quads = p.d / 4, tile_rows = p.few ? 32 : 128;
  const int64_t rows = p.m * p.ratio, count = (p.batch * p.kv_heads * p.tiles - p.whole) * tile_rows;
  const int64_t i = (first + blockIdx.x) * 256 + threadIdx.x;
  const int64_t r = i / quads;
  const int f = int(i - r * quads) * 4;
  if (r >= count) return;
  const int64_t slot = p.whole + r / tile_rows, pair = slot / p.tiles;
  const int64_t in = (slot - pair * p.tiles) * tile_rows + r % tile_rows;  // row of the key head
  if (in >= rows) return;
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
  v *= top == kMinusInf ? 0.f : 1.f / sum;
  const int64_t token = in / p.ratio;
  const int64_t batch = pair / p.kv_heads, head = (pair - batch * p.kv_heads) * p.ratio + in - token * p.ratio;
  *reinterpret_cast<u32x2*>(p.out + batch * p.os[0] + token * p.os[1] + head * p.os[2] + f) =
      u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
}

template <int D, bool FEW>
hipError_t launch_t(const AttentionArgs& a, hipStream_t stream) {
  constexpr int kThreads = attention_waves(D, FEW) * 64;
  AttentionArgs p = a;
  const int64_t tiles = a.batch * a.kv_heads * a.tiles;  // (with splits few enough for one launch)
  in_launches(a.splits > 1 ? a.whole + (tiles - a.whole) * a.splits : tiles, kThreads, [&](int64_t first, unsigned count) {
    p.first = first;
    if (a.mask)
      hipLaunchKernelGGL((attention_kernel<D, FEW, true>), dim3(count), dim3(kThreads), 0, stream, p);
    else
      hipLaunchKernelGGL((attention_kernel<D, FEW, false>), dim3(count), dim3(kThreads), 0, stream, p);
  });
  if (a.splits > 1) {
    const int64_t values = (tiles - a.whole) * (a.few ? 32 : 128) * (a.d / 4);
    in_launches((values + 255) / 256, 256, [&](int64_t first, unsigned count) {
      hipLaunchKernelGGL(attention_join_kernel, dim3(count), dim3(256), 0, stream, p, first);
    });
  }
  return hipGetLastError();
}

template <int D>
hipError_t launch_d(const AttentionArgs& a, hipStream_t stream) {
  return a.few ? launch_t<D, true>(a, stream) : launch_t<D, false>(a, stream);
}

}  // namespace

AttentionPlan plan_attention(int64_t batch, int64_t kv_heads, int64_t rows, int64_t l, int d) {
  AttentionPlan plan{};
  const int64_t cus = device_cu_count(), heads = batch * kv_heads;
  auto blocks = [&](int64_t n) { return heads * ((rows + n - 1) / n); };
  // The waves of a workgroup take the same queries where no more workgroups
  // than CUs come of it: 1 x 32760, 40 query heads on 8 of 128, 42.7 us against
  // 44.5; 64 x 32760, 8 heads, 41.4 against 46.3; 300 x 2000, 8 heads, 19.1
  // against 22.4.  With up to twice as many, 2000 x 333, 8 heads: 19.9 against 13.8.
  plan.few = blocks(32) <= cus;
  plan.rows = plan.few ? 32 : 128;
  plan.tiles = (rows + plan.rows - 1) / plan.rows;
  plan.splits = 1;
  const int64_t total = heads * plan.tiles, most = (l + 127) / 128 / 4;  // (512 keys to a part at least)
  auto split = [&](int64_t whole, int64_t want) {
    want = want < most ? want : most;
    if (want > 1) {
      plan.splits = int(want);
      plan.whole = int(whole);
    }
  };
  // Fewer tiles than CUs are split so that each CU has work.  Of more, those of
  // a last round that would leave places free are split to fill them, counting
  // two places to a CU, beyond 128 features one.  (Up to 64 features a third
  // workgroup fits, but three take the time of three there: 520 tiles of 1100
  // keys 35.6 us with the last 8 split, 37.6 without; 640 tiles of 1100 keys 41.8
  // and 39.6, of 4096 115 and 121; with three places in the count 1080 tiles of
  // 4096 keys 198 instead of 186, though 800 tiles 140 instead of 166.)
  // Up to a quarter of the places: 4608 x 4608, 30 heads of 64, 223 -> 208 us, 2176
  // x 1024, 31 of 128, 59 -> 54.  Up to a half where what is saved outweighs the
  // parts' way through memory: beyond 128 features (4096 x 4096, 20 of 160, 297 ->
  // 271), or with 12288 keys.  1280, 720 and 700 tiles of 128 features, split and
  // not: 4096 keys 345 / 335, 207 / 202, 203 / 200 us; 8192 663 / 656, 392 / 393, 385
  // / 389; 12288 976 / 983, 584 / 606, 573 / 588; 32760 2518 / 2574, 1503 / 1592, 1463
  // / 1557; of 96 features 8192 keys 572 / 570, 345 / 350, 337 / 344; 12288 843 / 848,
  // 507 / 518, 495 / 511.  Of 64 features the tiles that fit three to a CU run at
  // once: 12288 keys 607 / 618, but 381 / 372, 375 / 363; 32760 1599 / 1649, but 988
  // / 975, 975 / 956.
  const int64_t places = (plan.few || d > 128 ? 1 : 2) * cus;
  const bool half = d > 128 || (l >= 12288 && (d > 64 || total > 3 * cus));
  if (total > 0 && total < cus) {
    split(0, cus / total);
  } else if (total > places && total <= (1 << 20)) {
    const int64_t last = total % places;
    if (last > 0 && last <= (half ? places / 2 : places / 4)) split(total - last, places / last);
  }
  return plan;
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t stream) {
  if (a.d <= 64) return launch_d<64>(a, stream);
  if (a.d <= 96) return launch_d<96>(a, stream);
  if (a.d <= 128) return launch_d<128>(a, stream);
  if (a.d <= 160) return launch_d<160>(a, stream);
  return launch_d<192>(a, stream);
}

}  // namespace convrot
