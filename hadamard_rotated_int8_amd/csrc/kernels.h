// Host-side launchers of the convrot kernels (internal to libconvrot.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convrot {

// launch(first, count) for the workgroups first .. first + count - 1 of
// `blocks`, in as many launches as that takes.  A grid names at most 2^32 - 1
// threads along an axis; HIP takes a larger one without an error and runs the
// remainder only.
template <typename F>
inline void in_launches(int64_t blocks, int threads, F&& launch) {
  const int64_t most = ((int64_t(1) << 32) - 1) / threads;
  for (int64_t first = 0; first < blocks; first += most)
    launch(first, unsigned(blocks - first < most ? blocks - first : most));
}

// Compute units of the current device (cached per device).
int device_cu_count();

// Launch shape of the activation pack for a row length k (k % 16 == 0).
struct PackPlan {
  int threads;            // workgroup size, 64..1024
  int chunks_per_thread;  // 16-feature chunks per thread per segment (1 or 2)
  int segments;           // > 1 only for very long rows: X is then read twice
};
PackPlan plan_pack(int64_t k);

hipError_t launch_pack(const void* x, bool bf16, int64_t ldx, int64_t m, int64_t k, int log4g,
                       int8_t* q, float* scale, hipStream_t stream);

hipError_t launch_wprep(const float* w, int64_t n, int64_t k, int64_t ldw, int log4g,
                        int8_t* q, float* scale, hipStream_t stream);

constexpr int kMaxGemmGroup = 8;  // weight matrices per grouped launch

struct GemmWeight {
  const int8_t* qw;   // [n, k]
  const float* sw;    // [n]
  const float* bias;  // [n] or nullptr
  void* y;            // [m, ldy] float32 or int32
  int64_t n, ldy;
  // Low-rank adapter added in the epilogue (rank 0: none): Y += U B^T.
  const uint16_t* lu = nullptr;  // U bfloat16 [m, ldu]
  const uint16_t* lb = nullptr;  // B bfloat16 [n, rank]
  int64_t ldu = 0;
  int rank = 0;
};

struct GemmArgs {
  const int8_t* qx;   // [m, k]
  const float* sx;    // [m]
  int64_t m, k;
  int count;          // 1 .. kMaxGemmGroup
  GemmWeight w[kMaxGemmGroup];
  bool raw_i32;
  bool gelu;
  bool lora = false;  // add each weight's adapter (GemmWeight::rank > 0) in the epilogue
};
hipError_t launch_gemm(const GemmArgs& a, hipStream_t stream);
// Outputs with few 256 x 192 tiles (short M or narrow N, no adapters): the
// split-K path (64 x 128 or 64 x 64 tiles; with several K slices int32
// atomic sums into Y, then the scaling pass).  gemm_split_wanted decides and
// picks the number of K slices and the tile width (64 or 128).
bool gemm_split_wanted(const GemmArgs& a, int cus, int* slices, int* tile_n);
hipError_t launch_gemm_split(const GemmArgs& a, int slices, int tile_n, hipStream_t stream);

constexpr int kLoraMaxRank = 256;        // adapter ranks 16, 32, ..., 256
constexpr int64_t kLoraMaxLdu = 1 << 20;  // U row stride limit (32-bit buffer offsets)
constexpr int64_t kLoraMaxLdx = 1 << 21;  // X row stride limit of the down projection (same)

// U = bf16(scale X A^T) (bfloat16 [m, r], row stride ldu); X [m, k] bf16 or
// float32, A bfloat16 [r, k].
hipError_t launch_lora_down(const void* x, bool bf16, int64_t ldx, int64_t m, int64_t k,
                            const uint16_t* a, int r, float scale, uint16_t* u, int64_t ldu,
                            hipStream_t stream);
// Y [m, n] (row stride ldy) += U B^T; U bfloat16 [m, r] (row stride ldu),
// B bfloat16 [n, r].
hipError_t launch_lora_up_add(const uint16_t* u, int64_t ldu, const uint16_t* b, int64_t m,
                              int64_t n, int r, float* y, int64_t ldy, hipStream_t stream);

// FP8 (E4M3) blocks of 128: q [m, k] and E8M0 scales [ceil(k / 128), lds] of X; q [n, k]
// and scales [ceil(n / 128), ceil(k / 128)] of W.
hipError_t launch_fp8_pack(const void* x, bool bf16, int64_t ldx, int64_t m, int64_t k,
                           uint8_t* q, uint8_t* scale, int64_t lds, hipStream_t stream);
hipError_t launch_fp8_wquant(const void* w, bool bf16, int64_t ldw, int64_t n, int64_t k,
                             uint8_t* q, uint8_t* scale, hipStream_t stream);

struct Fp8Weight {
  const uint8_t* q;
  const void* scale;  // E8M0 bytes or float32 (Fp8GemmArgs::f32_scale)
  const float* bias;  // or nullptr
  void* y;
  int64_t n, ldy;
};

struct Fp8GemmArgs {
  const uint8_t* qx;  // the packed activation ...
  const uint8_t* sx;
  const void* x;      // ... or X itself, a few rows (row stride ldx)
  int64_t ldx;
  bool x_bf16;
  int64_t lds, m, k;
  int count;
  Fp8Weight w[kMaxGemmGroup];
  bool f32_scale, y_bf16, gelu;
  // Gated: w[0] is the gate (with y), w[1] the up projection, act one of kAct*.
  bool gated;
  int act;
  void* kept[2];  // both projections as bfloat16 [m, ldk], or nullptr
  int64_t ldk;
};
constexpr int kActGelu = 1, kActSilu = 2;
hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t stream);
// A few rows of X itself (fp8_gemm_rows.hip).
constexpr int kFp8RawBytes = 49152;  // codes of an unpacked X (at most 16 rows of whole blocks)
hipError_t launch_fp8_gemm_rows(const Fp8GemmArgs& a, hipStream_t stream);
// Outputs with many tiles of 256 x 256 (fp8_gemm_wide.hip).
bool fp8_wide_wanted(const Fp8GemmArgs& a);
hipError_t launch_fp8_gemm_wide(const Fp8GemmArgs& a, hipStream_t stream);
hipError_t launch_fp8_gated_wide(const Fp8GemmArgs& a, hipStream_t stream);  // (fp8_gated.hip)
// A gated pair's way back and the transposed weights it takes (fp8_gated.hip).
struct GatedBackArgs {
  const void* dy;
  const uint16_t *gate, *up;  // the kept projections
  uint16_t *dgate, *dup;
  uint8_t *q, *q_scale;  // both gradients packed: [m, 2 * (n rounded up to 128)]
  int64_t m, n, lddy, ldk, ldd, lds;
  bool dy_bf16;
  int act;
};
hipError_t launch_gated_back(const GatedBackArgs& a, hipStream_t stream);
// q_out [k, ldq] = q^T, zeros up to the next multiple of 128 columns, and its
// blocks' scales [ceil(k / 128), ldq / 128].
struct Fp8TransposeArgs {
  const uint8_t* q;
  const void* scale;
  int64_t n, k;
  uint8_t* q_out;
  void* scale_out;
  int64_t ldq;
  bool f32_scale;
};
hipError_t launch_fp8_transpose(const Fp8TransposeArgs& a, hipStream_t stream);

// The norms around a block (block_norm.hip).
constexpr int64_t kMaxNormK = 32768;
enum { kNormNone = 0, kNormLayer = 1, kNormRms = 2 };

struct VectorArgs {  // a vector of k values for each `rows` consecutive rows, or absent
  const void* p;
  int64_t stride, rows;
  bool bf16;
};

struct NormArgs {
  int kind;
  float eps;
  VectorArgs weight, bias;
};

struct BlockNormArgs {
  const void* x;
  const void* branch;  // or nullptr
  void* h;             // of x's type, or nullptr
  void* y;             // or nullptr
  uint8_t* q;          // the FP8 packed y, or nullptr
  uint8_t* q_scale;
  int64_t m, k, ldx, ldb, ldh, ldy, lds;
  float residual_scale;
  bool x_bf16, branch_bf16, y_bf16;
  VectorArgs gate, scale, shift;
  NormArgs post, pre;
  int waves;      // of a row; the launcher's choice
  int64_t first;  // workgroup of the launch's first one
};
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream);

// Rotary positions (rope.hip).
constexpr int kMaxRopeTensors = 4;
enum { kPosI32 = 0, kPosI64 = 1, kPosF32 = 2 };

struct RopeTensor {
  const void* x;
  void* y;
  int64_t xs[3], ys[3];  // element strides of batch, token and head
  int heads;
  bool copy_rest;  // the features outside the rotated part are copied (not in place)
};

struct RopeArgs {
  const void* positions;
  const double* inv_freq;  // [rot / 2]
  const int32_t* axis;     // [rot / 2] or nullptr
  int64_t batch, tokens, pos_batch, pos_token;
  int axes;
  int count;
  int d, rot, start;
  float factor;
  int pos_type;
  bool half, inverse, x_bf16, y_bf16;
  RopeTensor t[kMaxRopeTensors];
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);

// Group norm, channels last (group_norm.hip).
constexpr int kMaxGroupNormC = 4096;
struct GroupNormArgs {
  const void* x;
  void* y;
  int64_t xs[2], ys[2];  // element strides of image and position
  int64_t batch, positions;
  int c, groups;
  float eps;
  bool x_bf16, y_bf16, silu;
  VectorArgs weight, bias;
  int64_t runs;  // of an image's positions, or 0: a group in one workgroup
  double* part;  // [batch][groups][runs] mean and squared differences, with runs
  float* stats;  // [batch][groups] mean, what its rounding took off, 1 / deviation, unused
  int64_t first;  // workgroup of the launch's first one
};
int64_t plan_group_norm(int64_t batch, int64_t positions, int c, int groups);
hipError_t launch_group_norm(const GroupNormArgs& a, hipStream_t stream);

// Attention (attention.hip).
struct AttentionArgs {
  const uint16_t *q, *k, *v;  // bfloat16
  uint16_t* out;
  int64_t qs[3], ks[3], vs[3], os[3];  // element strides of batch, token and head
  int64_t batch, m, l;
  int kv_heads, ratio, d;  // ratio: query heads that share a key head
  float scale;
  const int32_t* lengths;  // [batch] or nullptr
  const uint8_t* mask;     // [batch] rows of l bytes, or nullptr
  int64_t mask_stride;
  float* part;   // [splits][rows of the tiles whose keys are split][d]
  float* stats;  // ... and the maximum (in powers of two) and sum of each row
  int tiles, splits, whole;
  bool few;
  int64_t first;  // workgroup of the launch's first one
};
struct AttentionPlan {
  int64_t tiles;  // of a key head's queries, each of ...
  int rows;
  int splits;     // of the keys ...
  int whole;      // ... of all heads' tiles behind so many
  bool few;       // the waves of a workgroup share 32 queries (else each has 32)
};
AttentionPlan plan_attention(int64_t batch, int64_t kv_heads, int64_t rows, int64_t l, int d);
hipError_t launch_attention(const AttentionArgs& a, hipStream_t stream);

}  // namespace convrot
