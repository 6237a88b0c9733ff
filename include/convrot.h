/*
 * convrot.h — C ABI of libconvrot.so, the INT8 "convrot" linear layer on
 * AMD Instinct MI355X (gfx950).
 *
 * The method is the one described on the stable-diffusion.cpp documentation
 * page "INT8 Convrot Safetensors" (cited below as [ICS] with the section):
 *   - R is block diagonal; each block is R_G, the normalised Kronecker power
 *     of the 4x4 regular Hadamard matrix H4 printed in [ICS, How INT8 convrot
 *     works], applied to every contiguous group of G = 4^n input features;
 *   - weights are rotated offline (W_rot = W R) and quantised per output row
 *     [ICS, Weight quantization];
 *   - activations are rotated at run time (X_rot = X R) and quantised with one
 *     dynamic scale per row, giving the packed activation: int8 rows plus
 *     their float row scales [ICS, Runtime activation quantization];
 *   - A = Q_x Q_w^T accumulates in int32 and Y = A s_x[r] s_w[o] + b[o]
 *     [ICS, Runtime activation quantization].
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller; the library
 *     allocates no device memory and keeps no pointer after a call returns.
 *   - Matrices are row-major.  "ld" arguments are row strides in elements.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).  All
 *     work is enqueued asynchronously on it; nothing synchronises.
 *   - Every argument is validated on the host before any HIP call, so an
 *     invalid call returns an error code and launches nothing.  A launch
 *     failure reported by the HIP runtime returns CONVROT_ERR_HIP.  Nothing is
 *     printed and no C++ exception crosses the ABI.  The functions are
 *     reentrant; calls on different streams may overlap.
 *   - Rounding is round-half-away-from-zero; a row whose absmax is zero gets
 *     scale 0 and all-zero codes (the page leaves both open).
 *   - Inputs are assumed finite.
 *
 * Limits (all return an error code when violated):
 *   - group_size G = 4^n with 0 <= n <= 7 (1 .. 16384), and G divides k
 *     ([ICS, Checkpoint format]: a power of four dividing in_features);
 *   - 1 <= k <= CONVROT_MAX_K, so that k * 127 * 127 fits in int32, and
 *     k % 16 == 0 (16-byte rows; an extension limit of this library);
 *   - m, n >= 0 (0 is an empty call that launches nothing) and < 2^31;
 *   - X, codes and weight pointers 16-byte aligned, X row stride a multiple
 *     of 16 bytes; Y needs only 4-byte alignment (any ldy >= n).
 */
#ifndef CONVROT_H
#define CONVROT_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CONVROT_MAX_K 133136      /* largest k with k % 16 == 0 and k*127*127 < 2^31 */
#define CONVROT_MAX_LOG4_GROUP 7  /* group sizes 1, 4, 16, ..., 16384 */
#define CONVROT_MAX_GROUPED 8     /* weight matrices per convrot_linear_grouped call */
#define CONVROT_MAX_LORA_RANK 256 /* adapter ranks 16, 32, ..., 256 */

typedef enum convrot_status {
  CONVROT_OK = 0,
  CONVROT_ERR_NULL = 1,           /* a required pointer is NULL */
  CONVROT_ERR_SHAPE = 2,          /* m, n or k out of range, ld < row length */
  CONVROT_ERR_GROUP = 3,          /* G not a power of four in range, or G does not divide k */
  CONVROT_ERR_GROUP_MISMATCH = 4, /* packed activation and weights differ in G or k */
  CONVROT_ERR_DTYPE = 5,          /* unknown or unsupported dtype / activation code */
  CONVROT_ERR_UNSUPPORTED = 6,    /* k % 16 != 0, misaligned pointer or stride */
  CONVROT_ERR_HIP = 7             /* the HIP runtime reported an error */
} convrot_status;

typedef enum convrot_dtype {
  CONVROT_F32 = 0,
  CONVROT_BF16 = 1,
  CONVROT_I32 = 2,
  CONVROT_E8M0 = 3                /* a power of two as its exponent's byte; scales only */
} convrot_dtype;

typedef enum convrot_act {
  CONVROT_ACT_NONE = 0,
  CONVROT_ACT_GELU = 1            /* x * Phi(x), erf form; not on the page, used by DiT MLPs */
} convrot_act;

/*
 * The packed runtime activation of [ICS, Runtime activation quantization]:
 * int8 rows and one float32 scale per row.  It may feed any number of
 * convrot_linear calls whose weights share its k and group size.
 *   q     : device int8 [m, k], row stride exactly k bytes (caller-allocated)
 *   scale : device float32 [m]                               (caller-allocated)
 */
typedef struct convrot_packed {
  int8_t* q;
  float* scale;
  int64_t m;
  int64_t k;
  int32_t group_size;
} convrot_packed;

/*
 * Quantised weights of one linear layer, [ICS, Checkpoint format]: an int8
 * [out_features, in_features] matrix and one float scale per output row.
 *   q     : device int8 [n, k], row stride exactly k bytes
 *   scale : device float32 [n]
 *   bias  : device float32 [n], or NULL for no bias
 */
typedef struct convrot_weights {
  const int8_t* q;
  const float* scale;
  const float* bias;
  int64_t n;
  int64_t k;
  int32_t group_size;
} convrot_weights;

/*
 * Offline weight preparation, [ICS, How INT8 convrot works] (W_rot = W R) and
 * [ICS, Weight quantization]:
 *   s_w[o]    = max_i |W_rot[o, i]| / 127          (stored as float32)
 *   Q_w[o, i] = clamp(round(W_rot[o, i] / s_w[o]), -127, 127)
 * The rotation, absmax, division and rounding are done in float64; the float64
 * quotient max/127 is rounded once to float32 and the division uses that
 * stored float32 value.
 *   w         : device float32 [n, k], row stride ldw >= k (input, unchanged)
 *   q_out     : device int8 [n, k], row stride k (output)
 *   scale_out : device float32 [n] (output)
 * Errors: NULL, SHAPE, GROUP, UNSUPPORTED, HIP.
 */
convrot_status convrot_quantize_weights(const float* w, int64_t n, int64_t k, int64_t ldw,
                                        int32_t group_size, int8_t* q_out, float* scale_out,
                                        void* stream);

/*
 * Runtime activation rotation and quantisation into a packed activation,
 * [ICS, Runtime activation quantization]: each row of X is rotated group-wise
 * (X_rot = X R), then
 *   s_x[r]    = max_i |X_rot[r, i]| / 127
 *   Q_x[r, i] = clamp(round(X_rot[r, i] / s_x[r]), -127, 127)
 * in float32: the rotation is a radix-4 butterfly in float32; max/127 and
 * X_rot/s_x are correctly rounded float32 operations.  X is not modified (the
 * unrotated X stays available, e.g. for low-rank adapters).
 *   x       : device [m, k] of x_dtype (CONVROT_F32 or CONVROT_BF16), row stride ldx >= k
 *   out->q, out->scale : caller-allocated device buffers (see convrot_packed);
 *             on success the call sets out->m, out->k and out->group_size.
 * Errors: NULL, SHAPE, GROUP, DTYPE, UNSUPPORTED, HIP.
 */
convrot_status convrot_pack_activations(const void* x, int32_t x_dtype, int64_t m, int64_t k,
                                        int64_t ldx, int32_t group_size, convrot_packed* out,
                                        void* stream);

/*
 * The convrot linear on a packed activation, [ICS, Runtime activation
 * quantization]:
 *   A[r, o] = sum_i Q_x[r, i] Q_w[o, i]               (exact int32)
 *   Y[r, o] = A[r, o] * s_x[r] * s_w[o] + b[o]        (float32; then act)
 * y_dtype CONVROT_F32 writes Y (float32 [m, n], row stride ldy >= n; Y must
 * not overlap the inputs);
 * y_dtype CONVROT_I32 writes the raw int32 A (no scale, bias or act; act must
 * be CONVROT_ACT_NONE).  act CONVROT_ACT_GELU applies x*Phi(x) to Y.
 * The packed activation and the weights must have the same k and the same
 * group size ([ICS, Runtime activation quantization]: a packed tensor is
 * shared only by layers with the same input and group size).
 * Errors: NULL, SHAPE, GROUP_MISMATCH, DTYPE, UNSUPPORTED, HIP.
 */
convrot_status convrot_linear(const convrot_packed* x, const convrot_weights* w, void* y,
                              int32_t y_dtype, int64_t ldy, int32_t act, void* stream);

/*
 * Several convrot linears on ONE packed activation in one launch: the linear
 * layers that share an input and a group size reuse its packed tensor
 * ([ICS, Runtime activation quantization]), e.g. the Q, K and V projections
 * of an attention block.  Weight i writes y[i] (row stride ldy[i] >= w[i].n);
 * semantics per weight are those of convrot_linear, with one y_dtype and one
 * act for all.  Weights with n == 0 are skipped.  The outputs must not
 * overlap one another or any input (short outputs are accumulated in place,
 * as int32 partial sums, before they are scaled).
 *   w   : host array of `count` convrot_weights (device pointers inside)
 *   y   : host array of `count` device output pointers
 *   ldy : host array of `count` row strides
 *   1 <= count <= CONVROT_MAX_GROUPED
 * Errors: NULL, SHAPE, GROUP_MISMATCH, DTYPE, UNSUPPORTED, HIP.
 */
convrot_status convrot_linear_grouped(const convrot_packed* x, const convrot_weights* w,
                                      int32_t count, void* const* y, const int64_t* ldy,
                                      int32_t y_dtype, int32_t act, void* stream);

/*
 * Low-rank adapters ([ICS, Backend support]): LoRA-style adapters are applied
 * at run time without touching the int8 weights; the convrot linear gives the
 * base output and the adapter's correction, computed from the original
 * UNROTATED activation X, is added to it.  In the low-rank form, with down
 * weights A [rank, k], up weights B [n, rank] and a scale (alpha / rank):
 *   U = bf16(scale * X A^T)          (convrot_lora_down)
 *   Y += U B^T                       (fused: convrot_linear_lora;
 *                                     separate: convrot_lora_up_add)
 * Operands are bfloat16 with float32 accumulation; the scale is applied to
 * the float32 sum X A^T, which is then rounded to bfloat16 (nearest even).
 * (The page gives no formula or precision for the adapter path; this is the
 * library's reading.)
 */

/*
 * convrot_lora_down: U = bf16(scale * X A^T).
 *   x : device [m, k] of x_dtype (CONVROT_F32 or CONVROT_BF16), row stride
 *       k <= ldx <= 2^21; float32 X is rounded to bfloat16 (nearest even) first
 *   a : device bfloat16 [rank, k], row stride k
 *   u : device bfloat16 [m, ldu] (output; columns rank .. ldu-1 untouched, so
 *       several adapters' U can share one buffer)
 * Adapters with the same scale on the same X (the Q, K and V projections of
 * one block) can stack their A matrices, up to CONVROT_MAX_LORA_RANK rows in
 * all, into one call that reads X once and writes each adapter's U as a
 * column range of the shared buffer; each U column is computed the same way.
 *   rank a multiple of 16 in 16 .. CONVROT_MAX_LORA_RANK; k % 16 == 0;
 *   rank <= ldu <= 2^20 and ldu % 8 == 0;
 *   x, a, u 16-byte aligned, ldx in whole 16-byte units.
 * Errors: NULL, SHAPE, DTYPE, UNSUPPORTED, HIP.
 */
convrot_status convrot_lora_down(const void* x, int32_t x_dtype, int64_t m, int64_t k,
                                 int64_t ldx, const void* a, int32_t rank, float scale, void* u,
                                 int64_t ldu, void* stream);

/*
 * convrot_lora_up_add: Y[i, o] += sum_j U[i, j] B[o, j], a separate pass over Y.
 *   u : device bfloat16 [m, ldu] (from convrot_lora_down)
 *   b : device bfloat16 [n, rank], row stride rank
 *   y : device float32 [m, n], row stride ldy >= n (updated in place,
 *       typically the output of convrot_linear)
 *   rank and ldu as for convrot_lora_down; u and b 16-byte aligned, y 4-byte
 *   aligned; ceil(m / 128) * ceil(n / 128) <= INT32_MAX (128 x 128 tiles).
 * Errors: NULL, SHAPE, UNSUPPORTED, HIP.
 */
convrot_status convrot_lora_up_add(const void* u, int64_t ldu, const void* b, int64_t m,
                                   int64_t n, int32_t rank, float* y, int64_t ldy, void* stream);

/*
 * One weight's adapter for convrot_linear_lora.
 *   u    : device bfloat16 [m, ldu], this adapter's U from convrot_lora_down
 *   b    : device bfloat16 [n, rank], row stride rank
 *   ldu  : row stride of u in elements, rank <= ldu <= 2^20, ldu % 8 == 0
 *   rank : a multiple of 16 in 16 .. CONVROT_MAX_LORA_RANK, or 0 for a weight
 *          without an adapter (u, b and ldu are then ignored)
 */
typedef struct convrot_lora {
  const void* u;
  const void* b;
  int64_t ldu;
  int32_t rank;
} convrot_lora;

/*
 * convrot_linear_grouped (float32 output) with each weight's adapter added
 * in the GEMM epilogue, so Y is written once:
 *   Y_i = act(A_i s_x s_w,i + b_i + U_i B_i^T)
 * (act applies to the adapted output).  lora: host array of `count` adapters.
 * Errors: those of convrot_linear_grouped; SHAPE or UNSUPPORTED for an
 * adapter's rank, ldu or alignment; NULL for a missing u or b.
 */
convrot_status convrot_linear_lora(const convrot_packed* x, const convrot_weights* w,
                                   const convrot_lora* lora, int32_t count, void* const* y,
                                   const int64_t* ldy, int32_t act, void* stream);

/*
 * ---------------------------------------------------------------------------
 * FP8 linears: E4M3 codes with a scale for each block of 128 features.
 *
 * Activations have one scale per row and block, weights one per 128 x 128
 * block:
 *   Y[r, o] = act( sum_b sx[r, b] sw[o / 128, b] sum_{i in b} qx[r, i] qw[o, i] + bias[o] )
 * with float32 sums of exact products where Y is float32.  Where Y is bfloat16
 * the products of 8 consecutive features (8 j .. 8 j + 7) are first cut to a
 * multiple of 2^(e - 13), e the largest sum of two factors' exponents among
 * them (that of an E4M3 subnormal or zero is -6), and added exactly; these sums
 * are added in float32.  A bfloat16 output is therefore off by less than
 * 7 2^-13 times the sum of the groups' largest products (all codes E4M3 normal
 * numbers), besides the float32 additions and its own rounding of 2^-8: for
 * ordinary data 1.5e-5 to 4e-5 of its size, but an output that is small because
 * larger products cancel has that error of the larger ones.
 * No rotation is applied.  E4M3 is the OCP "fn" format (largest value 448, no
 * infinity).  The library writes power-of-two scales
 * (E8M0: the byte e + 127 stands for 2^e, 255 for NaN): the least e in
 * [-126, 127] for which the block's largest magnitude is at most 448 2^e,
 * and 0 for a block of zeros.  A code is then the E4M3 value nearest to
 * x 2^-e, ties to even.  A block that holds an infinity or a NaN becomes NaN
 * throughout.  Every code times its scale is a finite float32 number (with
 * others' scales beyond that, outputs may be infinite where a sum is not).
 * k need not be a multiple of 128 (the last block is shorter),
 * but k % 16 == 0 and k <= CONVROT_MAX_K.
 * ---------------------------------------------------------------------------
 */

#define CONVROT_FP8_BLOCK 128 /* features (and weight rows) per scale */

/*
 * An FP8 activation.
 *   q     : device E4M3 [m, k], row stride exactly k bytes, 16-byte aligned
 *   scale : device E8M0 [ceil(k / 128), lds] bytes: the scales of one block
 *           of features side by side, row r's at [b * lds + r]; lds >= m,
 *           lds % 4 == 0, 4-byte aligned (bytes m .. are padding, whatever
 *           they hold)
 */
typedef struct convrot_fp8_packed {
  void* q;
  void* scale;
  int64_t m;
  int64_t k;
  int64_t lds;
} convrot_fp8_packed;

/*
 * FP8 weights of one linear layer.
 *   q     : device E4M3 [n, k], row stride exactly k bytes, 16-byte aligned
 *   scale : device [ceil(n / 128), ceil(k / 128)], contiguous, of scale_dtype
 *           (CONVROT_E8M0, or CONVROT_F32 for checkpoints with any scales)
 *   bias  : device float32 [n], or NULL for no bias
 */
typedef struct convrot_fp8_weights {
  const void* q;
  const void* scale;
  const float* bias;
  int64_t n;
  int64_t k;
  int32_t scale_dtype;
} convrot_fp8_weights;

/*
 * Offline weight quantisation in blocks of 128 x 128 with E8M0 scales.
 *   w         : device [n, k] of w_dtype (CONVROT_F32 or CONVROT_BF16), row stride ldw >= k
 *   q_out     : device E4M3 [n, k], row stride k, 16-byte aligned
 *   scale_out : device E8M0 [ceil(n / 128), ceil(k / 128)]
 * Errors: NULL, SHAPE, DTYPE, UNSUPPORTED, HIP.
 */
convrot_status convrot_fp8_quantize_weights(const void* w, int32_t w_dtype, int64_t n, int64_t k,
                                            int64_t ldw, void* q_out, void* scale_out,
                                            void* stream);

/*
 * Activation quantisation in blocks of 1 x 128 with E8M0 scales.
 *   x   : device [m, k] of x_dtype (CONVROT_F32 or CONVROT_BF16), row stride ldx >= k, 16-byte
 *         aligned rows
 *   out : q, scale and lds are the caller's; the call sets m and k
 * Errors: NULL, SHAPE, DTYPE, UNSUPPORTED, HIP.
 */
convrot_status convrot_fp8_pack_activations(const void* x, int32_t x_dtype, int64_t m, int64_t k,
                                            int64_t ldx, convrot_fp8_packed* out, void* stream);

/*
 * One or several FP8 linears on one packed activation, in one launch.
 * Weight i writes y[i] (row stride ldy[i] >= w[i].n) as y_dtype (CONVROT_F32
 * or CONVROT_BF16, rounded once), after act.  All weights have the same
 * scale_dtype.  The outputs must not overlap one another or any input; y
 * needs its element's alignment only.
 *   1 <= count <= CONVROT_MAX_GROUPED
 * Errors: NULL, SHAPE, DTYPE, UNSUPPORTED, HIP.
 */
convrot_status convrot_fp8_linear_grouped(const convrot_fp8_packed* x,
                                          const convrot_fp8_weights* w, int32_t count,
                                          void* const* y, const int64_t* ldy, int32_t y_dtype,
                                          int32_t act, void* stream);

/*
 * The same on X itself, which is quantised on the way as
 * convrot_fp8_pack_activations does, in one launch: for single tokens.  At
 * most CONVROT_FP8_MAX_ROWS rows, and m * 128 * ceil(k / 128) at most
 * CONVROT_FP8_MAX_ROWS_BYTES (48 KB of codes).
 *   x : device [m, k] of x_dtype (CONVROT_F32 or CONVROT_BF16), row stride ldx >= k, 16-byte
 *       aligned rows
 * Errors: NULL, SHAPE, DTYPE, UNSUPPORTED, HIP.
 */
#define CONVROT_FP8_MAX_ROWS 16
#define CONVROT_FP8_MAX_ROWS_BYTES 49152
convrot_status convrot_fp8_linear_rows(const void* x, int32_t x_dtype, int64_t m, int64_t k,
                                       int64_t ldx, const convrot_fp8_weights* w, int32_t count,
                                       void* const* y, const int64_t* ldy, int32_t y_dtype,
                                       int32_t act, void* stream);

/*
 * ---------------------------------------------------------------------------
 * The norms around a transformer block, with its gate and residual.
 *   h = residual_scale * x + gate * post(branch)       (with a branch; else h = x)
 *   y = pre(h) * (1 + scale) + shift
 * post and pre are
 *   CONVROT_NORM_LAYER  (v - mean) / sqrt(mean (v - mean)^2 + eps) * weight + bias
 *   CONVROT_NORM_RMS    v / sqrt(mean v^2 + eps) * weight + bias
 *   CONVROT_NORM_NONE   v
 * in float32 throughout; y is computed from h before h is rounded to its
 * type.  gate, scale, shift, weight and bias may each be absent (data NULL):
 * a factor of one, an addend of zero.
 * ---------------------------------------------------------------------------
 */
#define CONVROT_MAX_NORM_K 32768

typedef enum convrot_norm_kind {
  CONVROT_NORM_NONE = 0,
  CONVROT_NORM_LAYER = 1,
  CONVROT_NORM_RMS = 2
} convrot_norm_kind;

/*
 * Vectors of k values (CONVROT_F32 or CONVROT_BF16), `stride` elements apart,
 * each shared by `rows` >= 1 consecutive rows: row r takes vector r / rows.
 * data NULL: absent.  A norm's weight and bias are one vector for all rows
 * (their stride and rows are not read).
 */
typedef struct convrot_vector {
  const void* data;
  int64_t stride;
  int64_t rows;
  int32_t dtype;
} convrot_vector;

typedef struct convrot_norm {
  int32_t kind; /* convrot_norm_kind */
  float eps;    /* >= 0 */
  convrot_vector weight, bias;
} convrot_norm;

/*
 *   x      : [m, k] of x_dtype, row stride ldx
 *   branch : [m, k] of branch_dtype, row stride ldb, or NULL (then h, gate and
 *            post are absent too, and residual_scale is 1)
 *   h      : [m, k] of x_dtype, row stride ldh, or NULL when not wanted
 *   y      : [m, k] of y_dtype, row stride ldy, or NULL when not wanted
 *   packed : y as an FP8 activation (see convrot_fp8_packed; k % 16 == 0)
 *            instead of y, or NULL; the call sets its m and k
 * At least one output is wanted.  h or y may be x itself (same pointer, type
 * and stride), not both; no other output may overlap an input or another
 * output.
 * Pointers need their element's alignment only.  1 <= k <= CONVROT_MAX_NORM_K.
 */
typedef struct convrot_block {
  const void* x;
  const void* branch;
  void* h;
  void* y;
  convrot_fp8_packed* packed;
  int64_t m, k;
  int64_t ldx, ldb, ldh, ldy;
  int32_t x_dtype, branch_dtype, y_dtype;
  float residual_scale;
  convrot_vector gate, scale, shift;
  convrot_norm post, pre;
} convrot_block;

/* Errors: NULL, SHAPE, DTYPE, UNSUPPORTED, HIP. */
convrot_status convrot_block_norm(const convrot_block* b, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Rotary positions.  In each head of d features the pairs of the slice
 * [start, start + rot) turn by angle = positions[token, axis[j]] * inv_freq[j]:
 *   (a, b) -> (a c - b s, b c + a s),   c = factor cos(angle), s = factor sin(angle)
 * (s of the opposite sign with `inverse`).  Pair j is features (2j, 2j + 1)
 * of the slice (interleaved) or (j, j + rot / 2) (half).  The other features
 * pass through.  Angles are formed in float64, turned in float32.
 * ---------------------------------------------------------------------------
 */
#define CONVROT_MAX_ROPE_TENSORS 4

typedef enum convrot_rope_layout {
  CONVROT_ROPE_INTERLEAVED = 0,
  CONVROT_ROPE_HALF = 1
} convrot_rope_layout;

typedef enum convrot_position_type {
  CONVROT_POS_I32 = 0,
  CONVROT_POS_I64 = 1,
  CONVROT_POS_F32 = 2
} convrot_position_type;

/*
 * One tensor [batch, tokens, heads, d] with any element strides of the first
 * three axes (stride 1 along d).  y may be x itself with the same strides and
 * type; otherwise they must not overlap, nor may y overlap another tensor of
 * the call.
 */
typedef struct convrot_rope_tensor {
  const void* x;
  void* y;
  int64_t x_stride[3];
  int64_t y_stride[3];
  int64_t heads;
} convrot_rope_tensor;

/*
 *   inv_freq  : device float64 [rot / 2]
 *   axis      : device int32 [rot / 2], values in 0 .. axes - 1, or NULL (axis
 *               0).  A pair with another value has no position: its results
 *               are NaN.
 *   positions : device, of position_type: [batch, tokens, axes] with element
 *               strides pos_stride[0] (0: the same for every batch entry) and
 *               pos_stride[1]; the axes of a token are consecutive
 *   x_dtype, y_dtype : CONVROT_F32 or CONVROT_BF16, the same for all tensors
 *   rot even, 2 <= rot, 0 <= start, start + rot <= d <= 4096; heads <= 4096
 *   and heads * d <= 2^18 in each tensor; batch * tokens < 2^31
 */
typedef struct convrot_rope {
  const double* inv_freq;
  const int32_t* axis;
  const void* positions;
  int64_t pos_stride[2];
  int64_t batch, tokens;
  int32_t position_type;
  int32_t d, rot, start;
  int32_t layout, inverse;
  int32_t x_dtype, y_dtype;
  float factor;
  int32_t count; /* 1 .. CONVROT_MAX_ROPE_TENSORS */
  int32_t axes;  /* positions of a token, >= 1 */
  convrot_rope_tensor t[CONVROT_MAX_ROPE_TENSORS];
} convrot_rope;

/* Errors: NULL, SHAPE, DTYPE, UNSUPPORTED, HIP. */
convrot_status convrot_rope_apply(const convrot_rope* r, void* stream);

/* A static, human-readable name for a status code (never NULL). */
const char* convrot_status_string(convrot_status status);

/* Library version as major*10000 + minor*100 + patch. */
int32_t convrot_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CONVROT_H */
