// C ABI of the FP8 linears, the block norms and the rotary positions:
// argument validation (on the host, before any HIP call) and dispatch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/convrot.h"
#include "checks.h"
#include "kernels.h"

using convrot::aligned;
using convrot::aligned16;
using convrot::from_hip;
using convrot::kMaxRows;

namespace {

// Row strides of the elementwise operators: row * stride * 4 bytes stays
// far inside 64 bits.
constexpr int64_t kMaxStride = int64_t(1) << 40;

bool float_type(int32_t t) { return t == CONVROT_F32 || t == CONVROT_BF16; }
unsigned size_of(int32_t t) { return t == CONVROT_BF16 ? 2 : 4; }
// Whether every row starts at a multiple of 16 bytes.
bool rows_at_16(const void* x, int64_t m, int64_t ldx, int32_t type) {
  return aligned16(x) && (m == 1 || ldx * size_of(type) % 16 == 0);
}
int64_t blocks(int64_t n) { return (n + CONVROT_FP8_BLOCK - 1) / CONVROT_FP8_BLOCK; }

convrot_status check_k(int64_t k) {
  if (k < 1 || k > CONVROT_MAX_K) return CONVROT_ERR_SHAPE;
  return k % 16 == 0 ? CONVROT_OK : CONVROT_ERR_UNSUPPORTED;
}

// The buffers of an FP8 activation [m, k] that exists (m > 0).
convrot_status check_fp8_buffers(const convrot_fp8_packed* p) {
  if (!p->q || !p->scale) return CONVROT_ERR_NULL;
  return aligned16(p->q) && aligned(p->scale, 4) ? CONVROT_OK : CONVROT_ERR_UNSUPPORTED;
}

convrot_status check_fp8_stride(int64_t lds, int64_t m) {
  if (lds < m || lds > kMaxStride) return CONVROT_ERR_SHAPE;
  return m == 0 || lds % 4 == 0 ? CONVROT_OK : CONVROT_ERR_UNSUPPORTED;
}

convrot_status fill_vector(const convrot_vector& v, int64_t k, bool grouped, convrot::VectorArgs* out) {
  *out = convrot::VectorArgs{};
  if (!v.data) return CONVROT_OK;
  if (!float_type(v.dtype)) return CONVROT_ERR_DTYPE;
  if (grouped && (v.stride < 0 || v.stride > kMaxStride || v.rows < 1)) return CONVROT_ERR_SHAPE;
  if (!aligned(v.data, size_of(v.dtype))) return CONVROT_ERR_UNSUPPORTED;
  out->p = v.data;
  out->stride = grouped ? v.stride : 0;
  out->rows = grouped ? v.rows : 1;
  out->bf16 = v.dtype == CONVROT_BF16;
  return CONVROT_OK;
}

convrot_status fill_norm(const convrot_norm& n, int64_t k, convrot::NormArgs* out) {
  *out = convrot::NormArgs{};
  if (n.kind == CONVROT_NORM_NONE)  // (a weight without a norm is no norm's)
    return n.weight.data || n.bias.data ? CONVROT_ERR_UNSUPPORTED : CONVROT_OK;
  if (n.kind != CONVROT_NORM_LAYER && n.kind != CONVROT_NORM_RMS) return CONVROT_ERR_DTYPE;
  if (!(n.eps >= 0.f)) return CONVROT_ERR_UNSUPPORTED;  // a NaN too
  out->kind = n.kind == CONVROT_NORM_LAYER ? convrot::kNormLayer : convrot::kNormRms;
  out->eps = n.eps;
  const convrot_status st = fill_vector(n.weight, k, false, &out->weight);
  return st != CONVROT_OK ? st : fill_vector(n.bias, k, false, &out->bias);
}

// A matrix operand's type, row stride and alignment.
convrot_status check_matrix(const void* p, int32_t dtype, int64_t ld, int64_t k) {
  if (!float_type(dtype)) return CONVROT_ERR_DTYPE;
  if (ld < k || ld > kMaxStride) return CONVROT_ERR_SHAPE;
  return aligned(p, size_of(dtype)) ? CONVROT_OK : CONVROT_ERR_UNSUPPORTED;
}

// The weights and outputs of an FP8 linear whose m and k are filled in; fills
// the launch's weights (those with rows) and modes.
convrot_status check_fp8_linear(const convrot_fp8_weights* w, int32_t count, void* const* y,
                                const int64_t* ldy, int32_t y_dtype, int32_t act,
                                convrot::Fp8GemmArgs* a) {
  if (!w || !y || !ldy) return CONVROT_ERR_NULL;
  if (count < 1 || count > CONVROT_MAX_GROUPED) return CONVROT_ERR_SHAPE;
  const convrot_status st = check_k(a->k);
  if (st != CONVROT_OK) return st;
  if (a->m < 0 || a->m > kMaxRows) return CONVROT_ERR_SHAPE;
  if (!float_type(y_dtype)) return CONVROT_ERR_DTYPE;
  if (act != CONVROT_ACT_NONE && act != CONVROT_ACT_GELU) return CONVROT_ERR_DTYPE;
  a->f32_scale = w[0].scale_dtype == CONVROT_F32;
  a->y_bf16 = y_dtype == CONVROT_BF16;
  a->gelu = act == CONVROT_ACT_GELU;
  int64_t tiles = 0;
  for (int32_t i = 0; i < count; ++i) {
    const convrot_fp8_weights& wi = w[i];
    if (wi.k != a->k || wi.n < 0 || wi.n > kMaxRows || ldy[i] < wi.n || ldy[i] > kMaxStride)
      return CONVROT_ERR_SHAPE;
    if ((wi.scale_dtype != CONVROT_F32 && wi.scale_dtype != CONVROT_E8M0) ||
        wi.scale_dtype != w[0].scale_dtype)
      return CONVROT_ERR_DTYPE;
    if (wi.n == 0 || a->m == 0) continue;  // empty weights launch nothing
    if (!wi.q || !wi.scale || !y[i]) return CONVROT_ERR_NULL;
    if (!aligned16(wi.q) || (a->f32_scale && !aligned(wi.scale, 4)) ||
        (wi.bias && !aligned(wi.bias, 4)) || !aligned(y[i], size_of(y_dtype)))
      return CONVROT_ERR_UNSUPPORTED;
    a->w[a->count++] = {static_cast<const uint8_t*>(wi.q), wi.scale, wi.bias, y[i], wi.n, ldy[i]};
    tiles += (wi.n + 31) / 32;
  }
  // (32 x 32 tiles, smaller than any kernel's, are counted in 32 bits)
  return tiles * ((a->m + 31) / 32) > int64_t(INT32_MAX) ? CONVROT_ERR_SHAPE : CONVROT_OK;
}

}  // namespace

extern "C" {

convrot_status convrot_fp8_quantize_weights(const void* w, int32_t w_dtype, int64_t n, int64_t k,
                                            int64_t ldw, void* q_out, void* scale_out,
                                            void* stream) {
  const convrot_status st = check_k(k);
  if (st != CONVROT_OK) return st;
  if (n < 0 || n > kMaxRows || ldw < k || ldw > kMaxStride || blocks(n) * blocks(k) > INT32_MAX)
    return CONVROT_ERR_SHAPE;
  if (!float_type(w_dtype)) return CONVROT_ERR_DTYPE;
  if (n == 0) return CONVROT_OK;
  if (!w || !q_out || !scale_out) return CONVROT_ERR_NULL;
  if (!aligned16(q_out) || !aligned(w, size_of(w_dtype))) return CONVROT_ERR_UNSUPPORTED;
  return from_hip(convrot::launch_fp8_wquant(w, w_dtype == CONVROT_BF16, ldw, n, k,
                                             static_cast<uint8_t*>(q_out),
                                             static_cast<uint8_t*>(scale_out),
                                             static_cast<hipStream_t>(stream)));
}

convrot_status convrot_fp8_pack_activations(const void* x, int32_t x_dtype, int64_t m, int64_t k,
                                            int64_t ldx, convrot_fp8_packed* out, void* stream) {
  if (!out) return CONVROT_ERR_NULL;
  convrot_status st = check_k(k);
  if (st != CONVROT_OK) return st;
  if (m < 0 || m > kMaxRows || ldx < k || ldx > kMaxStride) return CONVROT_ERR_SHAPE;
  if (!float_type(x_dtype)) return CONVROT_ERR_DTYPE;
  st = check_fp8_stride(out->lds, m);
  if (st != CONVROT_OK) return st;
  if (m > 0) {
    if (!x) return CONVROT_ERR_NULL;
    st = check_fp8_buffers(out);
    if (st != CONVROT_OK) return st;
    if (!rows_at_16(x, m, ldx, x_dtype)) return CONVROT_ERR_UNSUPPORTED;
  }
  out->m = m;
  out->k = k;
  if (m == 0) return CONVROT_OK;
  return from_hip(convrot::launch_fp8_pack(x, x_dtype == CONVROT_BF16, ldx, m, k,
                                           static_cast<uint8_t*>(out->q),
                                           static_cast<uint8_t*>(out->scale), out->lds,
                                           static_cast<hipStream_t>(stream)));
}

convrot_status convrot_fp8_linear_grouped(const convrot_fp8_packed* x,
                                          const convrot_fp8_weights* w, int32_t count,
                                          void* const* y, const int64_t* ldy, int32_t y_dtype,
                                          int32_t act, void* stream) {
  if (!x) return CONVROT_ERR_NULL;
  convrot::Fp8GemmArgs a{};
  a.qx = static_cast<const uint8_t*>(x->q);
  a.sx = static_cast<const uint8_t*>(x->scale);
  a.lds = x->lds;
  a.m = x->m;
  a.k = x->k;
  convrot_status st = check_fp8_linear(w, count, y, ldy, y_dtype, act, &a);
  if (st != CONVROT_OK) return st;
  st = check_fp8_stride(x->lds, x->m);
  if (st != CONVROT_OK) return st;
  if (x->m == 0 || a.count == 0) return CONVROT_OK;
  st = check_fp8_buffers(x);
  if (st != CONVROT_OK) return st;
  return from_hip(convrot::launch_fp8_gemm(a, static_cast<hipStream_t>(stream)));
}

convrot_status convrot_fp8_linear_rows(const void* x, int32_t x_dtype, int64_t m, int64_t k,
                                       int64_t ldx, const convrot_fp8_weights* w, int32_t count,
                                       void* const* y, const int64_t* ldy, int32_t y_dtype,
                                       int32_t act, void* stream) {
  static_assert(convrot::kFp8RawBytes == CONVROT_FP8_MAX_ROWS_BYTES, "header");
  if (k < 1 || k > CONVROT_MAX_K || m > CONVROT_FP8_MAX_ROWS ||
      (m > 0 && blocks(k) * 128 > CONVROT_FP8_MAX_ROWS_BYTES / m))
    return CONVROT_ERR_SHAPE;
  convrot::Fp8GemmArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.x_bf16 = x_dtype == CONVROT_BF16;
  a.m = m;
  a.k = k;
  const convrot_status st = check_fp8_linear(w, count, y, ldy, y_dtype, act, &a);
  if (st != CONVROT_OK) return st;
  if (ldx < k || ldx > kMaxStride) return CONVROT_ERR_SHAPE;
  if (!float_type(x_dtype)) return CONVROT_ERR_DTYPE;
  if (m == 0 || a.count == 0) return CONVROT_OK;
  if (!x) return CONVROT_ERR_NULL;
  if (!rows_at_16(x, m, ldx, x_dtype)) return CONVROT_ERR_UNSUPPORTED;
  return from_hip(convrot::launch_fp8_gemm_rows(a, static_cast<hipStream_t>(stream)));
}

convrot_status convrot_block_norm(const convrot_block* b, void* stream) {
  if (!b) return CONVROT_ERR_NULL;
  if (b->k < 1 || b->k > CONVROT_MAX_NORM_K || b->m < 0 || b->m > kMaxRows)
    return CONVROT_ERR_SHAPE;
  if (b->y && b->packed) return CONVROT_ERR_UNSUPPORTED;
  // (an empty call's pointers say nothing)
  if (b->m > 0 && !b->branch &&
      (b->h || b->gate.data || b->post.kind != CONVROT_NORM_NONE || b->residual_scale != 1.f))
    return CONVROT_ERR_UNSUPPORTED;
  const bool wants_y = b->y || b->packed;
  if (b->m > 0 && !wants_y &&
      (b->pre.kind != CONVROT_NORM_NONE || b->scale.data || b->shift.data))
    return CONVROT_ERR_UNSUPPORTED;
  convrot::BlockNormArgs a{};
  convrot_status st = check_matrix(b->x, b->x_dtype, b->ldx, b->k);
  if (st != CONVROT_OK) return st;
  if (b->branch && (st = check_matrix(b->branch, b->branch_dtype, b->ldb, b->k)) != CONVROT_OK)
    return st;
  if (b->h && (st = check_matrix(b->h, b->x_dtype, b->ldh, b->k)) != CONVROT_OK) return st;
  if (b->y && (st = check_matrix(b->y, b->y_dtype, b->ldy, b->k)) != CONVROT_OK) return st;
  if (b->packed) {
    if ((st = check_k(b->k)) != CONVROT_OK) return st;
    if ((st = check_fp8_stride(b->packed->lds, b->m)) != CONVROT_OK) return st;
  }
  if ((st = fill_vector(b->gate, b->k, true, &a.gate)) != CONVROT_OK) return st;
  if ((st = fill_vector(b->scale, b->k, true, &a.scale)) != CONVROT_OK) return st;
  if ((st = fill_vector(b->shift, b->k, true, &a.shift)) != CONVROT_OK) return st;
  if ((st = fill_norm(b->post, b->k, &a.post)) != CONVROT_OK) return st;
  if ((st = fill_norm(b->pre, b->k, &a.pre)) != CONVROT_OK) return st;
  if (b->m > 0) {
    if (!b->x || (!b->h && !wants_y)) return CONVROT_ERR_NULL;
    if (b->packed && (st = check_fp8_buffers(b->packed)) != CONVROT_OK) return st;
    // In place: over x, row by row; nothing else is read and written.
    if ((b->h && (b->h == b->y || b->h == b->branch || (b->h == b->x && b->ldh != b->ldx))) ||
        (b->y && (b->y == b->branch ||
                  (b->y == b->x && (b->ldy != b->ldx || b->y_dtype != b->x_dtype)))))
      return CONVROT_ERR_UNSUPPORTED;
  }
  if (b->packed) {
    b->packed->m = b->m;
    b->packed->k = b->k;
    a.q = static_cast<uint8_t*>(b->packed->q);
    a.q_scale = static_cast<uint8_t*>(b->packed->scale);
    a.lds = b->packed->lds;
  }
  if (b->m == 0) return CONVROT_OK;
  a.x = b->x;
  a.branch = b->branch;
  a.h = b->h;
  a.y = b->y;
  a.m = b->m;
  a.k = b->k;
  a.ldx = b->ldx;
  a.ldb = b->ldb;
  a.ldh = b->ldh;
  a.ldy = b->ldy;
  a.residual_scale = b->residual_scale;
  a.x_bf16 = b->x_dtype == CONVROT_BF16;
  a.branch_bf16 = b->branch_dtype == CONVROT_BF16;
  a.y_bf16 = b->y_dtype == CONVROT_BF16;
  return from_hip(convrot::launch_block_norm(a, static_cast<hipStream_t>(stream)));
}

convrot_status convrot_rope_apply(const convrot_rope* r, void* stream) {
  if (!r) return CONVROT_ERR_NULL;
  if (r->batch < 0 || r->tokens < 0 || r->batch > kMaxRows || r->tokens > kMaxRows ||
      r->count < 1 || r->count > CONVROT_MAX_ROPE_TENSORS || r->axes < 1 || r->d < 2 || r->d > 4096 ||
      r->rot < 2 || r->rot % 2 != 0 || r->start < 0 || r->start > r->d - r->rot)
    return CONVROT_ERR_SHAPE;
  if (r->batch * r->tokens > kMaxRows) return CONVROT_ERR_SHAPE;
  if (!float_type(r->x_dtype) || !float_type(r->y_dtype)) return CONVROT_ERR_DTYPE;
  if (r->position_type < CONVROT_POS_I32 || r->position_type > CONVROT_POS_F32 ||
      (r->layout != CONVROT_ROPE_INTERLEAVED && r->layout != CONVROT_ROPE_HALF))
    return CONVROT_ERR_DTYPE;
  convrot::RopeArgs a{};
  const bool empty = r->batch == 0 || r->tokens == 0;
  for (int32_t i = 0; i < r->count; ++i) {
    const convrot_rope_tensor& t = r->t[i];
    if (t.heads < 0 || t.heads > 4096 || t.heads * r->d > (1 << 18)) return CONVROT_ERR_SHAPE;
    for (int j = 0; j < 3; ++j)
      if (t.x_stride[j] < 0 || t.x_stride[j] > kMaxStride || t.y_stride[j] < 0 ||
          t.y_stride[j] > kMaxStride)
        return CONVROT_ERR_SHAPE;
    if (t.heads == 0 || empty) continue;
    if (!t.x || !t.y) return CONVROT_ERR_NULL;
    if (!aligned(t.x, size_of(r->x_dtype)) || !aligned(t.y, size_of(r->y_dtype)))
      return CONVROT_ERR_UNSUPPORTED;
    if (t.x == t.y) {  // in place: the same places of the same type
      if (r->x_dtype != r->y_dtype) return CONVROT_ERR_UNSUPPORTED;
      for (int j = 0; j < 3; ++j)
        if (t.x_stride[j] != t.y_stride[j]) return CONVROT_ERR_UNSUPPORTED;
    }
    for (int j = 0; j < a.count; ++j)  // another tensor's place, before it is read or after
      if (t.y == a.t[j].y || t.y == a.t[j].x || t.x == a.t[j].y) return CONVROT_ERR_UNSUPPORTED;
    convrot::RopeTensor& o = a.t[a.count++];
    o.x = t.x;
    o.y = t.y;
    for (int j = 0; j < 3; ++j) {
      o.xs[j] = t.x_stride[j];
      o.ys[j] = t.y_stride[j];
    }
    o.heads = int(t.heads);
    o.copy_rest = t.x != t.y;
  }
  for (int j = 0; j < 2; ++j)
    if (r->pos_stride[j] < 0 || r->pos_stride[j] > kMaxStride) return CONVROT_ERR_SHAPE;
  if (a.count == 0) return CONVROT_OK;
  if (!r->inv_freq || !r->positions) return CONVROT_ERR_NULL;
  if (!aligned(r->inv_freq, 8) || (r->axis && !aligned(r->axis, 4)) ||
      !aligned(r->positions, r->position_type == CONVROT_POS_I64 ? 8 : 4))
    return CONVROT_ERR_UNSUPPORTED;
  a.positions = r->positions;
  a.inv_freq = r->inv_freq;
  a.axis = r->axis;
  a.batch = r->batch;
  a.tokens = r->tokens;
  a.axes = r->axes;
  a.pos_batch = r->pos_stride[0];
  a.pos_token = r->pos_stride[1];
  a.d = r->d;
  a.rot = r->rot;
  a.start = r->start;
  a.factor = r->factor;
  a.pos_type = r->position_type == CONVROT_POS_I32   ? convrot::kPosI32
               : r->position_type == CONVROT_POS_I64 ? convrot::kPosI64
                                                     : convrot::kPosF32;
  a.half = r->layout == CONVROT_ROPE_HALF;
  a.inverse = r->inverse != 0;
  a.x_bf16 = r->x_dtype == CONVROT_BF16;
  a.y_bf16 = r->y_dtype == CONVROT_BF16;
  return from_hip(convrot::launch_rope(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
