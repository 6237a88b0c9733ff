// C ABI of attention: argument validation (on the host, before any HIP call)
// and dispatch.
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

constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr float kMaxScale = 2.35e38f;  // (times log2 e it is finite)
// 128 rows of keys or values lie in 31 bits.
constexpr int64_t kMaxKeyStride = int64_t(1) << 23;

convrot_status check_sizes(const convrot_attention& a) {
  if (a.batch < 0 || a.m < 0 || a.l < 0 || a.batch > kMaxRows || a.m > kMaxRows || a.l > kMaxRows ||
      a.heads < 1 || a.heads > 4096 || a.kv_heads < 1 || a.heads % a.kv_heads != 0 || a.d < 1 ||
      a.d > CONVROT_MAX_HEAD_DIM)
    return CONVROT_ERR_SHAPE;
  // (workgroups, of 32 queries at least, are counted in 32 bits)
  const int64_t rows = a.m * (a.heads / a.kv_heads);
  if (rows > kMaxRows || (rows + 31) / 32 * a.kv_heads > kMaxRows / (a.batch > 0 ? a.batch : 1))
    return CONVROT_ERR_SHAPE;
  return a.d % 8 == 0 ? CONVROT_OK : CONVROT_ERR_UNSUPPORTED;
}

// The parts of split keys: sums, then a maximum and a sum.
int64_t part_rows(const convrot_attention& a, const convrot::AttentionPlan& plan) {
  return plan.splits > 1 ? plan.splits * (a.batch * a.kv_heads * plan.tiles - plan.whole) * plan.rows : 0;
}
int64_t workspace_bytes(const convrot_attention& a, const convrot::AttentionPlan& plan) {
  return part_rows(a, plan) * (a.d + 2) * 4;
}

convrot::AttentionPlan plan_of(const convrot_attention& a) {
  return convrot::plan_attention(a.batch, a.kv_heads, a.m * (a.heads / a.kv_heads), a.l, a.d);
}

// A tensor's strides and alignment; `key`: its rows are loaded by tiles.
convrot_status check_tensor(const void* p, const int64_t* stride, int64_t tokens, int32_t d, bool key) {
  for (int i = 0; i < 3; ++i)
    if (stride[i] < 0 || stride[i] > (key && i == 1 ? kMaxKeyStride : kMaxStride)) return CONVROT_ERR_SHAPE;
  if (key && tokens > 1 && stride[1] != 0 && stride[1] < d) return CONVROT_ERR_SHAPE;
  for (int i = 0; i < 3; ++i)
    if (stride[i] % 8 != 0) return CONVROT_ERR_UNSUPPORTED;
  if (!p) return CONVROT_ERR_NULL;
  return aligned16(p) ? CONVROT_OK : CONVROT_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

convrot_status convrot_attention_workspace(const convrot_attention* a, int64_t* bytes) {
  if (!a || !bytes) return CONVROT_ERR_NULL;
  const convrot_status st = check_sizes(*a);
  if (st != CONVROT_OK) return st;
  *bytes = a->batch == 0 || a->m == 0 ? 0 : workspace_bytes(*a, plan_of(*a));
  return CONVROT_OK;
}

convrot_status convrot_attention_apply(const convrot_attention* a, void* stream) {
  if (!a) return CONVROT_ERR_NULL;
  convrot_status st = check_sizes(*a);
  if (st != CONVROT_OK) return st;
  if (!(a->scale > 0.f && a->scale <= kMaxScale)) return CONVROT_ERR_UNSUPPORTED;  // a NaN too
  if (a->mask && (a->mask_stride < 0 || a->mask_stride > kMaxStride)) return CONVROT_ERR_SHAPE;
  if (a->batch == 0 || a->m == 0) return CONVROT_OK;
  if ((st = check_tensor(a->q, a->q_stride, a->m, a->d, false)) != CONVROT_OK) return st;
  if ((st = check_tensor(a->out, a->out_stride, a->m, a->d, false)) != CONVROT_OK) return st;
  if (a->l > 0) {
    if ((st = check_tensor(a->k, a->k_stride, a->l, a->d, true)) != CONVROT_OK) return st;
    if ((st = check_tensor(a->v, a->v_stride, a->l, a->d, true)) != CONVROT_OK) return st;
  }
  if (!aligned(a->lengths, 4)) return CONVROT_ERR_UNSUPPORTED;
  if (a->out == a->q || a->out == a->k || a->out == a->v) return CONVROT_ERR_UNSUPPORTED;
  const convrot::AttentionPlan plan = plan_of(*a);
  const int64_t bytes = workspace_bytes(*a, plan);
  if (bytes > 0) {
    if (!a->workspace) return CONVROT_ERR_NULL;
    if (a->workspace_bytes < bytes) return CONVROT_ERR_SHAPE;
    if (!aligned16(a->workspace)) return CONVROT_ERR_UNSUPPORTED;
  }
  convrot::AttentionArgs p{};
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.out = static_cast<uint16_t*>(a->out);
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = a->q_stride[i];
    p.ks[i] = a->k_stride[i];
    p.vs[i] = a->v_stride[i];
    p.os[i] = a->out_stride[i];
  }
  p.batch = a->batch;
  p.m = a->m;
  p.l = a->l;
  p.kv_heads = a->kv_heads;
  p.ratio = a->heads / a->kv_heads;
  p.d = a->d;
  p.scale = a->scale;
  p.lengths = a->lengths;
  p.mask = a->mask;
  p.mask_stride = a->mask_stride;
  p.tiles = int(plan.tiles);
  p.splits = plan.splits;
  p.whole = plan.whole;
  p.few = plan.few;
  p.part = static_cast<float*>(a->workspace);
  p.stats = p.part + part_rows(*a, plan) * a->d;
  return from_hip(convrot::launch_attention(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
