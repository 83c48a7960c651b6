// C ABI of the operators around the experts (declared in include/moe.h):
// routing and the dense product, with their gradients.  Host-side validation;
// the launches are in route.hip and linear.hip.
#include <hip/hip_runtime.h>

#include <math.h>
#include <string.h>

#include "moe.h"
#include "layer_internal.h"

using namespace moe;

namespace {

int hip_rc(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }
size_t item(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

constexpr int64_t kMaxPitch = 1 << 21;

// checks shared by the routing calls; fills in the defaults of opts and ld
int check_route(int64_t tokens, int32_t experts, int32_t top_k, const void* logits, int32_t dtype, int64_t* ld,
                const moe_route_opts* opts, moe_route_opts* o) {
  if (tokens < 0 || tokens > (1ll << 26)) return MOE_EINVAL;
  if (experts < 1 || experts > 1024 || top_k < 1 || top_k > 32 || top_k > experts) return MOE_EINVAL;
  if (dtype < MOE_BF16 || dtype > MOE_F32) return MOE_EINVAL;
  if (*ld == 0) *ld = experts;
  if (*ld < experts || *ld > kMaxPitch) return MOE_EINVAL;
  if (!aligned_to(logits, item(dtype))) return MOE_EINVAL;
  memset(o, 0, sizeof(*o));
  if (opts) *o = *opts;
  if (o->score != MOE_SCORE_SOFTMAX && o->score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
  o->renorm = o->renorm != 0;
  if (o->scale == 0.0f) o->scale = 1.0f;
  if (!(o->scale > 0.0f) || !isfinite(o->scale)) return MOE_EINVAL;
  return MOE_OK;
}

int check_groups(int32_t experts, int32_t top_k, moe_route_opts* o) {
  if (o->n_group == 0) o->n_group = 1;
  if (o->n_group < 1 || o->n_group > 64 || experts % o->n_group != 0) return MOE_EINVAL;
  if (o->topk_group == 0) o->topk_group = o->n_group;
  if (o->topk_group < 1 || o->topk_group > o->n_group) return MOE_EINVAL;
  if (o->group_score != MOE_GROUP_MAX && o->group_score != MOE_GROUP_TOP2) return MOE_EINVAL;
  const int size = experts / o->n_group;
  if (o->n_group > 1 && o->group_score == MOE_GROUP_TOP2 && size < 2) return MOE_EINVAL;
  if (top_k > (int64_t)o->topk_group * size) return MOE_EINVAL;
  return MOE_OK;
}

// checks a dense product's sizes and fills in its row pitches
int check_linear(const moe_linear_desc* desc, moe_linear_desc* d) {
  if (!desc) return MOE_EINVAL;
  *d = *desc;
  if (d->rows < 0 || d->rows > kMaxPitch) return MOE_EINVAL;
  if (d->cols < 1 || d->cols > (1 << 20)) return MOE_EINVAL;
  if (d->depth < 8 || d->depth > (1 << 20) || d->depth % 8 != 0) return MOE_EINVAL;
  if (d->dtype != MOE_BF16 && d->dtype != MOE_F16) return MOE_EINVAL;
  if (d->out_dtype != d->dtype && d->out_dtype != MOE_F32) return MOE_EINVAL;
  if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_SWIGLU || d->pad != 0) return MOE_EINVAL;
  const int64_t n = (int64_t)d->cols * (d->act == MOE_ACT_SWIGLU ? 2 : 1);
  struct { int64_t* ld; int64_t least, unit; } pitches[] = {
      {&d->ld_x, d->depth, 8}, {&d->ld_w, d->depth, 8}, {&d->ld_residual, d->cols, 1}, {&d->ld_pre, n, 1},
      {&d->ld_out, d->cols, 1}, {&d->ld_dx, d->depth, 1}, {&d->ld_dw, d->depth, 1}};
  for (auto& p : pitches) {
    if (*p.ld == 0) *p.ld = p.least;
    if (*p.ld < p.least || *p.ld > kMaxPitch || *p.ld % p.unit != 0) return MOE_EINVAL;
  }
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_route(int64_t tokens, int32_t experts, int32_t top_k, const void* logits, int32_t dtype, int64_t ld,
              const float* bias, const moe_route_opts* opts, int32_t* topk_ids, float* topk_w, void* stream) {
  moe_route_opts o;
  int rc = check_route(tokens, experts, top_k, logits, dtype, &ld, opts, &o);
  if (!rc) rc = check_groups(experts, top_k, &o);
  if (rc) return rc;
  if (!aligned_to(bias, 4) || !aligned_to(topk_ids, 4) || !aligned_to(topk_w, 4)) return MOE_EINVAL;
  if (tokens > 0 && (!logits || !topk_ids || !topk_w)) return MOE_EINVAL;
  rc = prepare_device();
  if (rc || tokens == 0) return rc;
  return hip_rc(launch_route(tokens, experts, top_k, logits, dtype, ld, bias, o, topk_ids, topk_w, (hipStream_t)stream));
}

int moe_route_backward(int64_t tokens, int32_t experts, int32_t top_k, const void* logits, int32_t dtype,
                       int64_t ld, const int32_t* topk_ids, const float* topk_w, const float* d_topk_w,
                       const moe_route_opts* opts, void* d_logits, int64_t ld_d, void* stream) {
  moe_route_opts o;
  int rc = check_route(tokens, experts, top_k, logits, dtype, &ld, opts, &o);
  if (rc) return rc;
  if (ld_d == 0) ld_d = experts;
  if (ld_d < experts || ld_d > kMaxPitch) return MOE_EINVAL;
  if (!aligned_to(topk_ids, 4) || !aligned_to(topk_w, 4) || !aligned_to(d_topk_w, 4) ||
      !aligned_to(d_logits, item(dtype)))
    return MOE_EINVAL;
  if (tokens > 0 && (!logits || !topk_ids || !topk_w || !d_topk_w || !d_logits)) return MOE_EINVAL;
  rc = prepare_device();
  if (rc || tokens == 0) return rc;
  return hip_rc(launch_route_backward(tokens, experts, top_k, logits, dtype, ld, topk_ids, topk_w, d_topk_w, o,
                                      d_logits, ld_d, (hipStream_t)stream));
}

int moe_linear_sizes(const moe_linear_desc* desc, size_t* forward_bytes, size_t* backward_bytes) {
  moe_linear_desc d;
  int rc = check_linear(desc, &d);
  if (rc) return rc;
  if (forward_bytes) *forward_bytes = linear_ws_bytes(d);
  if (backward_bytes) *backward_bytes = linear_back_ws_bytes(d);
  return MOE_OK;
}

int moe_linear(const moe_linear_desc* desc, const void* x, const void* w, const void* bias, const void* residual,
               void* pre, void* out, void* ws, void* stream) {
  moe_linear_desc d;
  int rc = check_linear(desc, &d);
  if (rc) return rc;
  const size_t o = item(d.out_dtype);
  if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(bias, 2) || !aligned_to(residual, o) ||
      !aligned_to(pre, 2) || !aligned_to(out, o) || !aligned_to(ws, 256))
    return MOE_EINVAL;
  if (d.rows > 0 && (!x || !w || !out)) return MOE_EINVAL;
  if (residual && residual == out && d.ld_residual != d.ld_out) return MOE_EINVAL;
  if (!ws && linear_ws_bytes(d) > 0) return MOE_EINVAL;
  rc = prepare_device();
  if (rc || d.rows == 0) return rc;
  LinearBuffers b = {x, w, bias, residual, pre, out};
  return hip_rc(launch_linear(d, b, ws, (hipStream_t)stream));
}

int moe_linear_backward(const moe_linear_desc* desc, const void* x, const void* w, const void* pre,
                        const void* d_out, void* dx, void* dw, void* dbias, void* ws, void* stream) {
  moe_linear_desc d;
  int rc = check_linear(desc, &d);
  if (rc) return rc;
  if (!dx && !dw && !dbias) return MOE_EINVAL;
  if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(pre, 2) || !aligned_to(d_out, item(d.out_dtype)) ||
      !aligned_to(dx, 2) || !aligned_to(dw, 2) || !aligned_to(dbias, 2) || !ws || !aligned_to(ws, 256))
    return MOE_EINVAL;
  if (d.rows > 0 && (!d_out || (dw && !x) || (dx && !w) || (d.act != MOE_ACT_NONE && !pre))) return MOE_EINVAL;
  rc = prepare_device();
  if (rc) return rc;
  LinearGrads b = {x, w, pre, d_out, dx, dw, dbias};
  return hip_rc(launch_linear_backward(d, b, ws, (hipStream_t)stream));
}

}  // extern "C"
