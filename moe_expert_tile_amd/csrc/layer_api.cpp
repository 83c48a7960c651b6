// C ABI of the operators around the experts (declared in include/moe.h):
// routing, the dense product and the rows sorted by expert, with their
// gradients, and microscaled 4-bit rows.  Host-side validation; the launches are
// in route.hip, linear.hip, rows.hip and mx.hip.
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

// checks shared by the calls on sorted rows; fills in the row pitches
int check_rows(const moe_rows_desc* desc, const int32_t* pos, moe_rows_desc* d) {
  if (!desc) return MOE_EINVAL;
  *d = *desc;
  if (d->tokens < 0 || d->tokens > (1ll << 26) || d->rows < 0 || d->rows > INT32_MAX) return MOE_EINVAL;
  if (d->top_k < 1 || d->top_k > 32 || d->cols < 1 || d->cols > (1 << 20)) return MOE_EINVAL;
  if (d->dtype < MOE_BF16 || d->dtype > MOE_F32 || d->pad != 0) return MOE_EINVAL;
  for (int64_t* ld : {&d->ld_x, &d->ld_rows, &d->ld_d_rows}) {
    if (*ld == 0) *ld = d->cols;
    if (*ld < d->cols || *ld > kMaxPitch) return MOE_EINVAL;
  }
  if (!aligned_to(pos, 4) || (d->tokens > 0 && !pos)) return MOE_EINVAL;
  return MOE_OK;
}

// whether a buffer of `count` rows is there and aligned to its elements
bool row_buffer(const moe_rows_desc& d, const void* p, int64_t count) {
  return aligned_to(p, item(d.dtype)) && (p || count == 0);
}

// checks shared by the quantisation calls; fills in the pitches
int check_mx_rows(int64_t rows, int32_t depth, const void* x, int32_t dtype, int64_t* ld_x, const uint8_t* q,
                  int64_t* ld_q, const uint8_t* scale, int64_t* ld_s) {
  if (rows < 0 || rows > INT32_MAX || depth < 32 || depth > (1 << 20) || depth % 32 != 0) return MOE_EINVAL;
  if (dtype < MOE_BF16 || dtype > MOE_F32) return MOE_EINVAL;
  if (*ld_x == 0) *ld_x = depth;
  if (*ld_q == 0) *ld_q = depth / 2;
  if (*ld_s == 0) *ld_s = depth / 32;
  if (*ld_x < depth || *ld_x > kMaxPitch || *ld_q < depth / 2 || *ld_q > kMaxPitch || *ld_q % 16 != 0 ||
      *ld_s < depth / 32 || *ld_s > kMaxPitch)
    return MOE_EINVAL;
  if (!aligned_to(x, item(dtype)) || !aligned_to(q, 16)) return MOE_EINVAL;
  if (rows > 0 && (!x || !q || !scale)) return MOE_EINVAL;
  return MOE_OK;
}

// checks a product's sizes and fills in its pitches
int check_mx_linear(const moe_mx_linear_desc* desc, moe_mx_linear_desc* d) {
  if (!desc) return MOE_EINVAL;
  *d = *desc;
  if (d->rows < 0 || d->rows > (1ll << 26) || d->experts < 1 || d->experts > 1024) return MOE_EINVAL;
  if (d->cols < 1 || d->cols > (1 << 20)) return MOE_EINVAL;
  if (d->depth < 32 || d->depth > (1 << 20) || d->depth % 32 != 0) return MOE_EINVAL;
  const bool mx = d->dtype == MOE_MXFP4;
  if (d->dtype != MOE_BF16 && d->dtype != MOE_F16 && !mx) return MOE_EINVAL;
  if (d->out_dtype < MOE_BF16 || d->out_dtype > MOE_F32 || (!mx && d->out_dtype != d->dtype && d->out_dtype != MOE_F32))
    return MOE_EINVAL;
  if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_SWIGLU) return MOE_EINVAL;
  const int64_t n = (int64_t)d->cols * (d->act == MOE_ACT_SWIGLU ? 2 : 1);
  struct { int64_t* ld; int64_t least, unit; } pitches[] = {
      {&d->ld_x, mx ? d->depth / 2 : d->depth, mx ? 16 : 8}, {&d->ld_x_scale, d->depth / 32, 1},
      {&d->ld_w, d->depth / 2, 16}, {&d->ld_w_scale, d->depth / 32, 1}, {&d->ld_out, d->cols, 1}};
  for (auto& p : pitches) {
    if (*p.ld == 0) *p.ld = p.least;
    if (*p.ld < p.least || *p.ld > kMaxPitch || *p.ld % p.unit != 0) return MOE_EINVAL;
  }
  if (d->expert_w == 0) d->expert_w = n * d->ld_w;
  if (d->expert_w_scale == 0) d->expert_w_scale = n * d->ld_w_scale;
  const int64_t most = 1ll << 42;
  if (d->expert_w < 0 || d->expert_w > most || d->expert_w % 16 != 0 || d->expert_w_scale < 0 || d->expert_w_scale > most)
    return MOE_EINVAL;
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
  const bool none = !dx && !dw && !dbias;     // (without rows: perhaps dx, which then has no elements)
  if (none && d.rows > 0) return MOE_EINVAL;
  if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(pre, 2) || !aligned_to(d_out, item(d.out_dtype)) ||
      !aligned_to(dx, 2) || !aligned_to(dw, 2) || !aligned_to(dbias, 2) || !ws || !aligned_to(ws, 256))
    return MOE_EINVAL;
  if (d.rows > 0 && (!d_out || (dw && !x) || (dx && !w) || (d.act != MOE_ACT_NONE && !pre))) return MOE_EINVAL;
  rc = prepare_device();
  if (rc || none) return rc;
  LinearGrads b = {x, w, pre, d_out, dx, dw, dbias};
  return hip_rc(launch_linear_backward(d, b, ws, (hipStream_t)stream));
}

int moe_sort_sizes(int64_t tokens, int32_t top_k, int32_t experts, size_t* ws_bytes) {
  if (tokens < 0 || tokens > (1ll << 26) || top_k < 1 || top_k > 32 || tokens * top_k > INT32_MAX) return MOE_EINVAL;
  if (experts < 1 || experts > 1024 || !ws_bytes) return MOE_EINVAL;
  *ws_bytes = sort_ws_bytes(tokens * top_k, experts);
  return MOE_OK;
}

int moe_sort(int64_t tokens, int32_t top_k, int32_t experts, int32_t first, const int32_t* topk_ids, int32_t* pos,
             int32_t* src, int32_t* offsets, void* ws, void* stream) {
  size_t bytes;
  int rc = moe_sort_sizes(tokens, top_k, experts, &bytes);
  if (rc) return rc;
  if (first < 0 || first > INT32_MAX - experts + 1 || !aligned_to(topk_ids, 4) || !aligned_to(pos, 4) || !aligned_to(src, 4) || !aligned_to(offsets, 4) ||
      !aligned_to(ws, 256))
    return MOE_EINVAL;
  if (!offsets || (tokens > 0 && (!topk_ids || !pos)) || (bytes > 0 && !ws)) return MOE_EINVAL;
  rc = prepare_device();
  if (rc) return rc;
  return hip_rc(launch_sort(tokens * top_k, experts, first, topk_ids, pos, src, offsets, ws, (hipStream_t)stream));
}

int moe_permute(const moe_rows_desc* desc, const void* x, const int32_t* pos, void* rows, void* stream) {
  moe_rows_desc d;
  int rc = check_rows(desc, pos, &d);
  if (rc) return rc;
  if (!row_buffer(d, x, d.tokens) || !row_buffer(d, rows, d.rows)) return MOE_EINVAL;
  rc = prepare_device();
  if (rc || d.tokens == 0 || d.rows == 0) return rc;
  return hip_rc(launch_permute(d, x, pos, rows, (hipStream_t)stream));
}

int moe_unpermute(const moe_rows_desc* desc, const void* rows, const int32_t* pos, const float* topk_w, void* out,
                  void* stream) {
  moe_rows_desc d;
  int rc = check_rows(desc, pos, &d);
  if (rc) return rc;
  if (!row_buffer(d, rows, d.rows) || !row_buffer(d, out, d.tokens) || !aligned_to(topk_w, 4)) return MOE_EINVAL;
  rc = prepare_device();
  if (rc || d.tokens == 0) return rc;
  return hip_rc(launch_unpermute(d, rows, pos, topk_w, out, (hipStream_t)stream));
}

int moe_permute_backward(const moe_rows_desc* desc, const void* d_rows, const int32_t* pos, void* dx, void* stream) {
  return moe_unpermute(desc, d_rows, pos, nullptr, dx, stream);   // the same sum, without weights
}

int moe_unpermute_backward(const moe_rows_desc* desc, const void* rows, const int32_t* pos, const float* topk_w,
                           const void* d_out, void* d_rows, float* d_topk_w, void* stream) {
  moe_rows_desc d;
  int rc = check_rows(desc, pos, &d);
  if (rc) return rc;
  // a gradient without elements may be null as well, and nothing be left to write
  const bool none = !d_rows && !d_topk_w;
  if (none && d.tokens > 0 && d.rows > 0) return MOE_EINVAL;
  if (!row_buffer(d, d_out, d.tokens) || !row_buffer(d, d_rows, 0) || !row_buffer(d, rows, d_topk_w ? d.rows : 0) ||
      !aligned_to(topk_w, 4) || !aligned_to(d_topk_w, 4))
    return MOE_EINVAL;
  rc = prepare_device();
  if (rc || d.tokens == 0 || none) return rc;
  return hip_rc(launch_unpermute_backward(d, rows, pos, topk_w, d_out, d_rows, d_topk_w, (hipStream_t)stream));
}

int moe_mx_quantize(int64_t rows, int32_t depth, const void* x, int32_t dtype, int64_t ld_x, uint8_t* q, int64_t ld_q,
                    uint8_t* scale, int64_t ld_scale, void* stream) {
  int rc = check_mx_rows(rows, depth, x, dtype, &ld_x, q, &ld_q, scale, &ld_scale);
  if (!rc) rc = prepare_device();
  if (rc || rows == 0) return rc;
  return hip_rc(launch_mx_quantize(rows, depth, x, dtype, ld_x, q, ld_q, scale, ld_scale, (hipStream_t)stream));
}

int moe_mx_dequantize(int64_t rows, int32_t depth, const uint8_t* q, int64_t ld_q, const uint8_t* scale,
                      int64_t ld_scale, void* out, int32_t dtype, int64_t ld_out, void* stream) {
  int rc = check_mx_rows(rows, depth, out, dtype, &ld_out, q, &ld_q, scale, &ld_scale);
  if (!rc) rc = prepare_device();
  if (rc || rows == 0) return rc;
  return hip_rc(launch_mx_dequantize(rows, depth, q, ld_q, scale, ld_scale, out, dtype, ld_out, (hipStream_t)stream));
}

int moe_mx_linear(const moe_mx_linear_desc* desc, const void* x, const uint8_t* x_scale, const uint8_t* w,
                  const uint8_t* w_scale, const int32_t* offsets, const void* bias, void* out, void* stream) {
  moe_mx_linear_desc d;
  int rc = check_mx_linear(desc, &d);
  if (rc) return rc;
  const size_t o = item(d.out_dtype);
  if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(offsets, 4) || !aligned_to(bias, o) || !aligned_to(out, o))
    return MOE_EINVAL;
  if (!offsets && d.experts != 1) return MOE_EINVAL;
  if (d.rows > 0 && (!x || !w || !w_scale || !out || (d.dtype == MOE_MXFP4 && !x_scale))) return MOE_EINVAL;
  rc = prepare_device();
  if (rc || d.rows == 0) return rc;
  return hip_rc(launch_mx_linear(d, x, x_scale, w, w_scale, offsets, bias, out, (hipStream_t)stream));
}

}  // extern "C"
