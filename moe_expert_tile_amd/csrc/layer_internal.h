// Internal declarations of the operators around the experts (routing, dense
// product, their gradients and the scale step's).  They are apart from
// moe_internal.h, which the grouped GEMMs compile from: counters measured on
// those stay valid while the operators change.
#ifndef MOE_EXPERT_TILE_LAYER_INTERNAL_H
#define MOE_EXPERT_TILE_LAYER_INTERNAL_H

#include "moe_internal.h"

namespace moe {

// gradient of the scale step (scale.hip)
hipError_t launch_scale_backward(const PlanLayout& L, const int32_t* ws, const uint16_t* recv_self,
                                 const float* topk_w, const uint16_t* d_out, uint16_t* d_recv, float* d_topk_w,
                                 hipStream_t s);

// routing (route.hip); `o` has its defaults filled in
hipError_t launch_route(int64_t T, int E, int k, const void* logits, int dtype, int64_t ld, const float* bias,
                        const moe_route_opts& o, int32_t* ids, float* w, hipStream_t s);
hipError_t launch_route_backward(int64_t T, int E, int k, const void* logits, int dtype, int64_t ld,
                                 const int32_t* ids, const float* w, const float* dw, const moe_route_opts& o,
                                 void* dz, int64_t ldd, hipStream_t s);

// dense product (linear.hip); `d` has its row pitches filled in
struct LinearBuffers {
  const void *x, *w, *bias, *residual;
  void *pre, *out;
};
struct LinearGrads {
  const void *x, *w, *pre, *d_out;
  void *dx, *dw, *dbias;
};
// workspace bytes of the forward product, and of the backward pass that
// computes all of its gradients
size_t linear_ws_bytes(const moe_linear_desc& d);
size_t linear_back_ws_bytes(const moe_linear_desc& d);
// for tests: tile (0 few rows, 1 64 x 128, 2 128 x 128, 3 256 x 256, 4 128 x 256) and splits of K of the forward
// product, of dx and of dw
void linear_cuts(const moe_linear_desc& d, int32_t cuts[6]);
hipError_t launch_linear(const moe_linear_desc& d, const LinearBuffers& b, void* ws, hipStream_t s);
hipError_t launch_linear_backward(const moe_linear_desc& d, const LinearGrads& b, void* ws, hipStream_t s);

// rows sorted by expert (rows.hip); `d` has its row pitches filled in
size_t sort_ws_bytes(int64_t pairs, int E);
hipError_t launch_sort(int64_t pairs, int E, int first, const int32_t* ids, int32_t* pos, int32_t* src,
                       int32_t* offsets, void* ws, hipStream_t s);
hipError_t launch_permute(const moe_rows_desc& d, const void* x, const int32_t* pos, void* rows, hipStream_t s);
hipError_t launch_unpermute(const moe_rows_desc& d, const void* rows, const int32_t* pos, const float* w, void* out,
                            hipStream_t s);
hipError_t launch_unpermute_backward(const moe_rows_desc& d, const void* rows, const int32_t* pos, const float* w,
                                     const void* d_out, void* d_rows, float* dw, hipStream_t s);

// microscaled 4-bit rows (mx.hip); pitches and `d` have their defaults filled in
hipError_t launch_mx_quantize(int64_t rows, int depth, const void* x, int dtype, int64_t ld_x, uint8_t* q, int64_t ld_q,
                              uint8_t* scale, int64_t ld_s, hipStream_t s);
hipError_t launch_mx_dequantize(int64_t rows, int depth, const uint8_t* q, int64_t ld_q, const uint8_t* scale,
                                int64_t ld_s, void* out, int dtype, int64_t ld_out, hipStream_t s);
// for tests: 0 few rows (then 16-row blocks of x, of w and wavefronts of a workgroup), 1 64 x 128, 2 128 x 128,
// 3 256 x 256, 4 128 x 256, 5 32 x 256 (x in 4 bits: 32 x 128)
void mx_choice(const moe_mx_linear_desc& d, int32_t out[4]);
hipError_t launch_mx_linear(const moe_mx_linear_desc& d, const void* x, const uint8_t* x_scale, const uint8_t* w,
                            const uint8_t* w_scale, const int32_t* offsets, const void* bias, void* out, hipStream_t s);

// the current device, checked to be a gfx950 (api.cpp); a moe_status
int prepare_device();

// Buffer descriptors: raw access of format 32, and an offset beyond every
// descriptor's extent (all below 2^31 bytes), where loads return zeros.
constexpr int kBufWord3 = 0x00020000;
constexpr uint32_t kPastEnd = 0x80000000u;

inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace moe

#endif  // MOE_EXPERT_TILE_LAYER_INTERNAL_H
