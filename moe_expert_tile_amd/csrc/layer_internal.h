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

// the current device, checked to be a gfx950 (api.cpp); a moe_status
int prepare_device();

// Buffer descriptors: raw access of format 32, and an offset beyond every
// descriptor's extent (all below 2^31 bytes), where loads return zeros.
constexpr int kBufWord3 = 0x00020000;
constexpr uint32_t kPastEnd = 0x80000000u;

inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace moe

#endif  // MOE_EXPERT_TILE_LAYER_INTERNAL_H
