// Routing: router logits -> the top-k expert ids and gate weights that the
// plan and the scale step take (include/moe.h, moe_route), and the gradient
// of the weights with respect to the logits (moe_route_backward).
//
// Forward.  A row of logits is held by LPR lanes of a wavefront, VPL values
// each, so 64 / LPR tokens go through a wavefront at once.  The lanes of a row
// are divided among its expert groups (each group has the same number of
// lanes), which makes a group's best scores a reduction over neighbouring
// lanes.  Every value becomes a 64-bit key that orders by (value descending,
// expert ascending): the float's bits, remapped so that they order as an
// integer, above 10 bits of the expert's index, all in the fraction of a
// double in [1, 2), so that one v_max_f64 compares two keys.  Each lane sorts
// its keys with a fixed network of v_max_f64 / v_min_f64; then every pick is
// the largest head over the row's lanes, and the lane that held it moves its
// list up.
//
// Which values are ranked.  Without a bias the scores are an increasing
// function of the logits, so the logits themselves are ranked, exactly.  With
// a bias (or where groups are ranked by sums of scores) c = s + b is ranked in
// 32 bits; where two values that decide something lie closer than the error of
// that, the row is ranked again in 64 bits (exact_row), one row at a time by
// the whole wavefront.
//
// What bounds it: instructions.  32768 tokens x 256 experts (grouped sigmoid with
// bias, fp32) take 28 us (29-32 by the profiler) against 7 us for their bytes: about 1500 vector
// instructions a wavefront of 4 tokens, a quarter of them the picks, a fifth
// keys and sorting; the bound loads, keys and one-pass shape took it there from
// 96 us.  A late row ranked in 64 bits adds about 4 us; where every row is (scores
// closer than the bound throughout: a peaked softmax's small ones, or sigmoids of
// far negative logits, under equal biases) 32768 x 256 take 83-90 us, 109 in groups.
// 64 tokens take 3.5 us, a launch and the picks' latency.
#include <type_traits>

#include "layer_internal.h"

namespace moe {
namespace {

constexpr int kRouteThreads = 256;
// a sigmoid below this logit counts as 0 (its value would be below 2^-1009),
// so that masking with a type's lowest value leaves renormalised weights of 0
constexpr float kSigmoidZero = -700.0f;

__device__ __forceinline__ float load_as_float(const void* p, int dtype, int64_t i) {
  if (dtype == MOE_F32) return ((const float*)p)[i];
  if (dtype == MOE_BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  return (float)((const _Float16*)p)[i];
}

// VPL values of a row into z: place i at byte offset row_off + item * (chunk
// i / 4 of this lane, `step` values apart); places from cnt on are -inf.  All
// loads are issued before the first use: bounds are left to the descriptor.
template <int DT, int VPL>
__device__ __forceinline__ void load_places(__amdgpu_buffer_rsrc_t r, uint32_t row_off, int step, int cnt, bool vec,
                                            float (&z)[VPL]) {
  constexpr int ITEM = DT == MOE_F32 ? 4 : 2;
  if (vec) {
    typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
    typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
    uint32_t raw[VPL / 4][ITEM];
#pragma unroll
    for (int c = 0; c < VPL / 4; ++c) {
      const uint32_t off = 4 * c < cnt ? row_off + ITEM * c * step : kPastEnd;
      if constexpr (DT == MOE_F32) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[c][i] = v[i];
      } else {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0);
        raw[c][0] = v[0];
        raw[c][1] = v[1];
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float f;
      if constexpr (DT == MOE_F32) f = __uint_as_float(raw[i / 4][i % 4]);
      else {
        const uint32_t w = raw[i / 4][(i % 4) / 2];
        if constexpr (DT == MOE_BF16) f = __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
        else f = (float)__builtin_bit_cast(_Float16, (uint16_t)(i % 2 ? w >> 16 : w));
      }
      z[i] = i < cnt ? f : -__builtin_inff();
    }
  } else {
    uint32_t raw[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t off = i < cnt ? row_off + ITEM * ((i / 4) * step + i % 4) : kPastEnd;
      if constexpr (DT == MOE_F32) raw[i] = __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
      else raw[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float f;
      if constexpr (DT == MOE_F32) f = __uint_as_float(raw[i]);
      else if constexpr (DT == MOE_BF16) f = __uint_as_float(raw[i] << 16);
      else f = (float)__builtin_bit_cast(_Float16, (uint16_t)raw[i]);
      z[i] = i < cnt ? f : -__builtin_inff();
    }
  }
}

// One step of an all-reduce over 2 S lanes whose halves are uniform already:
// f of the two halves' values.  Within 16 lanes any exchange between the halves
// will do (mirrors); across them the swap instructions give both halves at once.
template <int S>
__device__ __forceinline__ void halves(uint32_t v, uint32_t& a, uint32_t& b) {
  a = v;
  if constexpr (S == 1) b = __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);        // quad_perm 1 0 3 2
  else if constexpr (S == 2) b = __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);   // quad_perm 2 3 0 1
  else if constexpr (S == 4) b = __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);  // row_half_mirror
  else if constexpr (S == 8) b = __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true);  // row_mirror
  else {
    const auto r = S == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                           : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  }
}
template <int S, class F>
__device__ __forceinline__ float reduce_step(float v, F f) {
  uint32_t a, b;
  halves<S>(__float_as_uint(v), a, b);
  return f(__uint_as_float(a), __uint_as_float(b));
}
template <int S, class F>
__device__ __forceinline__ double reduce_step(double v, F f) {
  const uint64_t w = __builtin_bit_cast(uint64_t, v);
  uint32_t al, bl, ah, bh;
  halves<S>((uint32_t)w, al, bl);
  halves<S>((uint32_t)(w >> 32), ah, bh);
  return f(__builtin_bit_cast(double, ((uint64_t)ah << 32) | al), __builtin_bit_cast(double, ((uint64_t)bh << 32) | bl));
}

// keys are never NaN, so the bare instructions do (the compiler's fmax first
// quiets both operands, two more instructions)
__device__ __forceinline__ double max64(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double min64(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

template <int N, int S = 1, class F, class V>
__device__ __forceinline__ V reduce_lanes(V v, F f) {
  if constexpr (S < N) return reduce_lanes<N, 2 * S>(reduce_step<S>(v, f), f);
  else return v;
}
template <int N> __device__ __forceinline__ float max_lanes(float v) {
  return reduce_lanes<N>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int N> __device__ __forceinline__ float sum_lanes(float v) {
  return reduce_lanes<N>(v, [](float a, float b) { return a + b; });
}
// Keys.  `ord` maps a float's bits to an integer of the same order (not for
// NaN); low = 1023 - expert.  A lane's place without an expert holds kKeyAbsent,
// below every value.
__device__ __forceinline__ uint32_t ord(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);   // -0 as +0
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ double make_key(float v, uint32_t low, bool there) {
  const uint32_t o = ord(v);
  const uint32_t hi = there ? (o >> 12) | 0x3ff00000u : 0x3ff00000u;   // -inf, the lowest value, has 0x7ff below the exponent
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | ((o << 20) | low));
}
constexpr double kKeyAbsent = 1.0;
__device__ __forceinline__ int key_index(double k) { return 1023 - (int)(__builtin_bit_cast(uint64_t, k) & 1023); }
__device__ __forceinline__ float key_value(double k) {
  const uint32_t o = (uint32_t)(__builtin_bit_cast(uint64_t, k) >> 20);
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// descending sort of N = 2^n values in registers (Batcher's odd-even merges)
template <int N>
__device__ __forceinline__ void sort_desc(double (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2) {
#pragma unroll
    for (int q = p; q >= 1; q /= 2) {
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q) {
#pragma unroll
        for (int i = 0; i < q; ++i) {
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const double a = v[i + j], b = v[i + j + q];
            v[i + j] = max64(a, b);
            v[i + j + q] = min64(a, b);
          }
        }
      }
    }
  }
}

__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* w;
  int64_t T, ld;
  int E, k, dtype, score, renorm, groups, gsize, keep, top2;
  float scale;
  int lpg;       // lanes per group (a power of two)
  int vec;       // four values a load: group size and row pitch multiples of 4, the base aligned
};

// One row ranked in 64 bits by the whole wavefront, c in LDS (E doubles, then
// groups doubles): the picks go to `pick` (expert, or expert | 1 << 16 for a
// masked one).  Rare, but a late one holds up the launch, so each lane keeps
// the best of its own values and only the lane that gave a pick looks again.
// Masked values are kMasked, taken ones -inf.
constexpr double kMasked = -0x1p1000;
__device__ __forceinline__ void lds_wait() {   // this wavefront's LDS accesses so far, before those that follow
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
}
__device__ __forceinline__ void exact_row(const RouteArgs& a, int64_t t, double* c, double* gs, int* pick) {
  const int lane = threadIdx.x & 63;
  constexpr double kInf = __builtin_inf();
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  const int item = a.dtype == MOE_F32 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t zr = __builtin_amdgcn_make_buffer_rsrc(
      (char*)const_cast<void*>(a.logits) + t * a.ld * item, (short)0, a.E * item, kBufWord3);
  const __amdgpu_buffer_rsrc_t br =
      __builtin_amdgcn_make_buffer_rsrc((void*)a.bias, (short)0, a.bias ? a.E * 4 : 0, kBufWord3);
  // four values a lane at a time, so that their exponentials overlap
  auto load4 = [&](int e0, float (&z)[4]) {   // experts e0 + 64 i; past the end: zeros
    uint32_t raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      raw[i] = item == 4 ? __builtin_amdgcn_raw_buffer_load_b32(zr, (e0 + 64 * i) * 4, 0, 0)
                         : (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(zr, (e0 + 64 * i) * 2, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      z[i] = a.dtype == MOE_F32 ? __uint_as_float(raw[i])
             : a.dtype == MOE_BF16 ? __uint_as_float(raw[i] << 16)
                                   : (float)__builtin_bit_cast(_Float16, (uint16_t)raw[i]);
  };
  double m = 0.0, sum = 0.0;
  if (softmax) {
    float mf = -__builtin_inff();
#pragma unroll 1
    for (int e0 = lane; e0 < a.E; e0 += 256) {
      float z[4];
      load4(e0, z);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + 64 * i < a.E) mf = fmaxf(mf, z[i]);
    }
    m = (double)max_lanes<64>(mf);
  }
#pragma unroll 1
  for (int e0 = lane; e0 < a.E; e0 += 256) {
    float z[4];
    double x[4];
    load4(e0, z);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = exp(softmax ? (double)z[i] - m : -(double)z[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e0 + 64 * i < a.E) {
        sum += x[i];
        c[e0 + 64 * i] = z[i] > -__builtin_inff() ? x[i] : -1.0;   // -1 for masked and NaN
      }
    }
  }
  if (softmax) sum = reduce_lanes<64>(sum, [](double x, double y) { return x + y; });
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const double x = c[e];
    const double b = (double)__uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(br, e * 4, 0, 0));
    const double v = (softmax ? x : 1.0) / (softmax ? sum : 1.0 + x) + b;
    c[e] = x >= 0.0 && v > -kInf ? v : kMasked;   // (a NaN compares false)
  }
  lds_wait();
  if (a.groups > 1) {
    if (lane < a.groups) {   // at most 64
      double b1 = kMasked, b2 = kMasked;
#pragma unroll 8
      for (int i = 0; i < a.gsize; ++i) {
        const double v = c[lane * a.gsize + i];
        b2 = max64(b2, min64(b1, v));
        b1 = max64(b1, v);
      }
      gs[lane] = a.top2 ? (b2 == kMasked ? kMasked : b1 + b2) : b1;
    }
    lds_wait();
    if (lane < a.groups) {
      const double mine = gs[lane];
      int better = 0;
#pragma unroll 8
      for (int o = 0; o < a.groups; ++o) better += (gs[o] > mine || (gs[o] == mine && o < lane)) ? 1 : 0;
      if (better >= a.keep)
        for (int i = 0; i < a.gsize; ++i) c[lane * a.gsize + i] = kMasked;
    }
    lds_wait();
  }
  double bv = -kInf;
  int be = 0;
  auto best_of_mine = [&]() {
    bv = -kInf;
#pragma unroll 4
    for (int e = lane; e < a.E; e += 64) {
      const double v = c[e];
      if (v > bv) { bv = v; be = e; }   // ascending: equal ones keep the lower expert
    }
  };
  best_of_mine();
  for (int j = 0; j < a.k; ++j) {
    const double top = reduce_lanes<64>(bv, [](double x, double y) { return max64(x, y); });
    const int e = -(int)reduce_lanes<64>(bv == top ? (float)-be : -1e9f, [](float x, float y) { return fmaxf(x, y); });
    if (lane == 0) pick[j] = e | (top == kMasked ? 1 << 16 : 0);
    if ((e & 63) == lane) {
      c[e] = -kInf;
      best_of_mine();
    }
  }
  lds_wait();
}

// LPR lanes a row, VPL values a lane, at most KMAX picks; BYC: c = s + b is
// ranked (else the logits)
template <int LPR, int VPL, int KMAX, bool BYC>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  constexpr int RPW = 64 / LPR;                       // rows a wavefront
  constexpr int LOOK = KMAX + (BYC ? 1 : 0);          // picks looked at: with BYC the first one left out too
  constexpr int NS = (LOOK + LPR - 1) / LPR;          // picks a lane keeps
  constexpr int DEPTH = VPL < LOOK ? VPL : LOOK;      // places of the sorted list they can come from
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l = lane % LPR;                           // lane within the row
  const int g = l / a.lpg, sub = l % a.lpg;           // its group, and place among the group's lanes
  constexpr float kInf = __builtin_inff();
  // place i of this lane is value (i / 4) * step + sub * 4 + i % 4 of its
  // group; the first cnt places exist
  const int step = 4 * a.lpg;
  const int rem = a.gsize - sub * 4;
  const int cnt = g < a.groups && rem > 0 ? rem / step * 4 + min(rem % step, 4) : 0;
  const int e0 = g * a.gsize + sub * 4;               // its first expert
  const int64_t t0 = ((int64_t)blockIdx.x * (kRouteThreads / 64) + wave) * RPW;
  if (t0 >= a.T) return;
  const int64_t t = t0 + lane / LPR;
  const bool live = t < a.T;
  const int nrows = (int)min((int64_t)RPW, a.T - t0);
  const int item = a.dtype == MOE_F32 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t zr = __builtin_amdgcn_make_buffer_rsrc(
      (char*)const_cast<void*>(a.logits) + t0 * a.ld * item, (short)0,
      (int)(((nrows - 1) * a.ld + a.E) * item), kBufWord3);
  const uint32_t zoff = (uint32_t)((lane / LPR) * (uint32_t)a.ld + e0) * item;
  const int zcnt = live ? cnt : 0;
  float z[VPL];
  if (a.dtype == MOE_F32) load_places<MOE_F32, VPL>(zr, zoff, step, zcnt, a.vec, z);
  else if (a.dtype == MOE_BF16) load_places<MOE_BF16, VPL>(zr, zoff, step, zcnt, a.vec, z);
  else load_places<MOE_F16, VPL>(zr, zoff, step, zcnt, a.vec, z);
  float bv[BYC ? VPL : 1];
  if constexpr (BYC) {
    // a.vec says the group size is a multiple of 4; four-byte alignment is all a buffer load needs
    const __amdgpu_buffer_rsrc_t br =
        __builtin_amdgcn_make_buffer_rsrc((void*)a.bias, (short)0, a.bias ? a.E * 4 : 0, kBufWord3);
    load_places<MOE_F32, VPL>(br, 4 * e0, step, cnt, a.gsize % 4 == 0, bv);
  }
  // a NaN logit (or bias), or +inf under a softmax, has no weights: the
  // row's are NaN, its ids still k distinct experts
  bool bad = false;
#pragma unroll
  for (int i = 0; i < VPL; i += 2) bad |= __builtin_isunordered(z[i], z[i + 1]);
#pragma unroll
  for (int i = 0; i < VPL; ++i) z[i] = fmaxf(z[i], -kInf);   // a NaN ranks as masked
  // the softmax's maximum and sum, where full scores are wanted
  float zmax = 0.f, zsum = 1.f;
  const bool full = a.score == MOE_SCORE_SOFTMAX && (BYC || !a.renorm);
  if (full) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, z[i]);
    m = max_lanes<LPR>(m);
    zmax = m == -kInf ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s += exp_fast(z[i] - zmax);
    zsum = fmaxf(sum_lanes<LPR>(s), 1e-30f);   // every expert masked: zero scores
  }
  // what is ranked: the logits, or c
  const float zinv = 1.0f / zsum;
  float v[VPL];
  if constexpr (BYC) {
    if (a.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = exp_fast(z[i] - zmax) * zinv;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) v[i] = __builtin_amdgcn_rcpf(1.0f + exp_fast(-z[i]));
    }
    // without a bias its buffer reads zeros, and places past cnt -inf
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const float c = v[i] + bv[i];
      bad |= z[i] != -kInf && !(c == c);
      v[i] = fmaxf(z[i] == -kInf ? -kInf : c, -kInf);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = z[i];
  }
  bool near = false;   // BYC: a decision closer than the error of 32 bits
  // Error of c in 32 bits, u = 2^-24: the sum's rounding, u |c|; a sigmoid's
  // below 4 u (its exponent's rounding times s (1 - s) |z| < 1/4, exp, 1 + e
  // and the reciprocal); a softmax's below 64 u s + u (the terms' and the
  // sum's roundings).  Two of them, with s at most smax:
  auto error2 = [&](float cmax, float smax) {
    return fmaf(0x1p-22f, cmax, a.score == MOE_SCORE_SOFTMAX ? fmaf(0x1p-17f, smax, 0x1p-22f) : 0x1p-21f);
  };
  bool kept = true;
  if (a.groups > 1) {
    float b1 = -kInf, b2 = -kInf;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      b2 = fmaxf(b2, fminf(b1, v[i]));
      b1 = fmaxf(b1, v[i]);
    }
    auto merge = [&](auto tag) {
      constexpr int S = decltype(tag)::value;
      if (S < a.lpg) {
        uint32_t x1, y1, x2, y2;
        halves<S>(__float_as_uint(b1), x1, y1);
        halves<S>(__float_as_uint(b2), x2, y2);
        b1 = fmaxf(__uint_as_float(x1), __uint_as_float(y1));
        b2 = fmaxf(fmaxf(__uint_as_float(x2), __uint_as_float(y2)), fminf(__uint_as_float(x1), __uint_as_float(y1)));
      }
    };
    merge(std::integral_constant<int, 1>{});
    if constexpr (LPR > 2) merge(std::integral_constant<int, 2>{});
    if constexpr (LPR > 4) merge(std::integral_constant<int, 4>{});
    if constexpr (LPR > 8) merge(std::integral_constant<int, 8>{});
    if constexpr (LPR > 16) merge(std::integral_constant<int, 16>{});
    if constexpr (LPR > 32) merge(std::integral_constant<int, 32>{});
    const float sc = a.top2 ? (b2 == -kInf ? -kInf : b1 + b2) : b1;   // (+inf, of a bias, and masked ones: masked)
    int better = 0;
    for (int o = 0; o < a.groups; ++o) {
      const float os = __shfl(sc, (lane - l) + o * a.lpg);
      better += (os > sc || (os == sc && o < g)) ? 1 : 0;
    }
    kept = g < a.groups && better < a.keep;
    if constexpr (BYC) {
      // lowest kept and highest dropped group; infinities differ by NaN or
      // by infinity and so are never close
      const float lo = -max_lanes<LPR>(kept ? -sc : -kInf);
      const float hi = max_lanes<LPR>(!kept && g < a.groups ? sc : -kInf);
      // (twice the scores' error for sums of two; no score exceeds the best one's, zinv)
      const float size = fabsf(b1) + (a.top2 ? fabsf(b2) : 0.f);
      const float cmax = max_lanes<LPR>(size < kInf ? size : 0.f);
      near |= lo - hi <= 2.0f * error2(cmax, zinv);
    }
  }
  double key[VPL];
  const uint32_t low = 1023 - e0;
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    key[i] = make_key(kept ? v[i] : -kInf, low - ((i / 4) * step + i % 4), i < cnt);
  sort_desc<VPL>(key);

  double slot[NS];
#pragma unroll
  for (int r = 0; r < NS; ++r) slot[r] = kKeyAbsent;
  const int picks = BYC && a.k < a.E ? a.k + 1 : a.k;   // one more to see how near the first one left out lies
  for (int j = 0; j < picks; ++j) {
    const double best = reduce_lanes<LPR>(key[0], [](double x, double y) { return max64(x, y); });
#pragma unroll
    for (int r = 0; r < NS; ++r)
      if (j == r * LPR + l) slot[r] = best;
    // (a branch, not a select an element: that became indexed reads of the list)
    if (key[0] == best) {
#pragma unroll
      for (int i = 0; i + 1 < DEPTH; ++i) key[i] = key[i + 1];
      // the list's last place: once it has been picked nothing is left in it
      if constexpr (DEPTH == VPL) key[DEPTH - 1] = kKeyAbsent;
    }
  }
  int pick[NS];
#pragma unroll
  for (int r = 0; r < NS; ++r)
    pick[r] = key_index(slot[r]) | (key_value(slot[r]) == -kInf ? 1 << 16 : 0);
  float zpick[NS], bpick[NS];   // the picks' logits, and with BYC biases
  if constexpr (!BYC) {
#pragma unroll
    for (int r = 0; r < NS; ++r) zpick[r] = key_value(slot[r]);
  } else {
    // neighbours among the picks that are close, unless their logits and
    // biases are the same and the index decides (zero biases over 16-bit
    // logits are full of those).  The last pick and the first one left out are
    // held against the largest error of any score (`edge`): what is left out
    // further down may have a larger score, and error, than they have.
    bool edge = false;
    float pc = kInf, pz = 0.f, pb = 0.f, ps = 0.f;   // the last lane's pick of the previous round
#pragma unroll
    for (int r = 0; r < NS; ++r) {
      const int j = r * LPR + l;
      const bool on = live && j < picks;
      const float c = key_value(slot[r]);
      const float zj = on ? load_as_float(a.logits, a.dtype, t * a.ld + (pick[r] & 0xffff)) : 0.f;
      zpick[r] = zj;
      const float bj = on && a.bias ? a.bias[pick[r] & 0xffff] : 0.f;
      bpick[r] = bj;
      const float sj = exp_fast(zj - zmax) * zinv;   // of a softmax
      float qc = __shfl_up(c, 1, LPR), qz = __shfl_up(zj, 1, LPR), qb = __shfl_up(bj, 1, LPR);
      float qs = __shfl_up(sj, 1, LPR);
      if (l == 0) { qc = pc; qz = pz; qb = pb; qs = ps; }
      // (an infinite c, of a bias, is exact)
      if (j < a.k) near |= on && j > 0 && qc < kInf && qc - c <= error2(fabsf(qc), fmaxf(qs, sj)) && !(qz == zj && qb == bj);
      else edge |= on && qc < kInf && qc - c <= error2(fabsf(qc), zinv);
      if constexpr (NS > 1) {
        pc = __shfl(c, LPR - 1, LPR);
        pz = __shfl(zj, LPR - 1, LPR);
        pb = __shfl(bj, LPR - 1, LPR);
        ps = __shfl(sj, LPR - 1, LPR);
      }
    }
    if (__ballot(edge)) {
      // Everything left out within reach of the last pick, by its own error
      // then: the first one, and what the lanes' lists still hold (copies
      // that moving up left at a list's end are not below the last pick, or
      // are looked at twice).
      edge = max_lanes<LPR>(near ? 2.f : edge ? 1.f : 0.f) == 1.f;   // (not where the row is ranked again anyway)
      const int at = (lane - l) + (a.k - 1) % LPR;
      double last = kKeyAbsent;
      float zk = 0.f, bk = 0.f;
#pragma unroll
      for (int r = 0; r < NS; ++r) {
        if ((a.k - 1) / LPR == r) {
          last = __shfl(slot[r], at);
          zk = __shfl(zpick[r], at);
          bk = __shfl(bpick[r], at);
        }
      }
      const float ck = key_value(last);
      const float low = ck - 0.5f * error2(fabsf(ck), exp_fast(zk - zmax) * zinv);
      auto reaches = [&](float c, float s) { return c + 0.5f * error2(fabsf(c), s) >= low; };
      auto look = [&](float c, float zc, float bc) {
        if (reaches(c, exp_fast(zc - zmax) * zinv) && !(zc == zk && bc == bk)) near = true;
      };
#pragma unroll
      for (int r = 0; r < NS; ++r)
        if (edge && r * LPR + l == a.k) look(key_value(slot[r]), zpick[r], bpick[r]);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const float c = key_value(key[i]);
        if (edge && key[i] < last && reaches(c, zinv)) {
          const int e = key_index(key[i]);
          look(c, load_as_float(a.logits, a.dtype, t * a.ld + e), a.bias ? a.bias[e] : 0.f);
        }
      }
    }
    near = max_lanes<LPR>(near ? 1.f : 0.f) > 0.f;
    double* cbuf = (double*)smem + (size_t)wave * (a.E + a.groups + 16 + 1);
    double* gbuf = cbuf + a.E;
    int* pbuf = (int*)(gbuf + a.groups);
    uint64_t todo = __ballot(near && live && l == 0);
    while (todo) {
      const int at = __ffsll((unsigned long long)todo) - 1;
      todo &= todo - 1;
      exact_row(a, t0 + at / LPR, cbuf, gbuf, pbuf);
      if (lane / LPR == at / LPR) {
#pragma unroll
        for (int r = 0; r < NS; ++r)
          if (r * LPR + l < a.k) {
            pick[r] = pbuf[r * LPR + l];
            zpick[r] = load_as_float(a.logits, a.dtype, t * a.ld + (pick[r] & 0xffff));
          }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
  // weights of the picks
  float p[NS], zs[NS];
  float top = -kInf;
#pragma unroll
  for (int r = 0; r < NS; ++r) {
    const bool on = live && r * LPR + l < a.k && !(pick[r] >> 16);
    zs[r] = on ? zpick[r] : -kInf;
    top = fmaxf(top, zs[r]);
  }
  if (a.score == MOE_SCORE_SOFTMAX) bad |= top == kInf;
  const bool nan_row = max_lanes<LPR>(bad ? 1.f : 0.f) > 0.f;
  float total = 0.f;
  if (a.renorm) {
    // the weights' ratios need no common factor: the softmax's maximum is
    // taken over the picks, and sigmoids of far negative logits are scaled
    // up by e^-top, so that the sum does not vanish in 32 bits
    top = max_lanes<LPR>(top);
    const float shift = a.score == MOE_SCORE_SOFTMAX ? (top == -kInf ? 0.f : top) : fminf(0.f, top == -kInf ? 0.f : top);
#pragma unroll
    for (int r = 0; r < NS; ++r) {
      float q;
      if (zs[r] == -kInf) q = 0.f;
      else if (a.score == MOE_SCORE_SOFTMAX) q = expf(zs[r] - shift);
      else if (zs[r] < kSigmoidZero) q = 0.f;
      else q = zs[r] > 0.f ? 1.0f / (1.0f + expf(-zs[r])) : expf(zs[r] - shift) / (1.0f + expf(zs[r]));
      p[r] = q;
      total += q;
    }
    total = sum_lanes<LPR>(total);
  } else {
#pragma unroll
    for (int r = 0; r < NS; ++r) {
      if (zs[r] == -kInf) p[r] = 0.f;
      else if (a.score == MOE_SCORE_SOFTMAX) p[r] = expf(zs[r] - zmax) / zsum;
      else p[r] = 1.0f / (1.0f + expf(-zs[r]));
    }
  }
#pragma unroll
  for (int r = 0; r < NS; ++r) {
    const int j = r * LPR + l;
    if (live && j < a.k) {
      float wj = a.renorm ? (total > 0.f ? p[r] / total : 0.f) : p[r];
      wj *= a.scale;
      a.ids[t * a.k + j] = pick[r] & 0xffff;
      a.w[t * a.k + j] = nan_row ? __builtin_nanf("") : wj;
    }
  }
}

// --- backward ---------------------------------------------------------------
//
// ids, a bias and slots of weight 0 are constants.  With p the weights before
// the factor, S their sum and g the gradient of the weights:
//   softmax, renormalised:  dz_j = w_j (g_j - D / scale),      D = sum_i g_i w_i
//   softmax:                dz_e = [e = id_j] w_j g_j - s_e D
//   sigmoid, renormalised:  dz_j = w_j (1 - s_j) (g_j - D / scale)
//   sigmoid:                dz_j = w_j (1 - s_j) g_j
// (a sigmoid's slope is s (1 - s), and 1 - s_j = 1 / (1 + e^z_j)).  So only
// the full softmax reads whole rows of logits; the others read k of them.
// A wavefront builds its rows in LDS (zeros, then the k values, summed in slot
// order where an expert is listed twice) and writes them out whole.  Bound by
// those writes: 32768 x 256 fp32, 37 MB with the slots, take 10-11 us, 3.5
// TB/s; with the full softmax, which reads as much again, 16.5 us, 4.3 TB/s (bf16
// 11.5 us); 256 x 8 with the full softmax take 3.7 us, a launch.
struct RouteBackArgs {
  const void* logits;
  const int32_t* ids;
  const float* w;
  const float* dw;
  void* dz;
  int64_t T, ld, ldd;
  int E, k, dtype, score, renorm;
  float scale;
  int rows;   // rows a wavefront builds at once, at most 64 / SL
  int pitch;  // floats between them in LDS
  int vec;    // four values a store: E and ldd multiples of 4, the base aligned
  int zvec;   // ... and a load: E and ld, likewise
};

__device__ __forceinline__ void store_as(void* p, int dtype, int64_t i, float v) {
  if (dtype == MOE_F32) ((float*)p)[i] = v;
  else if (dtype == MOE_BF16) ((__bf16*)p)[i] = (__bf16)v;
  else ((_Float16*)p)[i] = (_Float16)v;
}
__device__ __forceinline__ void store4_as(void* p, int dtype, int64_t i, const float4& v) {
  if (dtype == MOE_F32) {
    *(float4*)((float*)p + i) = v;
  } else if (dtype == MOE_BF16) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    *(bf16x4*)((__bf16*)p + i) = bf16x4{(__bf16)v.x, (__bf16)v.y, (__bf16)v.z, (__bf16)v.w};
  } else {
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    *(f16x4*)((_Float16*)p + i) = f16x4{(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w};
  }
}

// Rows t0 .. t0 + n - 1 of the full softmax's gradient, tile - s dot, by SL
// lanes a row: its maximum and sum in one pass over the logits, 16 values a lane
// at a time, and the result in a second one (from registers where 16 SL values
// hold the row).
template <int DT, int SL>
__device__ __forceinline__ void full_softmax(const RouteBackArgs& a, int64_t t0, int n, float dot, const float* tile) {
  constexpr int V = 16;
  constexpr float kInf = __builtin_inff();
  const int lane = threadIdx.x & 63, row = lane / SL, j = lane % SL;
  const int item = DT == MOE_F32 ? 4 : 2;
  const __amdgpu_buffer_rsrc_t zr = __builtin_amdgcn_make_buffer_rsrc(
      (char*)const_cast<void*>(a.logits) + t0 * a.ld * item, (short)0, (int)(((n - 1) * a.ld + a.E) * item), kBufWord3);
  const int chunks = (a.E + V * SL - 1) / (V * SL);
  float z[V];
  // values e0 + (i / 4) * 4 SL + i % 4 of the row
  auto load = [&](int chunk) {
    const int e0 = chunk * V * SL + 4 * j, rem = a.E - e0;
    const int cnt = row < n && rem > 0 ? min(rem / (4 * SL) * 4 + min(rem % (4 * SL), 4), V) : 0;
    load_places<DT, V>(zr, (uint32_t)(row * (uint32_t)a.ld + e0) * item, 4 * SL, cnt, a.zvec, z);
    return cnt;
  };
  float m = -kInf, s = 0.f;
  int cnt = 0;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    cnt = load(c);
    float top = m;
#pragma unroll
    for (int i = 0; i < V; ++i) top = fmaxf(top, z[i]);
    if (top > -kInf) {
      s = m > -kInf ? s * exp_fast(m - top) : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s += exp_fast(z[i] - top);
    }
    m = top;
  }
  const float all = max_lanes<SL>(m);
  const float base = all == -kInf ? 0.f : all;
  s = sum_lanes<SL>(m > -kInf ? s * exp_fast(m - base) : 0.f);
  const float f = s == 0.f ? 0.f * dot : dot / s;   // every expert masked: no gradient (of a NaN row NaN)
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) cnt = load(c);
    const int e0 = c * V * SL + 4 * j;
    const int64_t out = (t0 + row) * a.ldd;
    const float* g = tile + row * a.pitch;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const int e = e0 + i * SL;
      if (i >= cnt) continue;
      const float4 h = *(const float4*)(g + e);   // (the pitch is a multiple of 4)
      const float4 v = make_float4(h.x - f * exp_fast(z[i] - base), h.y - f * exp_fast(z[i + 1] - base),
                                   h.z - f * exp_fast(z[i + 2] - base), h.w - f * exp_fast(z[i + 3] - base));
      if (a.vec) {
        store4_as(a.dz, a.dtype, out + e, v);
      } else {
        store_as(a.dz, a.dtype, out + e, v.x);
        if (i + 1 < cnt) store_as(a.dz, a.dtype, out + e + 1, v.y);
        if (i + 2 < cnt) store_as(a.dz, a.dtype, out + e + 2, v.z);
        if (i + 3 < cnt) store_as(a.dz, a.dtype, out + e + 3, v.w);
      }
    }
  }
}

// SL lanes hold the slots of a row (k <= SL)
template <int SL>
__global__ __launch_bounds__(kRouteThreads) void route_back_kernel(RouteBackArgs a) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  float* tile = (float*)smem + (size_t)wave * a.rows * a.pitch;
  const int row = lane / SL, j = lane % SL;
  const int64_t t0 = ((int64_t)blockIdx.x * (kRouteThreads / 64) + wave) * a.rows;
  if (t0 >= a.T) return;
  const int64_t t = t0 + row;
  const int n = (int)min((int64_t)a.rows, a.T - t0);
  const bool on = row < n && j < a.k;
  int id = -1;
  float w = 0.f, g = 0.f, z = 0.f;
  if (on) {
    id = a.ids[t * a.k + j];
    w = a.w[t * a.k + j];
    if (id < 0 || id >= a.E || w == 0.f) id = -1;   // constants, or no expert at all
    if (id >= 0) {
      g = a.dw[t * a.k + j];
      if (a.score == MOE_SCORE_SIGMOID) z = load_as_float(a.logits, a.dtype, t * a.ld + id);
    } else {
      w = 0.f;
    }
  }
  for (int i = lane * 4; i < n * a.pitch; i += 256) *(float4*)(tile + i) = make_float4(0.f, 0.f, 0.f, 0.f);
  lds_wait();
  float dot = id >= 0 ? g * w : 0.f;
  dot = sum_lanes<SL>(dot);
  float v = 0.f;
  if (id >= 0) {
    v = a.renorm ? w * (g - dot / a.scale) : w * g;
    if (a.score == MOE_SCORE_SIGMOID) v *= 1.0f / (1.0f + expf(z));
  }
  // an expert listed in several slots: the first of them adds all up
  float total = 0.f;
  bool first = true;
  for (int i = 0; i < a.k; ++i) {
    const int oid = __shfl(id, row * SL + i);
    const float ov = __shfl(v, row * SL + i);
    if (oid == id) {
      total += ov;
      if (i < j) first = false;
    }
  }
  if (id >= 0 && first) tile[row * a.pitch + id] = total;
  lds_wait();
  if (a.score == MOE_SCORE_SOFTMAX && !a.renorm) {
    // the other part of the full softmax, - s_e D: SL lanes a row
    if (a.dtype == MOE_F32) full_softmax<MOE_F32, SL>(a, t0, n, dot, tile);
    else if (a.dtype == MOE_BF16) full_softmax<MOE_BF16, SL>(a, t0, n, dot, tile);
    else full_softmax<MOE_F16, SL>(a, t0, n, dot, tile);
    return;
  }
  if (row >= n) return;
  const float* from = tile + row * a.pitch;
  const int64_t to = t * a.ldd;
  if (a.vec) {
    for (int e = 4 * j; e < a.E; e += 4 * SL) store4_as(a.dz, a.dtype, to + e, *(const float4*)(from + e));
  } else {
    for (int e = j; e < a.E; e += SL) store_as(a.dz, a.dtype, to + e, from[e]);
  }
}

// Workgroups of one launch: a launch's threads are counted in 32 bits, and 64
// lanes a row make 2^32 of them for the 2^26 tokens a call may have, so such a
// batch takes two launches.
constexpr int64_t kLaunchBlocks = 1 << 23;
static_assert(kLaunchBlocks * kRouteThreads < (1ll << 32), "threads of a launch");

template <int LPR, int VPL>
void launch_route_k(const RouteArgs& all, bool byc, hipStream_t s) {
  constexpr int RPW = 64 / LPR, WPB = kRouteThreads / 64;
  const size_t lds = byc ? (size_t)WPB * (all.E + all.groups + 16 + 1) * 8 : 0;
  for (int64_t t0 = 0; t0 < all.T; t0 += kLaunchBlocks * RPW * WPB) {
    RouteArgs a = all;
    a.T = all.T - t0 < kLaunchBlocks * RPW * WPB ? all.T - t0 : kLaunchBlocks * RPW * WPB;
    a.logits = (const char*)all.logits + t0 * all.ld * (all.dtype == MOE_F32 ? 4 : 2);
    a.ids += t0 * all.k;
    a.w += t0 * all.k;
    const unsigned grid = (unsigned)((a.T + RPW * WPB - 1) / (RPW * WPB));
    if (a.k <= 8) {
      if (byc) hipLaunchKernelGGL((route_kernel<LPR, VPL, 8, true>), dim3(grid), dim3(kRouteThreads), lds, s, a);
      else hipLaunchKernelGGL((route_kernel<LPR, VPL, 8, false>), dim3(grid), dim3(kRouteThreads), 0, s, a);
    } else {
      if (byc) hipLaunchKernelGGL((route_kernel<LPR, VPL, 32, true>), dim3(grid), dim3(kRouteThreads), lds, s, a);
      else hipLaunchKernelGGL((route_kernel<LPR, VPL, 32, false>), dim3(grid), dim3(kRouteThreads), 0, s, a);
    }
  }
}

}  // namespace

hipError_t launch_route(int64_t T, int E, int k, const void* logits, int dtype, int64_t ld, const float* bias,
                        const moe_route_opts& o, int32_t* ids, float* w, hipStream_t s) {
  RouteArgs a;
  a.logits = logits; a.bias = bias; a.ids = ids; a.w = w;
  a.T = T; a.ld = ld; a.E = E; a.k = k; a.dtype = dtype;
  a.score = o.score; a.renorm = o.renorm;
  a.groups = o.n_group; a.gsize = E / o.n_group; a.keep = o.topk_group;
  a.top2 = o.n_group > 1 && o.group_score == MOE_GROUP_TOP2;
  a.scale = o.scale;
  const size_t item = dtype == MOE_F32 ? 4 : 2;
  a.vec = a.gsize % 4 == 0 && ld % 4 == 0 && aligned_to(logits, 4 * item);
  const bool byc = bias != nullptr || a.top2;
  int gp = 1;
  while (gp < a.groups) gp *= 2;
  // Lanes a row.  Fewer hold more values each: more sorting, but a pick's
  // exchanges serve more rows.  At most 16 values a lane, and at least 8 lanes
  // past 16 experts.  Over 65 to 128 experts 16 lanes are quicker for a short
  // batch and 8 for a long one (128 experts, without bias: 64 tokens 3.7 and 4.4
  // us, 12288 5.6 and 6.1, 16384 6.4 and 6.3, 24576 8.3 and 7.4, 32768 10.0 and
  // 8.6; with one 64 tokens 4.9 and 6.4 us, 12288 10.2 and 10.9, 16384 12.8 and
  // 12.8, 24576 13.6 and 14.3, 32768 15.4 and 14.9); 32 lanes are slower for both (5.6 and
  // 35 us), and for 256 experts (5.7 and 36.5 us against 5.6 and 21.7 us with 16).
  auto places = [&](int lpr) { return (a.gsize + 4 * (lpr / gp) - 1) / (4 * (lpr / gp)) * 4; };
  int lpr = gp < 4 ? 4 : gp;
  if (E > 16 && lpr < 8) lpr = 8;
  if (E > 64 && lpr < 16 && T < 16384) lpr = 16;
  while (lpr < 64 && places(lpr) > (lpr == 4 ? 4 : 16)) lpr *= 2;
  const int vpl = places(lpr);
  a.lpg = lpr / gp;
  if (lpr == 4) launch_route_k<4, 4>(a, byc, s);
  else if (lpr == 8 && vpl <= 8) launch_route_k<8, 8>(a, byc, s);
  else if (lpr == 8) launch_route_k<8, 16>(a, byc, s);
  else if (lpr == 16 && vpl <= 8) launch_route_k<16, 8>(a, byc, s);
  else if (lpr == 16) launch_route_k<16, 16>(a, byc, s);
  else if (lpr == 32) launch_route_k<32, 16>(a, byc, s);
  else if (vpl <= 16) launch_route_k<64, 16>(a, byc, s);
  else launch_route_k<64, 32>(a, byc, s);
  return hipGetLastError();
}

hipError_t launch_route_backward(int64_t T, int E, int k, const void* logits, int dtype, int64_t ld,
                                 const int32_t* ids, const float* w, const float* dw, const moe_route_opts& o,
                                 void* dz, int64_t ldd, hipStream_t s) {
  RouteBackArgs a;
  a.logits = logits; a.ids = ids; a.w = w; a.dw = dw; a.dz = dz;
  a.T = T; a.ld = ld; a.ldd = ldd; a.E = E; a.k = k; a.dtype = dtype;
  a.score = o.score; a.renorm = o.renorm; a.scale = o.scale;
  const size_t item = dtype == MOE_F32 ? 4 : 2;
  a.vec = E % 4 == 0 && ldd % 4 == 0 && aligned_to(dz, 4 * item);
  a.zvec = E % 4 == 0 && ld % 4 == 0 && aligned_to(logits, 4 * item);
  a.pitch = (E + 3) / 4 * 4;
  const int sl = k <= 8 ? 8 : 32;
  // up to 8 KB of rows a wavefront
  int rows = 2048 / a.pitch;
  rows = rows < 1 ? 1 : rows;
  a.rows = rows < 64 / sl ? rows : 64 / sl;
  constexpr int WPB = kRouteThreads / 64;
  const size_t lds = (size_t)WPB * a.rows * a.pitch * 4;
  // (two rows a wavefront at least: 2^31 threads for 2^26 tokens)
  const unsigned grid = (unsigned)((T + (int64_t)a.rows * WPB - 1) / ((int64_t)a.rows * WPB));
  if (sl == 8) hipLaunchKernelGGL((route_back_kernel<8>), dim3(grid), dim3(kRouteThreads), lds, s, a);
  else hipLaunchKernelGGL((route_back_kernel<32>), dim3(grid), dim3(kRouteThreads), lds, s, a);
  return hipGetLastError();
}

}  // namespace moe
