// Shared by the matrix products (linear.hip, mx.hip): operand types, direct
// loads to LDS, activations, accesses at any alignment, tile order.
#ifndef MOE_EXPERT_TILE_PRODUCT_H
#define MOE_EXPERT_TILE_PRODUCT_H

#include <type_traits>

#include "layer_internal.h"

namespace moe {
namespace {

typedef unsigned int v4u32 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)(bytes < 0 ? 0 : bytes), kBufWord3);
}

// 1 KB of global memory into LDS at `dst` (16 bytes a lane, in lane order)
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t rsrc, void* dst, uint32_t off, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void_t*)dst, 16, (int)off, soff, 0, 0);
}

// the 16-bit operand types
template <bool F16>
struct Elem {
  typedef std::conditional_t<F16, f16x8, bf16x8> v8;
  static __device__ __forceinline__ float to_float(uint16_t b) {
    if constexpr (F16) return (float)__builtin_bit_cast(_Float16, b);
    else return __uint_as_float((uint32_t)b << 16);
  }
  static __device__ __forceinline__ uint16_t bits(float f) {
    if constexpr (F16) return __builtin_bit_cast(uint16_t, (_Float16)f);
    else return __builtin_bit_cast(uint16_t, (__bf16)f);
  }
  static __device__ __forceinline__ f32x16 mfma32(v8 a, v8 b, f32x16 c) {
    if constexpr (F16) return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mfma16(v8 a, v8 b, f32x4 c) {
    if constexpr (F16) return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};

// --- activations (fp32) -----------------------------------------------------

__device__ __forceinline__ float logistic(float z) {
  return 1.0f / (1.0f + __builtin_amdgcn_exp2f(-z * 1.4426950408889634f));
}
constexpr float kSqrtHalf = 0.70710678118654752f, kInvSqrt2Pi = 0.39894228040143268f;
// gelu_tanh(z) = z (1 + tanh u) / 2 = z logistic(2 u), u = sqrt(2/pi) (z + 0.044715 z^3)
constexpr float kTwoSqrt2OverPi = 1.5957691216057308f, kCubic = 0.044715f;

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.f ? z : (z == z ? 0.f : z);
  else if constexpr (ACT == MOE_ACT_SILU) return z * logistic(z);
  else if constexpr (ACT == MOE_ACT_GELU) return 0.5f * z * (1.0f + erff(z * kSqrtHalf));
  else if constexpr (ACT == MOE_ACT_GELU_TANH) return z * logistic(kTwoSqrt2OverPi * (z + kCubic * z * z * z));
  else return z;
}
template <int W>
__device__ __forceinline__ void activate_all(int act, const float (&z)[W], float (&y)[W]) {
  auto all = [&](auto tag) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < W; ++c) y[c] = activate<decltype(tag)::value>(z[c]);
  };
  switch (act) {
    case MOE_ACT_RELU: all(std::integral_constant<int, MOE_ACT_RELU>{}); break;
    case MOE_ACT_SILU: all(std::integral_constant<int, MOE_ACT_SILU>{}); break;
    case MOE_ACT_GELU: all(std::integral_constant<int, MOE_ACT_GELU>{}); break;
    case MOE_ACT_GELU_TANH: all(std::integral_constant<int, MOE_ACT_GELU_TANH>{}); break;
    default: all(std::integral_constant<int, MOE_ACT_NONE>{}); break;
  }
}

// Whole accesses at any alignment of the element type (rows of odd lengths
// start anywhere): the global memory instructions allow it.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <class V, int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) Loose {
  V v;
};

// W = 4 or 8 values of 16 bits, of which `left` are in the row
template <bool F16, int W>
__device__ __forceinline__ void load16(const uint16_t* p, int left, float (&v)[W]) {
  typedef std::conditional_t<W == 8, u32x4, u32x2> V;
  if (left >= W) {
    const V x = ((const Loose<V, 2>*)p)->v;
#pragma unroll
    for (int c = 0; c < W; ++c) v[c] = Elem<F16>::to_float((uint16_t)(x[c / 2] >> (c % 2 * 16)));
  } else {
#pragma unroll
    for (int c = 0; c < W; ++c) v[c] = c < left ? Elem<F16>::to_float(p[c]) : 0.f;
  }
}
template <bool F16, int W, bool WHOLE = false>
__device__ __forceinline__ void store16(uint16_t* p, int left, const float (&v)[W]) {
  typedef std::conditional_t<W == 8, u32x4, u32x2> V;
  V x;
#pragma unroll
  for (int c = 0; c < W / 2; ++c)
    x[c] = (uint32_t)Elem<F16>::bits(v[2 * c]) | ((uint32_t)Elem<F16>::bits(v[2 * c + 1]) << 16);
  if (WHOLE || left >= W) {
    ((Loose<V, 2>*)p)->v = x;
  } else {
#pragma unroll
    for (int c = 0; c < W; ++c)
      if (c < left) p[c] = (uint16_t)(x[c / 2] >> (c % 2 * 16));
  }
}
// the same for fp32
template <int W>
__device__ __forceinline__ void load32(const float* p, int left, float (&v)[W]) {
  typedef float V __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int h = 0; h < W; h += 4) {
    if (left >= h + 4) {
      const V x = ((const Loose<V, 4>*)(p + h))->v;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[h + c] = x[c];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) v[h + c] = h + c < left ? p[h + c] : 0.f;
    }
  }
}
template <int W>
__device__ __forceinline__ void store32(float* p, int left, const float (&v)[W]) {
  typedef float V __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int h = 0; h < W; h += 4) {
    if (left >= h + 4) {
      ((Loose<V, 4>*)(p + h))->v = V{v[h], v[h + 1], v[h + 2], v[h + 3]};
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (h + c < left) p[h + c] = v[h + c];
    }
  }
}

// a workgroup's place in the tile order: workgroup i runs on XCD i mod 8; each
// XCD gets a contiguous run, in which 8 row tiles x 4 column tiles share their
// operands in its L2
__device__ __forceinline__ int xcd_order(int i, int total) {
  const int q = total / 8, r = total % 8, x = i % 8;
  return x * q + min(x, r) + i / 8;
}

}  // namespace
}  // namespace moe

#endif  // MOE_EXPERT_TILE_PRODUCT_H
