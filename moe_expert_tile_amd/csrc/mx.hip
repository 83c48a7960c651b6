// Microscaled 4-bit rows (include/moe.h): moe_mx_quantize, moe_mx_dequantize and
// the product with 4-bit weights, expert by expert (moe_mx_linear).
//
// A row is elements of sign, two exponent bits and one fraction bit (0, 0.5, 1,
// 1.5, 2, 3, 4, 6), two a byte, and a power of two for every 32 of them, held as
// its exponent plus 127 in a byte (255: not a number).
//
// The product out[r] = act(x[r] w[e]^T + bias[e]), e the expert of row r, sums in
// fp32 MFMA registers.
//   * x in 16 bits: the weights are converted on their way from memory to the
//     matrix cores (v_cvt_scalef32_pk_*_fp4, a pair and its scale an instruction),
//     which then take 16-bit operands; bf16 holds every weight exactly.
//   * x in 4 bits too: v_mfma_scale_* take both as they are, with a scale byte a
//     lane and operand.
// Lanes of an MFMA may sum over any elements as long as both operands agree, so
// a lane always takes whole blocks of 32: 16 bytes of a row, one scale.
// The first MFMA operand is the weights', so a lane ends with 4 consecutive
// output columns per accumulator quad.
#include "product.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// 2^(s - 127) as v_cvt_scalef32_* take it: they read the exponent bits alone,
// so that s = 0 is 2^-127 and 255 not a number
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(s << 23); }

// eight 4-bit elements times a scale in a 16-bit type
template <bool F16>
__device__ __forceinline__ v4u32 widen(uint32_t q, float scale) {
  v4u32 r;
  if constexpr (F16) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, scale, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, scale, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, scale, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, scale, 3));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3));
  }
  return r;
}

// --- quantisation -------------------------------------------------------------
//
// Four neighbouring lanes share a block, eight elements each.  The largest
// magnitude is found among bit patterns (infinities and NaN are above all
// numbers that way), across the lanes by two DPP moves.  v_cvt_scalef32_pk_fp4_*
// round to the nearest element, ties to the even one, and saturate at 6.

struct QuantArgs {
  const char* x;
  uint8_t *q, *scale;
  int64_t n8;                       // groups of 8 elements in a row
  int64_t rows, ld_x, ld_q, ld_s;   // bytes
};

constexpr int kQuantUnroll = 4;

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));    // lanes 1 0 3 2
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true)); // lanes 2 3 0 1
}

template <int T>
__global__ __launch_bounds__(256) void quantize_kernel(QuantArgs a) {
  constexpr int W = T == MOE_F32 ? 2 : 1;   // 16-byte loads of 8 elements
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    for (int64_t i0 = (int64_t)blockIdx.x * 256 * kQuantUnroll + threadIdx.x; i0 < a.n8;
         i0 += (int64_t)gridDim.x * 256 * kQuantUnroll) {
      v4u32 v[kQuantUnroll][W];
#pragma unroll
      for (int u = 0; u < kQuantUnroll; ++u) {
        const int64_t i = i0 + 256 * u;
#pragma unroll
        for (int h = 0; h < W; ++h)
          v[u][h] = i < a.n8 ? ((const Loose<v4u32, T == MOE_F32 ? 4 : 2>*)(a.x + r * a.ld_x + (i * W + h) * 16))->v
                             : v4u32{0, 0, 0, 0};
      }
#pragma unroll
      for (int u = 0; u < kQuantUnroll; ++u) {
        const int64_t i = i0 + 256 * u;
        if (i >= a.n8) continue;      // whole blocks of four lanes
        uint32_t top = 0;
#pragma unroll
        for (int h = 0; h < W; ++h)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t b = v[u][h][c];
            if constexpr (T == MOE_F32) top = max(top, b & 0x7fffffffu);
            else top = max(top, max(b & 0x7fffu, (b >> 16) & 0x7fffu));
          }
        top = quad_max(top);
        // exponent bits of the largest one in fp32
        int e;
        if constexpr (T == MOE_F32) e = (int)(top >> 23);
        else if constexpr (T == MOE_BF16) e = (int)(top >> 7);
        else e = (int)(__float_as_uint(Elem<true>::to_float((uint16_t)top)) >> 23);
        const int s = e == 255 ? 255 : max(e - 2, 0);
        const float scale = __uint_as_float(max((uint32_t)s << 23, 0x00400000u));
        uint32_t q = 0;
        if (s < 255) {
          if constexpr (T == MOE_F32) {
            const v4u32 lo = v[u][0], hi = v[u][W - 1];
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(lo[0]), __uint_as_float(lo[1]), scale, 0);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(lo[2]), __uint_as_float(lo[3]), scale, 1);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(hi[0]), __uint_as_float(hi[1]), scale, 2);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(hi[2]), __uint_as_float(hi[3]), scale, 3);
          } else {
            const uint32_t p0 = v[u][0][0], p1 = v[u][0][1], p2 = v[u][0][2], p3 = v[u][0][3];
            if constexpr (T == MOE_BF16) {
              q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p0), scale, 0);
              q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p1), scale, 1);
              q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p2), scale, 2);
              q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, p3), scale, 3);
            } else {
              q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, p0), scale, 0);
              q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, p1), scale, 1);
              q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, p2), scale, 2);
              q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, p3), scale, 3);
            }
          }
        }
        *(uint32_t*)(a.q + r * a.ld_q + i * 4) = q;
        if (threadIdx.x % 4 == 0) a.scale[r * a.ld_s + i / 4] = (uint8_t)s;
      }
    }
  }
}

template <int T>
__global__ __launch_bounds__(256) void dequantize_kernel(QuantArgs a) {
  constexpr int W = T == MOE_F32 ? 2 : 1;
  char* out = const_cast<char*>(a.x);
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    for (int64_t i0 = (int64_t)blockIdx.x * 256 * kQuantUnroll + threadIdx.x; i0 < a.n8;
         i0 += (int64_t)gridDim.x * 256 * kQuantUnroll) {
      uint32_t q[kQuantUnroll], s[kQuantUnroll];
#pragma unroll
      for (int u = 0; u < kQuantUnroll; ++u) {
        const int64_t i = i0 + 256 * u;
        q[u] = i < a.n8 ? *(const uint32_t*)(a.q + r * a.ld_q + i * 4) : 0;
        s[u] = i < a.n8 ? a.scale[r * a.ld_s + i / 4] : 0;
      }
#pragma unroll
      for (int u = 0; u < kQuantUnroll; ++u) {
        const int64_t i = i0 + 256 * u;
        if (i >= a.n8) continue;
        const float scale = scale_of(s[u]);
        v4u32 v[W];
        if constexpr (T == MOE_F32) {
          const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], scale, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], scale, 1);
          const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], scale, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], scale, 3);
          v[0] = v4u32{__float_as_uint(p0[0]), __float_as_uint(p0[1]), __float_as_uint(p1[0]), __float_as_uint(p1[1])};
          v[W - 1] = v4u32{__float_as_uint(p2[0]), __float_as_uint(p2[1]), __float_as_uint(p3[0]), __float_as_uint(p3[1])};
        } else {
          v[0] = widen<T == MOE_F16>(q[u], scale);
        }
#pragma unroll
        for (int h = 0; h < W; ++h)
          ((Loose<v4u32, T == MOE_F32 ? 4 : 2>*)(out + r * a.ld_x + (i * W + h) * 16))->v = v[h];
      }
    }
  }
}

// --- product --------------------------------------------------------------------

struct MxArgs {
  const char *x, *w;
  const uint8_t *xs, *ws;
  const int32_t* offsets;          // null: one expert, all rows
  const void* bias;                // [experts, n] of the output's type, or null
  char* out;
  int64_t ld_x, ld_xs, ld_w, ld_ws, expert_w, expert_ws;   // bytes
  int64_t ld_out;                  // elements
  int64_t rows;
  int E, N, K, act, out_type;
  int nt0, n_nt;                   // column tiles of this launch: the first one, their number
};

struct RowTile {
  int expert, count;               // count: rows of the tile, 0 if there is none
  int64_t row;
};

// Row tile t of the experts' rows cut into pieces of bm, none of which holds
// rows of two experts.  Offsets out of order or out of range give other rows, but
// none outside [0, rows).  Called by whole wavefronts.
__device__ __forceinline__ RowTile find_tile(const MxArgs& a, int bm, int t) {
  const int rows = (int)a.rows;
  if (!a.offsets) {
    const int64_t row = (int64_t)t * bm;
    return {0, row < rows ? min(bm, (int)(rows - row)) : 0, row};
  }
  const int lane = threadIdx.x & 63;
  int done = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    const int e = e0 + lane;
    const int lo = e < a.E ? min(max(a.offsets[e], 0), rows) : 0;
    const int hi = e < a.E ? min(max(a.offsets[e + 1], 0), rows) : 0;
    const int n = hi > lo ? (hi - lo + bm - 1) / bm : 0;
    int upto = n;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int o = __shfl_up(upto, s);
      if (lane >= s) upto += o;
    }
    const int all = __shfl(upto, 63);
    if (t < done + all) {
      const uint64_t past = __ballot(t < done + upto);
      const int l = __builtin_ctzll(past);
      const int first = __shfl(lo, l), last = __shfl(hi, l), before = done + __shfl(upto - n, l);
      const int row = first + (t - before) * bm;
      return {e0 + l, min(bm, last - row), row};
    }
    done += all;
  }
  return {0, 0, 0};
}

// Columns n .. n + 3 of a row and their bias, of which `left` exist
__device__ __forceinline__ void load4(int type, const void* base, int64_t at, int left, float (&v)[4]) {
  if (type == MOE_F32) load32((const float*)base + at, left, v);
  else if (type == MOE_F16) load16<true>((const uint16_t*)base + at, left, v);
  else load16<false>((const uint16_t*)base + at, left, v);
}
template <int W>
__device__ __forceinline__ void store_row(int type, char* base, int64_t at, int left, const float (&v)[W]) {
  if (type == MOE_F32) store32((float*)base + at, left, v);
  else if (type == MOE_F16) store16<true>((uint16_t*)base + at, left, v);
  else store16<false>((uint16_t*)base + at, left, v);
}

// --- few rows -------------------------------------------------------------------
//
// Bound by reading the weights, which every (row tile, column tile) workgroup
// does once, straight into operand registers.  A workgroup owns 16 TT rows of
// one expert and 16 NB output columns (gated: 16 NB gate and up rows of w); its
// wavefronts take K in steps of 128 in turn and join their sums in LDS.
// Operand lane layout: row lane % 16, block lane / 16 of a step; with 16-bit
// operands dword i of the block is the lane's part of the step's i-th
// v_mfma_f32_16x16x32.  Result lane: row (of x) lane % 16, columns 4 (lane / 16) .. + 3.
constexpr int kFewWaves = 8;

template <int XT, bool GATED, int TT, int NB, int U>
__global__ __launch_bounds__(kFewWaves * 64) void few_rows_kernel(MxArgs a) {
  constexpr bool MX = XT == MOE_MXFP4, F16 = XT == MOE_F16;
  constexpr int G = GATED ? 2 : 1, XL = MX ? 1 : 4;      // 16-byte loads of a block of x
  __shared__ float4 part[kFewWaves][G * NB][TT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int n_nt = a.n_nt;
  const RowTile tile = find_tile(a, 16 * TT, blockIdx.x / n_nt);
  const int expert = __builtin_amdgcn_readfirstlane(tile.expert), rows = __builtin_amdgcn_readfirstlane(tile.count);
  const int64_t row0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)tile.row);
  if (rows <= 0) return;
  const int n0 = (a.nt0 + (int)(blockIdx.x % n_nt)) * 16 * NB;
  const int r = lane & 15, g = lane >> 4;
  const int cols = min(16 * NB, a.N - n0);
  const char* w = a.w + expert * a.expert_w + n0 * a.ld_w;
  const uint8_t* ws = a.ws + expert * a.expert_ws + n0 * a.ld_ws;
  __amdgpu_buffer_rsrc_t wr[G], sr[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    wr[h] = make_rsrc(w + (int64_t)h * a.N * a.ld_w, (cols - 1) * a.ld_w + a.K / 2);
    sr[h] = make_rsrc(ws + (int64_t)h * a.N * a.ld_ws, (cols - 1) * a.ld_ws + a.K / 32);
  }
  const int row_bytes = MX ? a.K / 2 : a.K * 2;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + row0 * a.ld_x, (rows - 1) * a.ld_x + row_bytes);
  const __amdgpu_buffer_rsrc_t xsr = make_rsrc(MX ? a.xs + row0 * a.ld_xs : nullptr, MX ? (rows - 1) * a.ld_xs + a.K / 32 : 0);
  uint32_t w_off[NB], s_off[NB], x_off[TT], xs_off[TT];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const bool on = 16 * b + r < cols;
    w_off[b] = on ? (uint32_t)(16 * b + r) * (uint32_t)a.ld_w + 16 * g : kPastEnd;
    s_off[b] = on ? (uint32_t)(16 * b + r) * (uint32_t)a.ld_ws + g : kPastEnd;
  }
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const bool on = 16 * i + r < rows;
    x_off[i] = on ? (uint32_t)(16 * i + r) * (uint32_t)a.ld_x + 16 * XL * g : kPastEnd;
    xs_off[i] = on ? (uint32_t)(16 * i + r) * (uint32_t)a.ld_xs + g : kPastEnd;
  }
  f32x4 acc[G][NB][TT];
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < TT; ++i) acc[h][b][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * 128; k0 < a.K; k0 += kFewWaves * 128 * U) {
    v4u32 wv[U][G][NB], xv[U][TT][XL];
    uint32_t sv[U][G][NB], xsv[U][TT];
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int k = k0 + s * kFewWaves * 128;
      const bool in = k + 32 * g < a.K;      // a lane's block is whole or absent
      auto at = [&](uint32_t off, int step) __attribute__((always_inline)) {
        return (int)(in && off != kPastEnd ? off + step : kPastEnd);
      };
#pragma unroll
      for (int h = 0; h < G; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          wv[s][h][b] = __builtin_amdgcn_raw_buffer_load_b128(wr[h], at(w_off[b], k / 2), 0, 0);
          sv[s][h][b] = __builtin_amdgcn_raw_buffer_load_b8(sr[h], at(s_off[b], k / 32), 0, 0);
        }
#pragma unroll
      for (int i = 0; i < TT; ++i) {
#pragma unroll
        for (int c = 0; c < XL; ++c)
          xv[s][i][c] = __builtin_amdgcn_raw_buffer_load_b128(xr, at(x_off[i], MX ? k / 2 : k * 2 + 16 * c), 0, 0);
        xsv[s][i] = MX ? __builtin_amdgcn_raw_buffer_load_b8(xsr, at(xs_off[i], k / 32), 0, 0) : 0;
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // all of them, before the first is waited for
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int h = 0; h < G; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const v4u32 q = wv[s][h][b];
          if constexpr (MX) {
            const i32x8 wq = {(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < TT; ++i) {
              const v4u32 p = xv[s][i][0];
              const i32x8 xq = {(int)p[0], (int)p[1], (int)p[2], (int)p[3], 0, 0, 0, 0};
              acc[h][b][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wq, xq, acc[h][b][i], 4, 4, 0, (int)sv[s][h][b],
                                                                               0, (int)xsv[s][i]);
            }
          } else {
            typedef typename Elem<F16>::v8 v8;
            const float scale = scale_of(sv[s][h][b]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const v8 wide = __builtin_bit_cast(v8, widen<F16>(q[c], scale));
#pragma unroll
              for (int i = 0; i < TT; ++i)
                acc[h][b][i] = Elem<F16>::mfma16(wide, __builtin_bit_cast(v8, xv[s][i][c]), acc[h][b][i]);
            }
          }
        }
  }
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < TT; ++i)
        part[wave][h * NB + b][i][lane] = make_float4(acc[h][b][i][0], acc[h][b][i][1], acc[h][b][i][2], acc[h][b][i][3]);
  __syncthreads();
  for (int j = wave; j < NB * TT; j += kFewWaves) {
    const int b = j / TT, i = j % TT;
    float z[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f}, y[4];
#pragma unroll
    for (int v = 0; v < kFewWaves; ++v) {
      const float4 p = part[v][b][i][lane];
      z[0] += p.x; z[1] += p.y; z[2] += p.z; z[3] += p.w;
      if constexpr (GATED) {
        const float4 o = part[v][(G - 1) * NB + b][i][lane];
        u[0] += o.x; u[1] += o.y; u[2] += o.z; u[3] += o.w;
      }
    }
    const int m = 16 * i + r, n = n0 + 16 * b + 4 * g;
    if (m >= rows || n >= a.N) continue;
    if (a.bias) {
      float add[4];
      load4(a.out_type, a.bias, (int64_t)expert * G * a.N + n, a.N - n, add);
#pragma unroll
      for (int c = 0; c < 4; ++c) z[c] += add[c];
      if constexpr (GATED) {
        load4(a.out_type, a.bias, (int64_t)expert * G * a.N + a.N + n, a.N - n, add);
#pragma unroll
        for (int c = 0; c < 4; ++c) u[c] += add[c];
      }
    }
    if constexpr (GATED) {
#pragma unroll
      for (int c = 0; c < 4; ++c) y[c] = z[c] * logistic(z[c]) * u[c];
    } else {
      activate_all(a.act, z, y);
    }
    store_row(a.out_type, a.out, (row0 + m) * a.ld_out + n, a.N - n, y);
  }
}

// --- host -------------------------------------------------------------------

template <class F>
void with_x(int dtype, F f) {
  if (dtype == MOE_BF16) f(std::integral_constant<int, MOE_BF16>{});
  else if (dtype == MOE_F16) f(std::integral_constant<int, MOE_F16>{});
  else f(std::integral_constant<int, MOE_MXFP4>{});
}

QuantArgs quant_args(int64_t rows, int depth, const void* x, int size, int64_t ld_x, uint8_t* q, int64_t ld_q,
                     uint8_t* scale, int64_t ld_s, dim3* grid) {
  QuantArgs a = {(const char*)x, q, scale, depth / 8, rows, ld_x * size, ld_q, ld_s};
  if (ld_x == depth && ld_q == depth / 2 && ld_s == depth / 32) {   // packed: one long row
    a.n8 *= rows;
    a.rows = 1;
  }
  const int64_t per = 256 * kQuantUnroll, across = (a.n8 + per - 1) / per;
  *grid = dim3((unsigned)(across < (1 << 16) ? across : 1 << 16), (unsigned)(a.rows < 4096 ? a.rows : 4096));
  if (across * a.rows > (1 << 20)) grid->x = (unsigned)(across < 256 ? across : 256);
  return a;
}

// column tiles of `width` and row tiles of `bm` in launches of fewer than 2^31 threads
template <class F>
void launch_tiles(MxArgs& a, int bm, int width, int threads, F go) {
  const int64_t row_tiles = a.offsets ? (a.rows / bm + a.E < a.rows ? a.rows / bm + a.E : a.rows) : (a.rows + bm - 1) / bm;
  const int all = (a.N + width - 1) / width;
  int64_t most = (1ll << 31) / threads / row_tiles;
  if (most < 1) most = 1;
  for (a.nt0 = 0; a.nt0 < all; a.nt0 += a.n_nt) {
    a.n_nt = (int)(all - a.nt0 < most ? all - a.nt0 : most);
    go(dim3((unsigned)(row_tiles * a.n_nt)));
  }
}

}  // namespace

hipError_t launch_mx_quantize(int64_t rows, int depth, const void* x, int dtype, int64_t ld_x, uint8_t* q, int64_t ld_q,
                              uint8_t* scale, int64_t ld_s, hipStream_t s) {
  dim3 grid;
  const QuantArgs a = quant_args(rows, depth, x, dtype == MOE_F32 ? 4 : 2, ld_x, q, ld_q, scale, ld_s, &grid);
  if (dtype == MOE_BF16) hipLaunchKernelGGL((quantize_kernel<MOE_BF16>), grid, dim3(256), 0, s, a);
  else if (dtype == MOE_F16) hipLaunchKernelGGL((quantize_kernel<MOE_F16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((quantize_kernel<MOE_F32>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(int64_t rows, int depth, const uint8_t* q, int64_t ld_q, const uint8_t* scale,
                                int64_t ld_s, void* out, int dtype, int64_t ld_out, hipStream_t s) {
  dim3 grid;
  const QuantArgs a = quant_args(rows, depth, out, dtype == MOE_F32 ? 4 : 2, ld_out, const_cast<uint8_t*>(q), ld_q,
                                 const_cast<uint8_t*>(scale), ld_s, &grid);
  if (dtype == MOE_BF16) hipLaunchKernelGGL((dequantize_kernel<MOE_BF16>), grid, dim3(256), 0, s, a);
  else if (dtype == MOE_F16) hipLaunchKernelGGL((dequantize_kernel<MOE_F16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((dequantize_kernel<MOE_F32>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_mx_linear(const moe_mx_linear_desc& d, const void* x, const uint8_t* x_scale, const uint8_t* w,
                            const uint8_t* w_scale, const int32_t* offsets, const void* bias, void* out, hipStream_t s) {
  MxArgs a = {};
  a.x = (const char*)x; a.w = (const char*)w; a.xs = x_scale; a.ws = w_scale;
  a.offsets = offsets; a.bias = bias; a.out = (char*)out;
  a.ld_x = d.dtype == MOE_MXFP4 ? d.ld_x : 2 * d.ld_x;
  a.ld_xs = d.ld_x_scale; a.ld_w = d.ld_w; a.ld_ws = d.ld_w_scale;
  a.expert_w = d.expert_w; a.expert_ws = d.expert_w_scale;
  a.ld_out = d.ld_out;
  a.rows = d.rows;
  a.E = d.experts; a.N = d.cols; a.K = d.depth; a.act = d.act; a.out_type = d.out_dtype;
  with_x(d.dtype, [&](auto xt) {
    constexpr int XT = decltype(xt)::value;
    launch_tiles(a, 16, 16, kFewWaves * 64, [&](dim3 grid) {
      if (d.act == MOE_ACT_SWIGLU) hipLaunchKernelGGL((few_rows_kernel<XT, true, 1, 1, 4>), grid, dim3(kFewWaves * 64), 0, s, a);
      else hipLaunchKernelGGL((few_rows_kernel<XT, false, 1, 1, 4>), grid, dim3(kFewWaves * 64), 0, s, a);
    });
  });
  return hipGetLastError();
}

}  // namespace moe
