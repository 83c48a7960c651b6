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
#include <math.h>

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
// round to the nearest element, ties to the even one, and saturate at 6.  A thread
// has four groups of eight in flight.  Bound by HBM: 16384 x 7168 from bf16 and back, 597 MB,
// 129 us a pair of calls (4.6 TB/s, a large copy 4.98), 72 (60 at best) and 56 us in the profiler's
// intervals; 64 x 2048 take a launch each.
// A packed matrix is taken as one long row, without divisions.

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

// inclusive sum over the wavefront's lanes: shifts inside rows of 16, then the
// rows' last lanes broadcast on
__device__ __forceinline__ int lane_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);    // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);    // 2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);    // 4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);    // 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
  return v;
}

// Rows of four experts from the lane's on: their first rows and numbers of tiles of bm.
// Four a lane, so that 256 experts' offsets are in flight together.
struct Four {
  int lo[4], hi[4], n[4], all;
};
__device__ __forceinline__ Four four_experts(const MxArgs& a, int bm, int e) {
  const int rows = (int)a.rows;
  int at[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) at[i] = a.offsets[min(e + i, a.E)];
  Four f;
  f.all = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {                 // past the last expert: no rows
    f.lo[i] = min(max(at[i], 0), rows);
    f.hi[i] = min(max(at[i + 1], 0), rows);
    f.n[i] = f.hi[i] > f.lo[i] ? (f.hi[i] - f.lo[i] + bm - 1) / bm : 0;
    f.all += f.n[i];
  }
  return f;
}

// Row tiles of bm of all experts' rows.  Called by whole wavefronts.
__device__ __forceinline__ int count_tiles(const MxArgs& a, int bm) {
  if (!a.offsets) return ((int)a.rows + bm - 1) / bm;
  int n = 0;
  for (int e = (threadIdx.x & 63) * 4; e < a.E; e += 256) n += four_experts(a, bm, e).all;
  return __builtin_amdgcn_readlane(lane_scan(n), 63);
}

// Row tile t of the experts' rows cut into pieces of bm, none of which holds
// rows of two experts.  Offsets out of order or out of range give other rows, but
// none outside [0, rows).  Called by whole wavefronts.
__device__ __forceinline__ RowTile find_tile(const MxArgs& a, int bm, int t) {
  if (!a.offsets) {
    const int64_t row = (int64_t)t * bm;
    return {0, row < a.rows ? min(bm, (int)(a.rows - row)) : 0, row};
  }
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < a.E; e0 += 256) {
    const Four f = four_experts(a, bm, e0 + 4 * lane);
    const int upto = lane_scan(f.all), all = __builtin_amdgcn_readlane(upto, 63);
    if (t < all) {
      int before = upto - f.all, expert = -1, row = 0, last = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t >= before && t < before + f.n[i]) {
          expert = e0 + 4 * lane + i;
          row = f.lo[i] + (t - before) * bm;
          last = f.hi[i];
        }
        before += f.n[i];
      }
      const int l = __builtin_ctzll(__ballot(expert >= 0));
      const int first = __builtin_amdgcn_readlane(row, l);
      return {__builtin_amdgcn_readlane(expert, l), min(bm, __builtin_amdgcn_readlane(last, l) - first), first};
    }
    t -= all;
  }
  return {0, 0, 0};
}

// W columns of a row in the output's type, of which `left` exist
template <int W>
__device__ __forceinline__ void load_row(int type, const void* base, int64_t at, int left, float (&v)[W]) {
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

// 16 bytes of a row's scales, zeros from byte `left` on, where the row ends; `before` of its bytes
// lie in front of p.  A row of 16 or more is read up to its end, in one load, and
// shifted (byte by byte 1536 rows over 128 experts of 2048 x 768 took 82 us).
__device__ __forceinline__ v4u32 load_scales(const uint8_t* p, int before, int left) {
  if (left >= 16) return ((const Loose<v4u32, 1>*)p)->v;
  v4u32 v = {0, 0, 0, 0};
  if (left <= 0) return v;
  if (before + left >= 16) {
    v = ((const Loose<v4u32, 1>*)(p + left - 16))->v;
    uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
    const int bits = 8 * (16 - left);          // 8 .. 120
    lo = bits >= 64 ? hi >> (bits - 64) : lo >> bits | hi << (64 - bits);
    hi = bits >= 64 ? 0 : hi >> bits;
    return v4u32{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
#pragma unroll
  for (int c = 0; c < 15; ++c)
    if (c < left) v[c / 4] |= (uint32_t)p[c] << (c % 4 * 8);
  return v;
}

// --- few rows -------------------------------------------------------------------
//
// Bound by reading the weights, which every (row tile, column tile) workgroup
// does once, straight into operand registers.  A workgroup owns 16 TT rows of
// one expert and 16 BLOCKS rows of w (gated: half of them gate, half up rows); its
// wavefronts take K in pieces of 512, 256 contiguous bytes of each weight row, in
// turn and join their sums in LDS.  A piece is four steps of 128: a lane holds
// row lane % 16, block lane / 16 of each; with 16-bit operands dword i of the
// block is the lane's part of the step's i-th v_mfma_f32_16x16x32.  A row's 16
// scales of a piece are one load, of which step s needs byte lane / 16 of dword s.
// Result lane: row (of x) lane % 16, columns 4 (lane / 16) .. + 3.
// Measured with the weights in no cache (a call among others): 8 rows over 8 experts of 2 x
// 2048 x 7168, 125 MB, 30.3 us (4.1 TB/s); 512 over 128 of 2 x 768 x 2048, 217 MB, 50 us
// (4.4 TB/s); replayed from a graph over 600 MB of weights 34 and 55 us, with x in 4 bits 26.7 and
// 47.5.  With pieces of 128 elements and 8 wavefronts a workgroup they took 46 and
// 133 us: 64 contiguous bytes a row and load, four times the loads of scales, and half as many
// workgroups a CU.  x's operands are read a step ahead alone (all four steps' cost the
// registers of a second workgroup: 62 instead of 57 us).
template <int XT, bool GATED, int TT, int BLOCKS, int W>
__global__ __launch_bounds__(W * 64) void few_rows_kernel(MxArgs a) {
  constexpr bool MX = XT == MOE_MXFP4, F16 = XT == MOE_F16;
  constexpr int G = GATED ? 2 : 1, NB = BLOCKS / G;      // 16-row blocks of gate, and of up rows
  constexpr int XL = MX ? 1 : 4;      // 16-byte loads of a block of x
  constexpr int AHEAD = MX ? 4 : 1;                      // steps of x in registers
  __shared__ float4 part[W][BLOCKS][TT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const RowTile tile = find_tile(a, 16 * TT, blockIdx.x / a.n_nt);
  const int expert = __builtin_amdgcn_readfirstlane(tile.expert), rows = __builtin_amdgcn_readfirstlane(tile.count);
  const int64_t row0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)tile.row);
  if (rows <= 0) return;
  const int n0 = (a.nt0 + (int)(blockIdx.x % a.n_nt)) * 16 * NB;
  const int r = lane & 15, g = lane >> 4;
  const int cols = min(16 * NB, a.N - n0);
  __amdgpu_buffer_rsrc_t wr[G];
  const uint8_t* ws[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const int64_t n = (int64_t)h * a.N + n0;
    wr[h] = make_rsrc(a.w + expert * a.expert_w + n * a.ld_w, (cols - 1) * a.ld_w + a.K / 2);
    ws[h] = a.ws + expert * a.expert_ws + n * a.ld_ws;
  }
  const int row_bytes = MX ? a.K / 2 : a.K * 2;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + row0 * a.ld_x, (rows - 1) * a.ld_x + row_bytes);
  const uint8_t* xs = MX ? a.xs + row0 * a.ld_xs : nullptr;
  // rows past the last one: no data; any scales, their results are not stored
  uint32_t w_off[NB], x_off[TT], s_off[NB], xs_off[TT];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    w_off[b] = 16 * b + r < cols ? (uint32_t)(16 * b + r) * (uint32_t)a.ld_w + 16 * g : kPastEnd;
    s_off[b] = (uint32_t)min(16 * b + r, cols - 1) * (uint32_t)a.ld_ws;
  }
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    x_off[i] = 16 * i + r < rows ? (uint32_t)(16 * i + r) * (uint32_t)a.ld_x + 16 * XL * g : kPastEnd;
    xs_off[i] = MX ? (uint32_t)min(16 * i + r, rows - 1) * (uint32_t)a.ld_xs : 0;
  }
  f32x4 acc[G][NB][TT];
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < TT; ++i) acc[h][b][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto piece = [&](int k0, auto whole_tag) __attribute__((always_inline)) {
    constexpr bool WHOLE = decltype(whole_tag)::value;
    v4u32 wv[4][G][NB], xv[AHEAD][TT][XL], sv[G][NB], xsv[TT];
    // scales of the piece; past K's end zeros, since a NaN there would count
    auto scales = [&](const uint8_t* p) __attribute__((always_inline)) {
      if constexpr (WHOLE) return ((const Loose<v4u32, 1>*)(p + k0 / 32))->v;
      else return load_scales(p + k0 / 32, k0 / 32, (a.K - k0) / 32);
    };
#pragma unroll
    for (int h = 0; h < G; ++h)
#pragma unroll
      for (int b = 0; b < NB; ++b) sv[h][b] = scales(ws[h] + s_off[b]);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int k = k0 + s * 128;
      const bool in = WHOLE || k + 32 * g < a.K;      // a lane's block is whole or absent
#pragma unroll
      for (int h = 0; h < G; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          wv[s][h][b] = __builtin_amdgcn_raw_buffer_load_b128(wr[h], (int)(in ? w_off[b] + k / 2 : kPastEnd), 0, 0);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
      if constexpr (MX) xsv[i] = scales(xs + xs_off[i]);
    auto rows_of = [&](int s) __attribute__((always_inline)) {
      const int k = k0 + s * 128;
      const bool in = WHOLE || k + 32 * g < a.K;
#pragma unroll
      for (int i = 0; i < TT; ++i)
#pragma unroll
        for (int c = 0; c < XL; ++c)
          xv[s % AHEAD][i][c] = __builtin_amdgcn_raw_buffer_load_b128(xr, (int)(in ? x_off[i] + (MX ? k / 2 : k * 2) + 16 * c : kPastEnd), 0, 0);
    };
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) rows_of(s);
    __builtin_amdgcn_sched_barrier(0);   // all of them, before the first is waited for
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int h = 0; h < G; ++h)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const v4u32 q = wv[s][h][b];
          const uint32_t sw = sv[h][b][s] >> (8 * g) & 0xff;
          if constexpr (MX) {
            const i32x8 wq = {(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < TT; ++i) {
              const v4u32 p = xv[s % AHEAD][i][0];
              const i32x8 xq = {(int)p[0], (int)p[1], (int)p[2], (int)p[3], 0, 0, 0, 0};
              acc[h][b][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wq, xq, acc[h][b][i], 4, 4, 0, (int)sw, 0,
                                                                               (int)(xsv[i][s] >> (8 * g) & 0xff));
            }
          } else {
            typedef typename Elem<F16>::v8 v8;
            const float scale = scale_of(sw);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const v8 wide = __builtin_bit_cast(v8, widen<F16>(q[c], scale));
#pragma unroll
              for (int i = 0; i < TT; ++i)
                acc[h][b][i] = Elem<F16>::mfma16(wide, __builtin_bit_cast(v8, xv[s % AHEAD][i][c]), acc[h][b][i]);
            }
          }
        }
      if (s + AHEAD < 4) rows_of(s + AHEAD);
    }
  };
  for (int k0 = wave * 512; k0 < a.K; k0 += W * 512) {
    if (k0 + 512 <= a.K) piece(k0, std::true_type{});
    else piece(k0, std::false_type{});
  }
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < TT; ++i)
        part[wave][h * NB + b][i][lane] = make_float4(acc[h][b][i][0], acc[h][b][i][1], acc[h][b][i][2], acc[h][b][i][3]);
  __syncthreads();
  for (int j = wave; j < NB * TT; j += W) {
    const int b = j / TT, i = j % TT;
    float z[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f}, y[4];
#pragma unroll
    for (int v = 0; v < W; ++v) {
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
      load_row(a.out_type, a.bias, (int64_t)expert * G * a.N + n, a.N - n, add);
#pragma unroll
      for (int c = 0; c < 4; ++c) z[c] += add[c];
      if constexpr (GATED) {
        load_row(a.out_type, a.bias, (int64_t)expert * G * a.N + a.N + n, a.N - n, add);
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

// --- tiles ----------------------------------------------------------------------
//
// Many rows: tiles of BM rows of one expert x BN rows of w, staged through LDS by
// direct-to-LDS buffer loads, MFMAs out of it.  A stage is 128 bytes of
// each row of x: 256 elements in 4 bits, 64 in 16, and as many elements of w.
// Rows past an operand's end and blocks past K get an offset past the buffer
// descriptor's bound, where loads return zeros.  Scales come through registers
// (their rows may start at any byte), some stages' at a time, into a table of
// their own in LDS, ahead of the stages that need them.
//
// Rates (gated, bf16 out, replayed from a graph).  x in 16 bits: 8192 x 2 x 2048 x 7168 368 us,
// 1.31 PFLOP/s; 16384 rows over 16 uneven experts of 2 x 1536 x 4096 366 us, 1.13.  x in 4
// bits: 46451 over 32 of 2 x 2048 x 7168 835 us, 3.27 PFLOP/s; 8192 x 8192 x 8192 plain
// 293 us, 3.75; 8192 x 2 x 4096 x 28672 899 us, 4.28.  The card's power limits both: with
// random operands in registers alone it reaches 1.91 PFLOP/s in v_mfma_f32_32x32x16_bf16, 2.25 in
// 16x16x32 and 6.8 in v_mfma_scale_f32_32x32x64 of 4 bits (9.4 with constant operands).
// With x in 4 bits there is more between: of the 1.99 us a stage of the 256 x 256 tile takes (1.26 at
// 6.8 PFLOP/s) 1.66 remain without its loads and 1.56 without its LDS reads either, so that 0.3 us
// are neither (all eight wavefronts meet at every stage; what else was not found); a tile adds 13 us (start 3,
// epilogue 10, its stores being two thirds of that), a fifth of the time at K = 7168, in which its CU
// multiplies nothing.  Measured beside it: four wavefronts
// of 128 x 128 4-10% slower; 128 x 256 tiles of 128-element stages, two workgroups a CU, 0-20%
// slower; 16 x 16 steps 40-80% slower (registers).  With x in 16 bits 128 x 256 tiles, whose
// two workgroups a CU overlap one's epilogue with the other's sums, take 366 us for 16384 rows where
// 256 x 256 ones take 391, and 193 us for 8192 x 7168 x 2048 (211); where tiles fit the CUs
// exactly and sums are long they are 3% slower.

// WAVES_SIMD: wavefronts a SIMD that the registers are limited for; B16, STAGES16: block of the
// matrix steps and stages in LDS with x in 16 bits
template <int BM_, int BN_, int WAVES_M, int WAVES_N, int WAVES_SIMD_, int B16_, int STAGES16_ = 3>
struct MxTile {
  static constexpr int BM = BM_, BN = BN_, WAVES_SIMD = WAVES_SIMD_, B16 = B16_, STAGES16 = STAGES16_;
  static constexpr int NW = WAVES_M * WAVES_N, NT = NW * 64, WN_ = WAVES_N;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int PITCH = WN + 4;            // floats of a row in the epilogue's staging
  static constexpr int EPI = NW * 32 * PITCH * 4;
};
typedef MxTile<256, 256, 2, 4, 2, 16> Mx256;     // x in 4 bits
typedef MxTile<128, 256, 2, 4, 4, 16> MxWide;    // x in 16 bits: two workgroups a CU
typedef MxTile<128, 128, 2, 2, 1, 32> Mx128;
typedef MxTile<32, 256, 1, 4, 1, 32, 5> Mx32;    // x in 16 bits: 12 to 40 rows an expert
typedef MxTile<32, 128, 1, 2, 1, 32> Mx32Both;   // the same with x in 4 bits: two wavefronts, three workgroups a CU
typedef MxTile<64, 128, 2, 2, 1, 32> Mx64;       // (16 x 16 steps: 4096 rows over 128 experts of 2 x 768 x 2048 84 us instead of 79)

// vmcnt(flying) lgkmcnt(0) and the workgroup's barrier
template <int FLYING>
__device__ __forceinline__ void meet() {
  static_assert(FLYING < 16, "vector memory counter's low bits");
  __builtin_amdgcn_s_waitcnt(0x70 | FLYING);
  __builtin_amdgcn_s_barrier();
}

// A workgroup's tile: its place among the row and column tiles.  Workgroup i runs
// on XCD i mod 8; each XCD gets a contiguous run, in which 8 row tiles x 4 column
// tiles share their operands in its L2.
struct Place {
  int expert, rows;     // rows: of the tile, 0 if there is none
  int64_t row;
  int n0, cols;         // output columns
};
template <int BM, int HB>
__device__ __forceinline__ Place place_of(const MxArgs& a) {
  const int n_mt = count_tiles(a, BM), total = n_mt * a.n_nt;
  if ((int)blockIdx.x >= total) return {0, 0, 0, 0, 0};
  int t = xcd_order(blockIdx.x, total);
  const int grp = t / (8 * a.n_nt), rows8 = min(8, n_mt - grp * 8);
  t -= grp * 8 * a.n_nt;
  const RowTile r = find_tile(a, BM, grp * 8 + t % rows8);
  const int n0 = (a.nt0 + t / rows8) * HB;
  return {__builtin_amdgcn_readfirstlane(r.expert), __builtin_amdgcn_readfirstlane(r.count),
          __builtin_amdgcn_readfirstlane((int)r.row), n0, min(HB, a.N - n0)};
}

// first row of w, inside the tile, of a wavefront's i-th block of B; gated: the first
// half of its blocks are gate rows, the others up rows
template <class C, bool GATED, int B>
__device__ __forceinline__ int block_row(int wave_n, int i) {
  constexpr int HALF = C::WN / 2;
  if constexpr (GATED) return B * i < HALF ? wave_n * HALF + B * i : C::BN / 2 + wave_n * HALF + B * i - HALF;
  else return wave_n * C::WN + B * i;
}

// whether any of a wavefront's part of the tile exists: at an expert's or w's end the
// others only load, and leave the matrix cores to those that share theirs (2048 rows over 32
// experts of 2 x 2048 x 7168, x in 4 bits, 152 -> 150 us; 4096 over 128 of 2 x 768 x 2048, bf16, 78 -> 76)
template <class C, bool GATED>
__device__ __forceinline__ bool has_results(const Place& p, int wave_m, int wave_n) {
  return wave_m * C::WM < p.rows && wave_n * (GATED ? C::WN / 2 : C::WN) < p.cols;
}

// 32 rows of a wavefront's columns at a time go through LDS, so that lanes hold
// neighbouring columns and every global access covers whole lines.
// put(j, to): the sums of rows 32 j .. + 31 to `to`, rows C::PITCH floats apart.
template <class C, bool GATED, class Put>
__device__ __forceinline__ void finish_tile(const MxArgs& a, const Place& p, char* lds, int wave, int lane, Put put) {
  constexpr int CW = GATED ? C::WN / 2 : C::WN, G = GATED ? 2 : 1;
  float* stage = (float*)lds + wave * 32 * C::PITCH;
  const int wave_m = wave / C::WN_, wave_n = wave % C::WN_;
  constexpr int LPR = CW / 8, RPP = 64 / LPR;   // lanes a row (8 columns each), rows a pass
  const int er = lane / LPR, ec = (lane % LPR) * 8;
  const int n = p.n0 + wave_n * CW + ec, left = a.N - n;
  float bz[8], bu[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) bz[c] = bu[c] = 0.f;
  if (a.bias && left > 0) {
    const int64_t at = (int64_t)p.expert * G * a.N + n;
    load_row(a.out_type, a.bias, at, left, bz);
    if constexpr (GATED) load_row(a.out_type, a.bias, at + a.N, left, bu);
  }
#pragma unroll
  for (int j = 0; j < C::WM / 32; ++j) {
    put(j, stage);
    __builtin_amdgcn_wave_barrier();
    auto staged8 = [&](int r, int col, float (&v)[8]) __attribute__((always_inline)) {
      const float4 x = *(const float4*)(stage + r * C::PITCH + col), y = *(const float4*)(stage + r * C::PITCH + col + 4);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    };
#pragma unroll 2
    for (int r = er; r < 32; r += RPP) {
      const int m = wave_m * C::WM + 32 * j + r;
      float z[8], u[8], y[8];
      staged8(r, ec, z);
      if constexpr (GATED) staged8(r, CW + ec, u);
      if (m >= p.rows || left <= 0) continue;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        z[c] += bz[c];
        if constexpr (GATED) y[c] = z[c] * logistic(z[c]) * (u[c] + bu[c]);
      }
      if constexpr (!GATED) activate_all(a.act, z, y);
      store_row(a.out_type, a.out, (p.row + m) * a.ld_out + n, left, y);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Both operands in 4 bits.  A stage's 16-byte chunks (one block each) of row r lie
// at c ^ (r / 2) % 8, free of bank conflicts.  Lane half h takes chunks 4 h + kk of
// a stage in MFMA step kk, so that its four scales are one dword.
template <class C, bool GATED>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::WAVES_SIMD)))
void mx_both_kernel(MxArgs a) {
  constexpr int FM = C::WM / 32, FN = C::WN / 32;           // blocks of v_mfma_scale_f32_32x32x64
  constexpr int A_BYTES = C::BM * 128, STAGE = A_BYTES + C::BN * 128;
  constexpr int SCALES = (C::BM + C::BN) * 32;              // four stages' scales
  constexpr int A_LOADS = C::BM / 8 / C::NW, B_LOADS = C::BN / 8 / C::NW;
  constexpr int S_CHUNKS = SCALES / 16, S_LOADS = (S_CHUNKS + C::NT - 1) / C::NT;
  constexpr int LDS = 2 * STAGE + 2 * SCALES;
  static_assert(LDS >= C::EPI && LDS <= 160 * 1024 && C::NW % 2 == 0 && B_LOADS % 2 == 0 && FN % 2 == 0, "tile");
  __shared__ __attribute__((aligned(1024))) char lds[LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave_m = wave / C::WN_, wave_n = wave % C::WN_;
  constexpr int HB = GATED ? C::BN / 2 : C::BN;
  const Place p = place_of<C::BM, HB>(a);
  if (p.rows <= 0) return;
  const int arows = p.rows, brows = p.cols;
  const int kbytes = a.K / 2, kscales = a.K / 32;
  const int KT = (kbytes + 127) / 128;

  const char* w = a.w + p.expert * a.expert_w + p.n0 * a.ld_w;
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(a.x + p.row * a.ld_x, (arows - 1) * a.ld_x + kbytes);
  const __amdgpu_buffer_rsrc_t br = make_rsrc(w, (brows - 1) * a.ld_w + kbytes);
  const __amdgpu_buffer_rsrc_t ur = GATED ? make_rsrc(w + a.N * a.ld_w, (brows - 1) * a.ld_w + kbytes) : br;
  uint32_t aoff[A_LOADS], boff[B_LOADS];
  const int chunk = (lane % 8) ^ ((wave * 4 + lane / 16) % 8);   // of a row in memory, the same in all of this lane's loads
#pragma unroll
  for (int i = 0; i < A_LOADS; ++i) {
    const int r = (wave + i * C::NW) * 8 + lane / 8;
    aoff[i] = r < arows ? (uint32_t)r * (uint32_t)a.ld_x + chunk * 16 : kPastEnd;
  }
#pragma unroll
  for (int i = 0; i < B_LOADS; ++i) {
    const int r = (wave + (GATED ? i % (B_LOADS / 2) : i) * C::NW) * 8 + lane / 8;   // the second half: up rows
    boff[i] = r < brows ? (uint32_t)r * (uint32_t)a.ld_w + chunk * 16 : kPastEnd;
  }
  auto issue = [&](int k) __attribute__((always_inline)) {
    char* base = lds + (k & 1) * STAGE;
    const bool on = chunk * 16 < kbytes - 128 * k;     // past K's end: zeros
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i)
      load_lds(ar, base + (wave + i * C::NW) * 1024, on ? aoff[i] : kPastEnd, 128 * k);
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i)
      load_lds(GATED && i >= B_LOADS / 2 ? ur : br, base + A_BYTES + (wave + i * C::NW) * 1024, on ? boff[i] : kPastEnd, 128 * k);
  };
  // scales of stages 4 s .. 4 s + 3: 32 bytes a row (x's rows, then w's), this thread's
  // 16-byte halves; halves of rows 8 .. 15 of 16 swapped, against bank conflicts
  v4u32 sc[S_LOADS];
  const uint8_t* srow[S_LOADS];
#pragma unroll
  for (int i = 0; i < S_LOADS; ++i) {
    const int id = min(i * C::NT + tid, S_CHUNKS - 1), r = id / 2;
    if (r < C::BM) {   // rows past the last one: any scales, their results are not stored
      srow[i] = a.xs + (p.row + min(r, arows - 1)) * a.ld_xs + id % 2 * 16;
    } else {
      const int q = r - C::BM, up = GATED && q >= HB ? 1 : 0, b = min(q - up * HB, brows - 1);
      srow[i] = a.ws + p.expert * a.expert_ws + ((int64_t)up * a.N + p.n0 + b) * a.ld_ws + id % 2 * 16;
    }
  }
  auto fetch_scales = [&](int s) __attribute__((always_inline)) {
    if (32 * s + 32 <= kscales) {
#pragma unroll
      for (int i = 0; i < S_LOADS; ++i) sc[i] = ((const Loose<v4u32, 1>*)(srow[i] + 32 * s))->v;
    } else {
#pragma unroll 1
      for (int i = 0; i < S_LOADS; ++i) {
        const int at = 32 * s + min(i * C::NT + tid, S_CHUNKS - 1) % 2 * 16;
        const v4u32 v = load_scales(srow[i] + 32 * s, at, kscales - at);
#pragma unroll
        for (int j = 0; j < S_LOADS; ++j) sc[j] = j == i ? v : sc[j];
      }
    }
  };
  auto keep_scales = [&](int s) __attribute__((always_inline)) {
    char* base = lds + 2 * STAGE + (s & 1) * SCALES;
#pragma unroll
    for (int i = 0; i < S_LOADS; ++i) {
      const int id = min(i * C::NT + tid, S_CHUNKS - 1), r = id / 2;
      *(v4u32*)(base + r * 32 + ((id % 2) ^ (r / 8 % 2)) * 16) = sc[i];
    }
  };

  const int lrow = lane & 31, lhalf = lane >> 5, rsw = lrow / 2 % 8, ssw = lrow / 8 % 2;
  f32x16 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  auto ready = [&](int k) __attribute__((always_inline)) {   // stage k is there, the next ones under way
    meet<0>();
    if ((k & 3) == 0 && k + 4 < KT) fetch_scales(k / 4 + 1);
    if ((k & 3) == 1 && k + 3 < KT) keep_scales(k / 4 + 1);
  };
  auto step = [&](int k) __attribute__((always_inline)) {
    ready(k);
    const char* sa = lds + (k & 1) * STAGE;
    const char* sb = sa + A_BYTES;
    const char* ss = lds + 2 * STAGE + (k / 4 & 1) * SCALES + (((k / 2 & 1) ^ ssw) * 16 + (k & 1) * 8 + lhalf * 4);
    int sw[FN], sx[FM];
    v4u32 pw[2][FN], px[2][FM];
    auto fetch = [&](int kk) __attribute__((always_inline)) {
      const int phys = ((4 * lhalf + kk) ^ rsw) * 16;
#pragma unroll
      for (int i = 0; i < FN; ++i) pw[kk & 1][i] = *(const v4u32*)(sb + (block_row<C, GATED, 32>(wave_n, i) + lrow) * 128 + phys);
#pragma unroll
      for (int j = 0; j < FM; ++j) px[kk & 1][j] = *(const v4u32*)(sa + (wave_m * C::WM + 32 * j + lrow) * 128 + phys);
    };
#pragma unroll
    for (int i = 0; i < FN; ++i) sw[i] = *(const int*)(ss + (C::BM + block_row<C, GATED, 32>(wave_n, i) + lrow) * 32);
#pragma unroll
    for (int j = 0; j < FM; ++j) sx[j] = *(const int*)(ss + (wave_m * C::WM + 32 * j + lrow) * 32);
    fetch(0);
    issue(k + 1);
    __builtin_amdgcn_sched_barrier(0);
    auto multiply = [&](auto kt) __attribute__((always_inline)) {
      constexpr int kk = decltype(kt)::value;
      if constexpr (kk < 3) fetch(kk + 1);
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          const v4u32 q = pw[kk & 1][i], r = px[kk & 1][j];
          const i32x8 wq = {(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
          const i32x8 xq = {(int)r[0], (int)r[1], (int)r[2], (int)r[3], 0, 0, 0, 0};
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wq, xq, acc[i][j], 4, 4, kk, sw[i], kk, sx[j]);
        }
    };
    multiply(std::integral_constant<int, 0>{});
    multiply(std::integral_constant<int, 1>{});
    multiply(std::integral_constant<int, 2>{});
    multiply(std::integral_constant<int, 3>{});
    // each MFMA step's operand reads before the previous step's MFMAs
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (kk < 3) __builtin_amdgcn_sched_group_barrier(0x100, FN + FM, 0);
      __builtin_amdgcn_sched_group_barrier(0x8, FN * FM, 0);
    }
  };
  fetch_scales(0);
  issue(0);
  keep_scales(0);
  if (has_results<C, GATED>(p, wave_m, wave_n)) {
#pragma unroll 1
    for (int k = 0; k < KT; ++k) step(k);
  } else {
#pragma unroll 1
    for (int k = 0; k < KT; ++k) {
      ready(k);
      issue(k + 1);
    }
  }
  meet<0>();   // every wave is done with the operands
  finish_tile<C, GATED>(a, p, lds, wave, lane, [&](int j, float* to) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(float4*)(to + lrow * C::PITCH + 32 * i + 8 * q + 4 * lhalf) =
            make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
  });
}

// Where the 16-byte chunks of a pair of rows (p of 8) lie: c ^ spread(p).  A 16-byte LDS
// read serves lanes 0-3, 12-15, 20-23 and 24-27 together, then the others of 32: with
// blocks of 16 rows pairs 0, 1, 6, 7 at one chunk and pairs 2-5 at the chunk two further, so
// that the latter's places have to be closed under that step.
__device__ __forceinline__ int spread(int p) { return (p & 4) | (p & 1) << 1 | ((p >> 2 ^ p >> 1) & 1); }

// Weights alone in 4 bits.  They lie in LDS as in memory, 32 bytes of a row a
// stage, and become 16-bit operands on the way out of it.  A lane group g (B lanes) takes
// the stage's elements from 8 KK g on, 8 for each of the KK matrix steps: of w 4 KK
// bytes, which are in one block, of x the 16-byte chunks KK g + kk.
template <class C, bool F16, bool GATED>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::WAVES_SIMD)))
void mx_weights_kernel(MxArgs a) {
  typedef typename Elem<F16>::v8 v8;
  constexpr int B = C::B16, GROUPS = 64 / B, KK = 8 / GROUPS;
  constexpr int FM = C::WM / B, FN = C::WN / B;
  typedef uint32_t part_t __attribute__((ext_vector_type(KK)));
  typedef std::conditional_t<B == 32, f32x16, f32x4> acc_t;
  constexpr int STAGES = C::STAGES16;
  constexpr int A_BYTES = C::BM * 128, STAGE = A_BYTES + C::BN * 32;
  constexpr int SCALES = C::BN * 16;                        // eight stages' scales
  constexpr int A_LOADS = C::BM / 8 / C::NW, B_LOADS = C::BN / 32 / C::NW;
  constexpr int RING = STAGES * STAGE + 2 * SCALES, LDS = RING > C::EPI ? RING : C::EPI;
  static_assert(LDS <= 160 * 1024 && C::NW % 2 == 0 && C::BN % (32 * C::NW) == 0 && C::BN <= C::NT && STAGES <= 6, "tile");
  __shared__ __attribute__((aligned(1024))) char lds[LDS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave_m = wave / C::WN_, wave_n = wave % C::WN_;
  constexpr int HB = GATED ? C::BN / 2 : C::BN;
  const Place p = place_of<C::BM, HB>(a);
  if (p.rows <= 0) return;
  const int arows = p.rows, brows = p.cols;
  const int kscales = a.K / 32;
  const int KT = (a.K + 63) / 64;

  const char* w = a.w + p.expert * a.expert_w + p.n0 * a.ld_w;
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(a.x + p.row * a.ld_x, (arows - 1) * a.ld_x + 2 * a.K);
  __amdgpu_buffer_rsrc_t br[B_LOADS];
  uint32_t aoff[A_LOADS], boff[B_LOADS];
  const int chunk = (lane % 8) ^ spread((wave * 4 + lane / 16) % 8);   // of a row in memory, the same in all of this lane's loads
#pragma unroll
  for (int i = 0; i < A_LOADS; ++i) {
    const int r = (wave + i * C::NW) * 8 + lane / 8;
    aoff[i] = r < arows ? (uint32_t)r * (uint32_t)a.ld_x + chunk * 16 : kPastEnd;
  }
  const int block = (lane % 2) ^ (lane / 16 % 2);           // blocks of rows 8 .. 15 of 16 swapped
#pragma unroll
  for (int i = 0; i < B_LOADS; ++i) {                        // 32 rows of w, all of one half of a gated tile
    const int first = (wave + i * C::NW) * 32, up = GATED && first >= HB ? 1 : 0;
    const int r = first - up * HB + lane / 2;
    br[i] = make_rsrc(w + (int64_t)up * a.N * a.ld_w, (brows - 1) * a.ld_w + a.K / 2);
    boff[i] = r < brows ? (uint32_t)r * (uint32_t)a.ld_w + block * 16 : kPastEnd;
  }
  auto issue = [&](int k, int slot) __attribute__((always_inline)) {
    char* base = lds + slot * STAGE;
    const int left = a.K - 64 * k;                           // past K's end: zeros
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i)
      load_lds(ar, base + (wave + i * C::NW) * 1024, chunk * 8 < left ? aoff[i] : kPastEnd, 128 * k);
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i)
      load_lds(br[i], base + A_BYTES + (wave + i * C::NW) * 1024, block * 32 < left ? boff[i] : kPastEnd, 32 * k);
  };
  // scales of stages 8 s .. 8 s + 7: 16 bytes of w's row tid
  v4u32 sc = {0, 0, 0, 0};
  const int sup = GATED && tid >= HB ? 1 : 0;
  const uint8_t* srow = a.ws + p.expert * a.expert_ws +
                        ((int64_t)sup * a.N + p.n0 + min(tid - sup * HB, brows - 1)) * a.ld_ws;
  auto fetch_scales = [&](int s) __attribute__((always_inline)) {
    if (C::NT > C::BN && tid >= C::BN) return;
    if (16 * s + 16 <= kscales) sc = ((const Loose<v4u32, 1>*)(srow + 16 * s))->v;
    else sc = load_scales(srow + 16 * s, 16 * s, kscales - 16 * s);
  };
  auto keep_scales = [&](int s) __attribute__((always_inline)) {
    if (C::NT > C::BN && tid >= C::BN) return;
    *(v4u32*)(lds + STAGES * STAGE + (s & 1) * SCALES + tid * 16) = sc;
  };

  const int lrow = lane % B, g = lane / B, rsw = spread(lrow / 2 % 8);
  const int half = g * 2 / GROUPS;                           // this group's block of a stage
  const int bat = lrow * 32 + (half ^ (lrow / 8 % 2)) * 16 + g % (GROUPS / 2) * 8;
  acc_t acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = acc_t{};

  // stage k in `slot`, the one STAGES - 1 ahead into `next`
  auto ready = [&](int k) __attribute__((always_inline)) {
    meet<(STAGES - 2) * (A_LOADS + B_LOADS)>();
    if ((k & 7) == 0 && k + 8 < KT) fetch_scales(k / 8 + 1);
    if ((k & 7) == 4 && k + 4 < KT) keep_scales(k / 8 + 1);
  };
  auto step = [&](int k, int slot, int next) __attribute__((always_inline)) {
    ready(k);
    const char* sa = lds + slot * STAGE + (wave_m * C::WM + lrow) * 128;
    const char* sb = lds + slot * STAGE + A_BYTES + bat;
    const uint8_t* ss = (const uint8_t*)lds + STAGES * STAGE + (k / 8 & 1) * SCALES + lrow * 16 + (k & 7) * 2 + half;
    float scale[FN];
    part_t q[FN];
    v8 px[2][FM];
    auto fetch = [&](int kk) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < FM; ++j) px[kk & 1][j] = *(const v8*)(sa + B * j * 128 + ((KK * g + kk) ^ rsw) * 16);
    };
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      q[i] = *(const part_t*)(sb + block_row<C, GATED, B>(wave_n, i) * 32);
      scale[i] = scale_of(ss[block_row<C, GATED, B>(wave_n, i) * 16]);
    }
    fetch(0);
    issue(k + STAGES - 1, next);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      if (kk + 1 < KK) fetch(kk + 1);
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const v8 wide = __builtin_bit_cast(v8, widen<F16>(q[i][kk], scale[i]));
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          if constexpr (B == 32) acc[i][j] = Elem<F16>::mfma32(wide, px[kk & 1][j], acc[i][j]);
          else acc[i][j] = Elem<F16>::mfma16(wide, px[kk & 1][j], acc[i][j]);
        }
      }
    }
  };
  fetch_scales(0);
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) issue(k, k);
  keep_scales(0);
  int slot = 0, next = STAGES - 1;
  auto all_stages = [&](auto one) __attribute__((always_inline)) {
#pragma unroll 1
    for (int k = 0; k < KT; ++k) {
      one(k);
      slot = slot + 1 == STAGES ? 0 : slot + 1;
      next = next + 1 == STAGES ? 0 : next + 1;
    }
  };
  if (has_results<C, GATED>(p, wave_m, wave_n)) {
    all_stages([&](int k) __attribute__((always_inline)) { step(k, slot, next); });
  } else {
    all_stages([&](int k) __attribute__((always_inline)) {
      ready(k);
      issue(k + STAGES - 1, next);
    });
  }
  meet<0>();   // every wave is done with the operands
  finish_tile<C, GATED>(a, p, lds, wave, lane, [&](int j, float* to) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 32 / B; ++h)
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int v = 0; v < (B == 32 ? 4 : 1); ++v) {
          const acc_t& z = acc[i][32 / B * j + h];
          *(float4*)(to + (16 * h + lrow) * C::PITCH + B * i + 8 * v + 4 * g) = make_float4(z[4 * v], z[4 * v + 1], z[4 * v + 2], z[4 * v + 3]);
        }
  });
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
  const int64_t gx = across < (1 << 16) ? across : 1 << 16, gy = (1 << 20) / gx;
  *grid = dim3((unsigned)gx, (unsigned)(a.rows < gy ? a.rows : (gy < 65535 ? gy : 65535)));
  return a;
}

template <class F>
void with_flag(bool b, F f) {
  if (b) f(std::true_type{});
  else f(std::false_type{});
}

// How a product is cut: few rows (16 tt rows, `blocks` blocks of w's rows, `waves`
// wavefronts a workgroup) or a tile.
enum MxKind { FEW, T64, T128, T256, WIDE, T32 };
struct MxChoice {
  MxKind kind;
  int tt, blocks, waves;   // FEW
};

// Time of each choice, the smallest wins.  Rows are taken to be spread evenly over the
// experts (the offsets are in device memory), half a row tile lost at each
// expert's end.  A stage of a tile takes a load's latency, or what the
// multiplications of the workgroups that share a CU take; a round of workgroups adds its
// start and epilogue.  A few-row workgroup takes a fixed time (another one in later
// rounds) and one for each piece of K its wavefronts take in turn; all of them together what their reads take.  Neither is
// faster than the weights' reading.  The constants are fitted to the times of every
// choice over 252 products of each kind (1 to 32768 rows, 1 to 128 experts;
// profiles/mx_choice_times.txt): the choice costs 2.8% over the best one on average with x
// in bf16, 3.5% in 4 bits, and more than a tenth for 29 and 35 of them.
// Both sides of typical decisions, in one run of replayed graphs, gated products with x in bf16: 8 rows over 8
// experts of 2 x 2048 x 7168 take 31 us as few rows (16 x 64) and 46 us in tiles of 64 rows; 1024 over 32 of them
// 240 us as few rows, 187 in 64 x 128 tiles, 192 in 128 x 256 (the choice) and 173 in 32 x 256; 384 over 32 of
// 7168 x 2048 (no gate) 77 us in 64 x 128 tiles and 66 in 32 x 256; 16384 over 16 of 2 x 1536 x 4096 493 us in
// 64 x 128, 449 in 128 x 128 and 380 in 128 x 256 ones.
MxChoice choose_mx(const moe_mx_linear_desc& d) {
  struct Fit { double latency, shared, round_us; };
  struct Few { double fixed, next, piece, w_kb, x_kb; };
  static const int bm[6] = {0, 64, 128, 256, 128, 32};
  static const int bn[2][6] = {{0, 128, 128, 256, 256, 256}, {0, 128, 128, 256, 256, 128}};
  static const int per_cu[2][6] = {{0, 3, 2, 0, 2, 2}, {0, 2, 2, 1, 0, 3}};
  static const Fit fits[2][6] = {{{}, {0.406, 0.284, 1.76}, {0.547, 0.436, 3.57}, {}, {0.673, 0.593, 7.72}, {0.467, 0.344, 3.56}},
                                 {{}, {0.549, 0.539, 2.97}, {0.544, 0.492, 5.33}, {1.48, 0.665, 8.52}, {}, {0.364, 0.449, 3.53}}};
  static const Few few[2] = {{1.98, 1.98, 2.83, 0.0778, 0.00733}, {1.98, 5.2, 1.98, 0.0467, 0.00993}};
  static const double tile_rate[2] = {3.15, 4.54}, few_rate[2] = {8.26, 4.57};   // MB/us of weights
  static const MxChoice fews[] = {{FEW, 1, 2, 2}, {FEW, 1, 2, 4}, {FEW, 1, 4, 4}, {FEW, 2, 4, 4}};
  constexpr double kCus = 256;
  const int mx = d.dtype == MOE_MXFP4;
  const double M = (double)(d.rows > 1 ? d.rows : 1), E = d.experts;
  const double n = (double)d.cols * (d.act == MOE_ACT_SWIGLU ? 2 : 1), K = d.depth;
  const double hit = M < E ? M : E, weights_mb = hit * n * K * 0.53e-6;
  auto row_tiles = [&](int rows) {
    if (d.experts == 1) return ceil(M / rows);
    const double t = M / rows + hit * 0.5;
    return t > hit ? t : hit;
  };
  MxChoice best = fews[0];
  double best_us = 1e30;
  auto take = [&](const MxChoice& c, double us) {
    if (us < best_us) {
      best_us = us;
      best = c;
    }
  };
  for (const MxChoice& c : fews) {
    const Few& f = few[mx];
    const double groups = row_tiles(16 * c.tt) * ceil(n / (16 * c.blocks)), pieces = ceil(K / 512);
    const double each = M / hit, rows = each < 16 * c.tt ? each : 16 * c.tt;
    const double rounds = groups / (kCus * (8 / c.waves) * 2), near = weights_mb < 0.3 ? 0.5 : 1;   // (in the L2)
    const double turns = ceil(pieces / c.waves) * f.piece;
    const double wait = f.fixed + turns * near + (rounds > 1 ? (rounds - 1) * (f.next + turns) : 0);
    const double read = f.fixed + groups * K / 512 * (16 * c.blocks * 0.266 * f.w_kb + rows * (mx ? 0.266 : 1) * f.x_kb) / kCus;
    const double all = weights_mb / few_rate[mx];
    take(c, wait > read ? (wait > all ? wait : all) : (read > all ? read : all));
  }
  for (int t : {(int)T64, (int)T128, (int)T256, (int)WIDE, (int)T32}) {
    if (per_cu[mx][t] == 0) continue;          // not with such an x
    const Fit& f = fits[mx][t];
    const double tiles = row_tiles(bm[t]) * ceil(n / bn[mx][t]), steps = ceil(K / (mx ? 256 : 64));
    double share = ceil(tiles / kCus);
    if (share > per_cu[mx][t]) share = per_cu[mx][t];
    const double step = share * f.shared > f.latency ? share * f.shared : f.latency;
    double rounds = tiles / (kCus * share);
    rounds = rounds < 4 ? (rounds > 1 ? ceil(rounds - 0.02) : 1) : rounds + 0.4;
    const double us = rounds * (steps * step + f.round_us), all = weights_mb / tile_rate[mx];
    take({(MxKind)t, 0, 0, 0}, us > all ? us : all);
  }
  return best;
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

void mx_choice(const moe_mx_linear_desc& d, int32_t out[4]) {
  const MxChoice c = choose_mx(d);
  out[0] = c.kind;
  out[1] = c.tt;
  out[2] = c.blocks;
  out[3] = c.waves;
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
  const MxChoice c = choose_mx(d);
  with_flag(d.act == MOE_ACT_SWIGLU, [&](auto g) {
    constexpr bool G = decltype(g)::value;
    if (c.kind == FEW) {
      with_x(d.dtype, [&](auto xt) {
        constexpr int XT = decltype(xt)::value;
        auto go = [&](auto tt, auto blocks, auto waves) {
          constexpr int TT = decltype(tt)::value, BLOCKS = decltype(blocks)::value, W = decltype(waves)::value;
          launch_tiles(a, 16 * TT, 16 * BLOCKS / (G ? 2 : 1), W * 64, [&](dim3 grid) {
            hipLaunchKernelGGL((few_rows_kernel<XT, G, TT, BLOCKS, W>), grid, dim3(W * 64), 0, s, a);
          });
        };
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        using Four = std::integral_constant<int, 4>;
        if (c.tt == 2) go(Two{}, Four{}, Four{});
        else if (c.blocks == 4) go(One{}, Four{}, Four{});
        else if (c.waves == 4) go(One{}, Two{}, Four{});
        else go(One{}, Two{}, Two{});
      });
    } else {
      auto go = [&](auto tile) {
        using C = decltype(tile);
        launch_tiles(a, C::BM, G ? C::BN / 2 : C::BN, C::NT, [&](dim3 grid) {
          if constexpr (!std::is_same_v<C, MxWide> && !std::is_same_v<C, Mx32>)
            if (d.dtype == MOE_MXFP4) hipLaunchKernelGGL((mx_both_kernel<C, G>), grid, dim3(C::NT), 0, s, a);
          if constexpr (!std::is_same_v<C, Mx256> && !std::is_same_v<C, Mx32Both>) {
            if (d.dtype == MOE_F16) hipLaunchKernelGGL((mx_weights_kernel<C, true, G>), grid, dim3(C::NT), 0, s, a);
            else if (d.dtype == MOE_BF16) hipLaunchKernelGGL((mx_weights_kernel<C, false, G>), grid, dim3(C::NT), 0, s, a);
          }
        });
      };
      if (c.kind == T32 && d.dtype == MOE_MXFP4) go(Mx32Both{});
      else if (c.kind == T32) go(Mx32{});
      else if (c.kind == T64) go(Mx64{});
      else if (c.kind == T128) go(Mx128{});
      else if (c.kind == WIDE) go(MxWide{});
      else go(Mx256{});
    }
  });
  return hipGetLastError();
}

}  // namespace moe
