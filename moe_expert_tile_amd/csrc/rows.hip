// A batch's tokens as rows sorted by expert, and back (include/moe.h): moe_sort,
// moe_permute, moe_unpermute and the last two's gradients.
//
// Sort.  A counting sort that keeps the order of equal keys.  A workgroup's 16
// wavefronts own consecutive runs of its (token, slot) pairs; each counts its
// keys in a table of its own in LDS, prefix sums over wavefronts and experts
// turn the counts into first places, and a second walk over the same pairs
// hands the places out: among 64 pairs a lane's rank is the number of lower
// lanes with its key, found with one ballot per key bit.  Long batches take two
// launches: per-workgroup histograms, then the same walk, in which every
// workgroup sums the histograms of those before it.  Integer sums only, so the
// result is the same in any order of the atomics.  Bound by latency: 64 x 8 ids over
// 128 experts 3.8 us (the kernel), 32768 x 8 over 256 2.7 + 9.3 us in its two kernels (its
// bytes, 3.1 MB, would take 0.6); 8 million pairs 22 + 85 us.
#include "product.h"

namespace moe {
namespace {

constexpr int kSortWaves = 16, kSortThreads = kSortWaves * 64;
constexpr int kSortUnroll = 8;     // groups of 64 pairs whose keys a wavefront loads together

struct SortArgs {
  const int32_t* ids;
  int32_t *pos, *src, *offsets;   // src may be null
  int32_t* hist;                  // [blocks][E], several workgroups only
  int64_t pairs, per;             // per: pairs of a workgroup, a multiple of kSortThreads
  int E, first, bits, blocks;
};

// an expert's place among the local ones; E or more: not here
__device__ __forceinline__ uint32_t local_of(const SortArgs& a, int64_t i, int64_t end) {
  return i < end ? (uint32_t)a.ids[i] - (uint32_t)a.first : 0xffffffffu;
}

// inclusive sum over the wavefront's lanes
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int o = __shfl_up(v, s);
    if (lane >= s) v += o;
  }
  return v;
}

__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(SortArgs a) {
  __shared__ int table[1024];
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) table[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * a.per, hi = min(a.pairs, lo + a.per);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads) {
    const uint32_t e = local_of(a, i, hi);
    if (e < (uint32_t)a.E) atomicAdd(&table[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) a.hist[(int64_t)blockIdx.x * a.E + e] = table[e];
}

template <bool MULTI>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  __shared__ int table[kSortWaves][1024];
  __shared__ int first_place[1024];
  __shared__ int wave_sum[kSortWaves];
  __shared__ int all[MULTI ? kSortThreads : 1], before[MULTI ? kSortThreads : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t run = a.per / kSortWaves;
  const int64_t lo = min(a.pairs, blockIdx.x * a.per + wave * run), hi = min(a.pairs, lo + run);
  int* mine = table[wave];
  uint32_t kept[kSortUnroll];      // the first ones stay for the second walk
#pragma unroll
  for (int u = 0; u < kSortUnroll; ++u) kept[u] = local_of(a, lo + 64 * u + lane, hi);
  for (int e = lane; e < a.E; e += 64) mine[e] = 0;
  int total = 0, earlier = 0;
  if constexpr (MULTI) {
    // column e of the histograms, summed by 1024 / 2^bits threads
    const int col = tid & ((1 << a.bits) - 1), groups = kSortThreads >> a.bits;
    if (col < a.E) {
#pragma unroll 8
      for (int b = tid >> a.bits; b < a.blocks; b += groups) {
        const int v = a.hist[(int64_t)b * a.E + col];
        total += v;
        earlier += b < (int)blockIdx.x ? v : 0;
      }
    }
    all[tid] = total;
    before[tid] = earlier;
  }
  auto walk = [&](auto step) __attribute__((always_inline)) {
    uint32_t e[kSortUnroll];
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) e[u] = kept[u];
    for (int64_t i = lo; i < hi;) {
#pragma unroll
      for (int u = 0; u < kSortUnroll; ++u)
        if (i + 64 * u < hi) step(i + 64 * u + lane, e[u]);
      i += 64 * kSortUnroll;
#pragma unroll
      for (int u = 0; u < kSortUnroll; ++u) e[u] = local_of(a, i + 64 * u + lane, hi);
    }
  };
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  walk([&](int64_t, uint32_t e) __attribute__((always_inline)) {
    if (e < (uint32_t)a.E) atomicAdd(&mine[e], 1);
  });
  __syncthreads();
  // expert tid: its wavefronts' counts to first places, its total and what earlier workgroups have of it
  int held = 0;
  if (tid < a.E) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = table[w][tid];
      table[w][tid] = held;
      held += c;
    }
  }
  if constexpr (MULTI) {
    held = earlier = 0;
    if (tid < a.E) {
      for (int g = tid; g < kSortThreads; g += 1 << a.bits) {
        held += all[g];
        earlier += before[g];
      }
    }
  }
  const int upto = wave_scan(held, lane);
  if (lane == 63) wave_sum[wave] = upto;
  __syncthreads();
  int start = upto - held;
  for (int w = 0; w < wave; ++w) start += wave_sum[w];
  if (tid < a.E) {
    first_place[tid] = start + earlier;
    if (blockIdx.x == 0) {
      a.offsets[tid] = start;
      if (tid == a.E - 1) a.offsets[a.E] = start + held;
    }
  }
  __syncthreads();
  walk([&](int64_t i, uint32_t e) __attribute__((always_inline)) {
    const bool here = e < (uint32_t)a.E;
    uint64_t same = __ballot(here);
    for (int b = 0; b < a.bits; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    int place = -1;
    const int leader = here ? __builtin_ctzll(same) : lane;
    int from = 0;
    if (here && lane == leader) from = first_place[e] + atomicAdd(&mine[e], __popcll(same));
    from = __shfl(from, leader);
    if (here) {
      place = from + __popcll(same & ((1ull << lane) - 1));
      if (a.src) a.src[place] = (int32_t)i;
    }
    if (i < hi) a.pos[i] = place;
  });
}

// --- rows ---------------------------------------------------------------------

struct RowArgs {
  const char *in, *in2;     // (in2: the second input of the sum's gradient)
  char* out;
  const int32_t* pos;
  const float* w;
  float* dw;
  int64_t tokens, rows;
  int64_t ld_in, ld_in2, ld_out;   // bytes
  int k, bytes;                    // bytes of a row
};

template <int T>
struct Type {                      // MOE_BF16, MOE_F16, MOE_F32
  static constexpr int SIZE = T == MOE_F32 ? 4 : 2, VE = 16 / SIZE;   // elements of 16 bytes
  static __device__ __forceinline__ void unpack(v4u32 x, float (&v)[VE]) {
#pragma unroll
    for (int c = 0; c < VE; ++c) {
      if constexpr (T == MOE_F32) v[c] = __uint_as_float(x[c]);
      else v[c] = Elem<T == MOE_F16>::to_float((uint16_t)(x[c / 2] >> (c % 2 * 16)));
    }
  }
  static __device__ __forceinline__ v4u32 pack(const float (&v)[VE]) {
    v4u32 x;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (T == MOE_F32) x[c] = __float_as_uint(v[c]);
      else x[c] = (uint32_t)Elem<T == MOE_F16>::bits(v[2 * c]) | ((uint32_t)Elem<T == MOE_F16>::bits(v[2 * c + 1]) << 16);
    }
    return x;
  }
};

// 16 bytes of a row from byte `at` on.  WHOLE: rows are 16-byte aligned and a
// multiple of 16 bytes long; a buffer descriptor of the row gives zeros past its end.
// Otherwise whole accesses at the elements' alignment, and the last ones by element.
template <int SIZE, bool WHOLE, int POLICY = 0>
struct Row {
  char* p;
  __amdgpu_buffer_rsrc_t rsrc;
  int bytes;
  __device__ __forceinline__ Row(const char* base, int64_t row, int64_t ld, int n, bool there) {
    bytes = there ? n : 0;
    p = const_cast<char*>(base) + (there ? row * ld : 0);
    if constexpr (WHOLE) rsrc = make_rsrc(p, bytes);
  }
  __device__ __forceinline__ v4u32 load(int at) const {
    if constexpr (WHOLE) return __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, 0, POLICY);
    v4u32 x = {0, 0, 0, 0};
    if (at + 16 <= bytes) {
      x = ((const Loose<v4u32, SIZE>*)(p + at))->v;
    } else if (at < bytes) {
#pragma unroll
      for (int c = 0; c < 16 / SIZE - 1; ++c)
        if (at + c * SIZE < bytes) {
          if constexpr (SIZE == 2) x[c / 2] |= (uint32_t)*(const uint16_t*)(p + at + 2 * c) << (c % 2 * 16);
          else x[c] = *(const uint32_t*)(p + at + 4 * c);
        }
    }
    return x;
  }
  __device__ __forceinline__ void store(int at, v4u32 x) const {
    if constexpr (WHOLE) {
      __builtin_amdgcn_raw_buffer_store_b128(x, rsrc, at, 0, POLICY);
    } else if (at + 16 <= bytes) {
      ((Loose<v4u32, SIZE>*)(p + at))->v = x;
    } else if (at < bytes) {
#pragma unroll
      for (int c = 0; c < 16 / SIZE - 1; ++c)
        if (at + c * SIZE < bytes) {
          if constexpr (SIZE == 2) *(uint16_t*)(p + at + 2 * c) = (uint16_t)(x[c / 2] >> (c % 2 * 16));
          else *(uint32_t*)(p + at + 4 * c) = x[c];
        }
    }
  }
};

__device__ __forceinline__ bool held(const RowArgs& a, int p) { return (uint64_t)(int64_t)p < (uint64_t)a.rows; }

// Each wavefront takes U KB of a token's row at a time, reads it once and writes
// it to the token's rows.  Bound by HBM: 8192 x 8 rows of 4096 bf16 columns, 604 MB,
// 105 us (5.7 TB/s); few tokens take 1 KB a wavefront, so that they spread over the CUs.
template <int SIZE, bool WHOLE, int POLICY, int U>
__global__ __launch_bounds__(256) void permute_kernel(RowArgs a) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int runs = (a.bytes + 1024 * U - 1) / (1024 * U);
  const int64_t total = a.tokens * runs;
  for (int64_t i = (int64_t)blockIdx.x * 4 + wave; i < total; i += (int64_t)gridDim.x * 4) {
    const int64_t t = i / runs;
    const int at = (int)(i - t * runs) * 1024 * U + lane * 16;
    const Row<SIZE, WHOLE> from(a.in, t, a.ld_in, a.bytes, true);
    v4u32 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = from.load(at + 1024 * u);
    for (int j = 0; j < a.k; ++j) {
      const int p = a.pos[t * a.k + j];
      if (!held(a, p)) continue;
      const Row<SIZE, WHOLE, POLICY> to(a.out, p, a.ld_out, a.bytes, true);
#pragma unroll
      for (int u = 0; u < U; ++u) to.store(at + 1024 * u, x[u]);
    }
  }
}

// Sum of a token's rows, weighted or not, in slot order in fp32: a wavefront
// takes U KB of a token's row and has the loads of four slots in flight.  Bound by HBM:
// the same size 102 us (5.9 TB/s), weighted or not; a decode step of 64 x 8 x 2048 4.4 us, a launch.
template <int T, bool WEIGHTED, bool WHOLE, int POLICY, int U>
__global__ __launch_bounds__(256) void unpermute_kernel(RowArgs a) {
  typedef Type<T> E;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int runs = (a.bytes + 1024 * U - 1) / (1024 * U);
  const int64_t total = a.tokens * runs;
  constexpr int KC = 4;
  for (int64_t i = (int64_t)blockIdx.x * 4 + wave; i < total; i += (int64_t)gridDim.x * 4) {
    const int64_t t = i / runs;
    const int at = (int)(i - t * runs) * 1024 * U + lane * 16;
    float acc[U][E::VE];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < E::VE; ++c) acc[u][c] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += KC) {
      v4u32 x[KC][U];
      float w[KC];
      bool on[KC];
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int64_t j = t * a.k + min(j0 + c, a.k - 1);
        const int p = a.pos[j];
        on[c] = j0 + c < a.k && held(a, p);
        w[c] = WEIGHTED ? a.w[j] : 1.f;
        const Row<E::SIZE, WHOLE, POLICY> from(a.in, p, a.ld_in, a.bytes, on[c]);
#pragma unroll
        for (int u = 0; u < U; ++u) x[c][u] = from.load(at + 1024 * u);
      }
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        if (!on[c]) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float v[E::VE];
          E::unpack(x[c][u], v);
#pragma unroll
          for (int q = 0; q < E::VE; ++q) acc[u][q] = WEIGHTED ? fmaf(w[c], v[q], acc[u][q]) : acc[u][q] + v[q];
        }
      }
    }
    const Row<E::SIZE, WHOLE> to(a.out, t, a.ld_out, a.bytes, true);
#pragma unroll
    for (int u = 0; u < U; ++u) to.store(at + 1024 * u, E::pack(acc[u]));
  }
}

// Gradients of the sum: a wavefront per slot reads the token's gradient and, for
// the weight's, the slot's row, writes the row's gradient and reduces the product
// in fp32.  A token's slots are neighbouring wavefronts, so its gradient comes
// from the caches after the first of them.  Bound by HBM: 4097 x 8 x 7168, 1.0 GB, 190 us a
// call (5.2 TB/s), 202 with ordinary accesses.
template <int T, bool DROWS, bool DW, bool WHOLE, int POLICY>
__global__ __launch_bounds__(256) void unpermute_back_kernel(RowArgs a) {
  typedef Type<T> E;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t total = a.tokens * a.k;
  for (int64_t i = (int64_t)blockIdx.x * 4 + wave; i < total; i += (int64_t)gridDim.x * 4) {
    const int64_t t = i / a.k;
    const int p = a.pos[i];
    if (!held(a, p)) {
      if (DW && lane == 0) a.dw[i] = 0.f;
      continue;
    }
    const float w = DROWS && a.w ? a.w[i] : 1.f;
    const Row<E::SIZE, WHOLE> grad(a.in, t, a.ld_in, a.bytes, true);
    const Row<E::SIZE, WHOLE, POLICY> row(a.in2, p, a.ld_in2, a.bytes, DW), to(a.out, p, a.ld_out, a.bytes, DROWS);
    float sum = 0.f;
    constexpr int U = 4;
    for (int at = lane * 16; at < a.bytes; at += 1024 * U) {
      v4u32 g[U], x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        g[u] = grad.load(at + 1024 * u);
        if constexpr (DW) x[u] = row.load(at + 1024 * u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float gv[E::VE], xv[E::VE];
        E::unpack(g[u], gv);
        if constexpr (DW) {
          E::unpack(x[u], xv);
#pragma unroll
          for (int c = 0; c < E::VE; ++c) sum = fmaf(gv[c], xv[c], sum);
        }
        if constexpr (DROWS) {
#pragma unroll
          for (int c = 0; c < E::VE; ++c) gv[c] *= w;
          to.store(at + 1024 * u, E::pack(gv));
        }
      }
    }
    if constexpr (DW) {
#pragma unroll
      for (int s = 32; s; s >>= 1) sum += __shfl_xor(sum, s);
      if (lane == 0) a.dw[i] = sum;
    }
  }
}

// --- host -------------------------------------------------------------------

// Pairs of a workgroup.  A short batch is one workgroup's, whose 16 wavefronts share it
// out; a longer one up to 256 workgroups', which each read all histograms.  Calls replayed
// from a graph: 4096 pairs over 128 experts 7.9 us in one workgroup and 8.4 in two
// launches, 8192 10.9 and 8.7; 32768 over 256 experts 9.3 us with 1024 pairs each
// and 10.5 with 2048; 262144 14.5 us with 1024, 12.4 with 2048 and 13.3 with 4096.
int64_t sort_per(int64_t pairs) {
  const int64_t least = pairs <= 4096 ? (pairs > 0 ? pairs : 1) : pairs <= 131072 ? 1024 : 2048, per = (pairs + 255) / 256;
  return ((per > least ? per : least) + kSortThreads - 1) / kSortThreads * kSortThreads;
}

unsigned row_grid(int64_t waves) {
  const int64_t blocks = (waves + 3) / 4;
  return (unsigned)(blocks < 65536 ? blocks : 65536);
}

template <class F>
void with_type(int dtype, F f) {
  if (dtype == MOE_BF16) f(std::integral_constant<int, MOE_BF16>{});
  else if (dtype == MOE_F16) f(std::integral_constant<int, MOE_F16>{});
  else f(std::integral_constant<int, MOE_F32>{});
}
template <class F>
void with_flag(bool b, F f) {
  if (b) f(std::true_type{});
  else f(std::false_type{});
}

// The sorted rows' accesses: what is larger than the last-level cache (256 MB) is
// read and written past it, 8192 x 8 rows of 4096 bf16 columns 122 -> 103 us; smaller
// ones may still be there, or be wanted from there by the experts' products.
template <class F>
void with_access(bool whole, int64_t bytes, F f) {
  using Ordinary = std::integral_constant<int, 0>;
  using Nontemporal = std::integral_constant<int, 2>;
  if (whole && bytes > (256ll << 20)) f(std::true_type{}, Nontemporal{});
  else if (whole) f(std::true_type{}, Ordinary{});
  else f(std::false_type{}, Ordinary{});
}

bool whole(const void* p, int64_t ld, int64_t bytes) { return !p || (aligned_to(p, 16) && ld % 16 == 0 && bytes % 16 == 0); }

}  // namespace

size_t sort_ws_bytes(int64_t pairs, int E) {
  const int64_t per = sort_per(pairs), blocks = (pairs + per - 1) / per;
  return blocks > 1 ? (size_t)blocks * E * 4 : 0;
}

hipError_t launch_sort(int64_t pairs, int E, int first, const int32_t* ids, int32_t* pos, int32_t* src,
                       int32_t* offsets, void* ws, hipStream_t s) {
  SortArgs a = {ids, pos, src, offsets, (int32_t*)ws, pairs, sort_per(pairs), E, first, 0, 1};
  while ((1 << a.bits) < E) ++a.bits;
  a.blocks = (int)((pairs + a.per - 1) / a.per);
  if (a.blocks <= 1) {
    hipLaunchKernelGGL((sort_place_kernel<false>), dim3(1), dim3(kSortThreads), 0, s, a);
  } else {
    hipLaunchKernelGGL(sort_hist_kernel, dim3((unsigned)a.blocks), dim3(kSortThreads), 0, s, a);
    hipLaunchKernelGGL((sort_place_kernel<true>), dim3((unsigned)a.blocks), dim3(kSortThreads), 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_permute(const moe_rows_desc& d, const void* x, const int32_t* pos, void* rows, hipStream_t s) {
  const int size = d.dtype == MOE_F32 ? 4 : 2;
  RowArgs a = {};
  a.in = (const char*)x; a.out = (char*)rows; a.pos = pos;
  a.tokens = d.tokens; a.rows = d.rows;
  a.ld_in = d.ld_x * size; a.ld_out = d.ld_rows * size;
  a.k = d.top_k; a.bytes = d.cols * size;
  const bool all = whole(x, a.ld_in, a.bytes) && whole(rows, a.ld_out, a.bytes);
  const int64_t long_runs = d.tokens * ((a.bytes + 4095) / 4096), short_runs = d.tokens * ((a.bytes + 1023) / 1024);
  const bool few = long_runs < 2048;     // short runs, so that few tokens spread over the CUs
  const dim3 grid(row_grid(few ? short_runs : long_runs)), block(256);
  with_flag(size == 2, [&](auto two) {
    with_access(all, d.tokens * d.top_k * a.bytes, [&](auto w, auto policy) {
      constexpr int SIZE = decltype(two)::value ? 2 : 4, P = decltype(policy)::value;
      constexpr bool W = decltype(w)::value;
      if (few) hipLaunchKernelGGL((permute_kernel<SIZE, W, P, 1>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((permute_kernel<SIZE, W, P, 4>), grid, block, 0, s, a);
    });
  });
  return hipGetLastError();
}

hipError_t launch_unpermute(const moe_rows_desc& d, const void* rows, const int32_t* pos, const float* w, void* out,
                            hipStream_t s) {
  const int size = d.dtype == MOE_F32 ? 4 : 2;
  RowArgs a = {};
  a.in = (const char*)rows; a.out = (char*)out; a.pos = pos; a.w = w;
  a.tokens = d.tokens; a.rows = d.rows;
  a.ld_in = d.ld_rows * size; a.ld_out = d.ld_x * size;
  a.k = d.top_k; a.bytes = d.cols * size;
  const bool all = whole(rows, a.ld_in, a.bytes) && whole(out, a.ld_out, a.bytes);
  const int64_t long_runs = d.tokens * ((a.bytes + 4095) / 4096), short_runs = d.tokens * ((a.bytes + 1023) / 1024);
  const bool few = long_runs < 2048;
  const dim3 grid(row_grid(few ? short_runs : long_runs)), block(256);
  with_type(d.dtype, [&](auto t) {
    with_flag(w != nullptr, [&](auto weighted) {
      with_access(all, d.tokens * d.top_k * a.bytes, [&](auto wh, auto policy) {
        constexpr int T = decltype(t)::value, P = decltype(policy)::value;
        constexpr bool G = decltype(weighted)::value, W = decltype(wh)::value;
        if (few) hipLaunchKernelGGL((unpermute_kernel<T, G, W, P, 1>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((unpermute_kernel<T, G, W, P, 4>), grid, block, 0, s, a);
      });
    });
  });
  return hipGetLastError();
}

hipError_t launch_unpermute_backward(const moe_rows_desc& d, const void* rows, const int32_t* pos, const float* w,
                                     const void* d_out, void* d_rows, float* dw, hipStream_t s) {
  const int size = d.dtype == MOE_F32 ? 4 : 2;
  RowArgs a = {};
  a.in = (const char*)d_out; a.in2 = (const char*)rows; a.out = (char*)d_rows; a.pos = pos; a.w = w; a.dw = dw;
  a.tokens = d.tokens; a.rows = d.rows;
  a.ld_in = d.ld_x * size; a.ld_in2 = d.ld_rows * size; a.ld_out = d.ld_d_rows * size;
  a.k = d.top_k; a.bytes = d.cols * size;
  const bool all = whole(d_out, a.ld_in, a.bytes) && (!dw || whole(rows, a.ld_in2, a.bytes)) &&
                   whole(d_rows, a.ld_out, a.bytes);
  const dim3 grid(row_grid(d.tokens * d.top_k)), block(256);
  with_type(d.dtype, [&](auto t) {
    with_access(all, d.tokens * d.top_k * a.bytes, [&](auto wh, auto policy) {
      constexpr int T = decltype(t)::value, P = decltype(policy)::value;
      constexpr bool W = decltype(wh)::value;
      if (d_rows && dw) hipLaunchKernelGGL((unpermute_back_kernel<T, true, true, W, P>), grid, block, 0, s, a);
      else if (d_rows) hipLaunchKernelGGL((unpermute_back_kernel<T, true, false, W, P>), grid, block, 0, s, a);
      else hipLaunchKernelGGL((unpermute_back_kernel<T, false, true, W, P>), grid, block, 0, s, a);
    });
  });
  return hipGetLastError();
}

}  // namespace moe
