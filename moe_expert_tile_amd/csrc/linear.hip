// Dense product with its epilogue, out = act(x w^T + bias) + residual
// (include/moe.h, moe_linear), and its gradients (moe_linear_backward).
//
// Every product here is C[m][n] = sum_k A(m, k) B(n, k); 16-bit operands, fp32
// accumulation in MFMA registers.
//   * Many rows: v_mfma_f32_32x32x16 over tiles staged through LDS by
//     direct-to-LDS buffer loads into a two-stage ring (K steps of 64), 16-byte
//     chunks XOR-swizzled so that operand fetches are free of bank conflicts.
//     An operand is contiguous along k (x and w in the forward product) or
//     across it (w in dx = dz w, both in dw = dz^T x); the latter is staged as
//     it lies and transposed on the way out of LDS (ds_read_b64_tr_b16).
//     Rows past an operand's end and chunks past K get an offset past the
//     buffer descriptor's bound, where loads return zeros.  Few tiles are also
//     split along K: fp32 partial sums in the workspace, summed in order by a
//     second launch, so results do not depend on timing.
//   * Few rows (decode): the weights are read once, straight into MFMA
//     operand registers (v_mfma_f32_16x16x32, 16 weight rows a workgroup), the
//     workgroup's wavefronts sharing out K and joining their sums in LDS.
// The first MFMA operand is the weight tile, so a lane ends with 4 consecutive
// output columns per accumulator quad, and a gated activation's pair of columns
// sits in one lane.
//
// Gradients.  dz = d_out act'(pre) is formed once (rounded to the operand type,
// which the matrix cores need; its column sums for the bias are taken before
// the rounding), then dx = dz w and dw = dz^T x are products of the same form.
// Without an activation dz is d_out itself where its type and layout allow.
// Fp16's range is narrow for that (gradients of a mean over many tokens lie
// below its smallest step): a dz rounded to fp16 is multiplied by the power of two
// that brings its largest value to 2^14 .. 2^15, found in a pass of its own, and the
// products' sums by its inverse.  A rounding is then off by half a step, 2^-11 of
// the value, or 2^-39 of the largest one, whichever is more.
#include "product.h"

namespace moe {
namespace {

constexpr int kCus = 256;                    // compute units the work is split for

template <int ACT>
__device__ __forceinline__ float slope(float z) {
  if constexpr (ACT == MOE_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  // far out the smooth activations' slopes are 0 and 1 to the last bit, and
  // their terms would be infinity times zero
  if (fabsf(z) > 100.f) return z > 0.f ? 1.f : 0.f;
  if constexpr (ACT == MOE_ACT_SILU) {
    return logistic(z) * (1.0f + z * logistic(-z));
  } else if constexpr (ACT == MOE_ACT_GELU) {
    return 0.5f * (1.0f + erff(z * kSqrtHalf)) + z * __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z) * kInvSqrt2Pi;
  } else {
    const float u = kTwoSqrt2OverPi * (z + kCubic * z * z * z);
    const float p = logistic(u);
    return p + z * p * logistic(-u) * kTwoSqrt2OverPi * (1.0f + 3.0f * kCubic * z * z);
  }
}

// --- epilogue ---------------------------------------------------------------

struct Epilogue {
  const uint16_t* bias;
  const void* res;
  uint16_t* pre;
  void* out;
  int64_t M, ldr, ldp, ldo;
  int N;         // output columns; a gated product has N gate and N up columns before the activation
  int act;
  int out_f32;
  const float* scale;   // a factor on the sums of a gradient's product, in device memory, or null
};

// The bias of columns n .. n + W - 1 (and of the up columns), and the residual
// there of row m; zeros without one.  Columns from N on read zeros.
template <bool F16, bool GATED, int W>
__device__ __forceinline__ void load_bias(const Epilogue& e, int n, float (&bz)[W], float (&bu)[W]) {
#pragma unroll
  for (int c = 0; c < W; ++c) bz[c] = bu[c] = 0.f;
  if (e.bias && n < e.N) {
    load16<F16>(e.bias + n, e.N - n, bz);
    if constexpr (GATED) load16<F16>(e.bias + e.N + n, e.N - n, bu);
  }
}
template <bool F16, int W>
__device__ __forceinline__ void load_residual(const Epilogue& e, int64_t m, int n, float (&r)[W]) {
#pragma unroll
  for (int c = 0; c < W; ++c) r[c] = 0.f;
  if (e.res && m < e.M && n < e.N) {
    if (e.out_f32) load32((const float*)e.res + m * e.ldr + n, e.N - n, r);
    else load16<F16>((const uint16_t*)e.res + m * e.ldr + n, e.N - n, r);
  }
}

template <bool F16, int W>
__device__ __forceinline__ void store_out(const Epilogue& e, int64_t m, int n, const float (&y)[W]) {
  if (e.out_f32) store32((float*)e.out + m * e.ldo + n, e.N - n, y);
  else store16<F16>((uint16_t*)e.out + m * e.ldo + n, e.N - n, y);
}

// Columns n .. n + W - 1 of row m, of which those below N exist (n < N, m < M):
// z the sums, u the up columns' sums of a gated product, bz, bu and r as above.
template <bool F16, bool GATED, int W>
__device__ __forceinline__ void finish(const Epilogue& e, int64_t m, int n, float (&z)[W], float (&u)[W],
                                       const float (&bz)[W], const float (&bu)[W], const float (&r)[W]) {
  const int left = e.N - n;
#pragma unroll
  for (int c = 0; c < W; ++c) {
    z[c] += bz[c];
    if constexpr (GATED) u[c] += bu[c];
  }
  if (e.pre) {
    store16<F16>(e.pre + m * e.ldp + n, left, z);
    if constexpr (GATED) store16<F16>(e.pre + m * e.ldp + e.N + n, left, u);
  }
  float y[W];
  if constexpr (GATED) {
#pragma unroll
    for (int c = 0; c < W; ++c) y[c] = z[c] * logistic(z[c]) * u[c];
  } else {
    activate_all(e.act, z, y);
  }
#pragma unroll
  for (int c = 0; c < W; ++c) y[c] += r[c];
  store_out<F16>(e, m, n, y);
}

// --- tiled product ----------------------------------------------------------
//
// Rates (bf16, 8192 rows, a call among others): 8192 x 4096 (gated) x 7168 387 us,
// 1.24 PFLOP/s; 8192 x 2048 x 7168 190 us, 1.26; its dx 220 us, 1.09, its dw 202
// us, 1.19; 8192 x 7168 x 2048 220 us, 1.10, with a residual 276.  (The library's
// plain 8192 x 4096 x 7168: 359-370 us in the same run, 307 at best.)  Counters of the gated one: 1.86 GHz under load, MFMA busy 62% of the
// time, LDS 24%, no bank conflicts, wavefronts waiting 36%: what is left is the
// loads' latency per CU.  Other shapes measured: 256 x 256 as four wavefronts of
// 128 x 128 5-10% slower; 256 x 128 with three stages, next to 128 x 256, 0.2% less
// over 104 products; the stage's first operand fetches moved in front of the
// meeting of the wavefronts within 1%.  The two-stage ring of a 256 x 256 tile takes
// 128 KB of LDS, so a CU holds one workgroup of it, two of 128 x 128 and three of
// 64 x 128, whose epilogues overlap other workgroups' multiplications: they win
// with little K or many splits (gated 20000 x 512 x 1024 69 us in 256 x 256, 64 us in
// 128 x 128).  Between them 128 x 256 keeps three stages in 144 KB, two of them in
// flight, for sums that are long where output tiles are few (8192 x 512 x 4096
// 59 us without it, 51 us with it; dw of 8192 x 256 x 7168 58 and 52 us).

struct ProdArgs {
  const uint16_t *a, *b;   // A [M, K] or, across k, [K, M]; B [N or 2N, K] or [K, N]
  int64_t lda, ldb;
  int64_t K;
  int64_t kper;            // K of one split (a multiple of 64)
  float* part;             // splits > 1: [splits][M][pitch] partial sums
  int64_t pitch;
  int up_col;              // ... where the up columns start in a row of them
  int n_mt, n_nt, splits;
  Epilogue e;
};

constexpr int kBK = 64;    // K step

template <int BM_, int BN_, int WAVES_M, int WAVES_N, int STAGES_ = 2>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, STAGES = STAGES_;
  static constexpr int NW = WAVES_M * WAVES_N, NT = NW * 64;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int FM = WM / 32, FN = WN / 32;
  static constexpr int KK = kBK / 16;             // MFMA steps a stage
  static constexpr int A_ELEMS = BM * kBK, B_ELEMS = BN * kBK;
  static constexpr int STAGE = A_ELEMS + B_ELEMS;
  // the epilogue's staging: a wave's columns (gate, then up) of 32 rows in
  // fp32, rows 4 floats further apart than they are long, so that the lanes'
  // 16-byte accesses to different rows fall on different banks
  template <bool GATED>
  struct staged {
    static constexpr int FG = GATED ? FN / 2 : FN;
    static constexpr int CW = FG * 32;
    static constexpr int PITCH = FN * 32 + 4;
  };
  static constexpr int EPI_ELEMS = NW * 32 * (FN * 32 + 4) * 2;
  static constexpr int LDS_ELEMS = STAGES * STAGE > EPI_ELEMS ? STAGES * STAGE : EPI_ELEMS;
  static constexpr int A_LOADS = BM / 8 / NW;     // 1 KB wave loads a stage (8 rows of 128 bytes)
  static constexpr int B_LOADS = BN / 8 / NW;
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "whole wave loads");
  static_assert(B_LOADS % 2 == 0, "gate and up rows in separate loads");
  static_assert(LDS_ELEMS * 2 <= 160 * 1024, "LDS");
};
typedef Tile<256, 256, 2, 4> Tile256;
typedef Tile<256, 256, 4, 2> Tile256G;    // gated: each wave's columns hold as many gate as up ones
typedef Tile<128, 128, 2, 2> Tile128;
typedef Tile<64, 128, 2, 2> Tile64;
typedef Tile<128, 256, 2, 4, 3> TileWide;

// An operand's tile in LDS.  Along k: ROWS rows of 64 k, row r's 16-byte chunk c
// at c ^ (r / 2) % 8.  Across k: 64 rows (k) of ROWS values, row r's chunk c at
// c ^ across_swizzle(r): a transposing read takes 4 rows x 32 values a half
// wavefront, 64 bytes of each row, which so fall on different banks (rows of
// 128 bytes are half a bank line apart already).  Either way a
// wavefront fills 1 KB at a time in LDS order, and the lane picks the chunk of
// global memory that belongs there.
template <int ROWS>
__device__ __forceinline__ int across_swizzle(int r) {
  return ROWS >= 128 ? 4 * (r % 4) : 4 * ((r / 2) % 2);
}
template <int ROWS, int NW, bool ACROSS>
struct Staged {
  static constexpr int LOADS = ROWS / 8 / NW;        // 1 KB loads a stage and wave
  static constexpr int LPR = ACROSS ? ROWS / 8 : 8;  // lanes (chunks) a row
  static constexpr int RPL = 64 / LPR;               // rows a load
  uint32_t off[LOADS];
  int chunk;   // along k: this lane's logical chunk of a row (the same in all of its loads)

  // rows: the operand's rows (across k, its columns) from the tile's first one on
  __device__ __forceinline__ void init(int wave, int lane, int rows, int64_t ld) {
    chunk = (lane % 8) ^ ((wave * 4 + lane / 16) % 8);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int r = (wave + i * NW) * RPL + lane / LPR;
      if constexpr (ACROSS) {
        const int c = (lane % LPR) ^ across_swizzle<ROWS>(r);
        off[i] = c * 8 < rows ? 2u * ((uint32_t)r * (uint32_t)ld + c * 8) : kPastEnd;
      } else {
        off[i] = r < rows ? 2u * ((uint32_t)r * (uint32_t)ld + chunk * 8) : kPastEnd;
      }
    }
  }
};

// the transposing LDS read of a 32-row MFMA operand block: lane l gets row
// l % 32, k = 8 (l / 32) .. + 7, as two reads of 4 k each.  (`restrict` gives
// the reads an alias scope; without one the compiler lets them wait for every
// load to LDS in flight, the next stage's among them: dx of 8192 x 4096 x 7168
// 546 us, with it 470 us.)
template <class V8>
__device__ __forceinline__ V8 read_across(const uint16_t* __restrict p, int pitch) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  struct { s16x4 lo, hi; } v;
  v.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  v.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * pitch));
  return __builtin_bit_cast(V8, v);
}

template <class C, bool F16, bool GATED, bool PART, bool AX, bool BX>
__global__ __launch_bounds__(C::NT) __attribute__((amdgpu_waves_per_eu(C::NW == 8 ? 2 : 1)))
void product_kernel(ProdArgs g) {
  static_assert(!GATED || !BX, "gated weights lie along k");
  typedef typename Elem<F16>::v8 v8;
  __shared__ __attribute__((aligned(1024))) uint16_t lds[C::LDS_ELEMS];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int WAVES_N = C::BN / C::WN;
  const int wave_m = wave / WAVES_N, wave_n = wave % WAVES_N;
  constexpr int HB = GATED ? C::BN / 2 : C::BN;    // output columns of a tile

  const int tiles = g.n_mt * g.n_nt;
  int t = xcd_order(blockIdx.x, tiles * g.splits);
  const int split = t / tiles;
  t -= split * tiles;
  const int grp = t / (8 * g.n_nt), rows8 = min(8, g.n_mt - grp * 8);
  t -= grp * 8 * g.n_nt;
  const int mt = grp * 8 + t % rows8, nt = t / rows8;

  const int64_t m0 = (int64_t)mt * C::BM;
  const int n0 = nt * HB;
  const int arows = (int)min((int64_t)C::BM, g.e.M - m0);
  const int brows = min(HB, g.e.N - n0);
  const int64_t kb = split * g.kper;
  const int64_t ke = min(g.K, kb + g.kper);
  const int KT = ke > kb ? (int)((ke - kb + kBK - 1) / kBK) : 0;
  const int klast = (int)(ke - kb) - (KT - 1) * kBK;   // columns of the last stage

  static_assert(C::NW % 2 == 0, "a wave's loads are all of one row parity");
  Staged<C::BM, C::NW, AX> sta;
  Staged<C::BN, C::NW, BX> stb;
  sta.init(wave, lane, arows, g.lda);
  stb.init(wave, lane, brows, g.ldb);
  if constexpr (GATED) {
    // the second half of the tile holds the up rows
#pragma unroll
    for (int i = C::B_LOADS / 2; i < C::B_LOADS; ++i) stb.off[i] = stb.off[i - C::B_LOADS / 2];
  }
  // (descriptors end with a whole 16-byte chunk: a length that is no multiple
  // of 8 is dz's, whose rows have zeros up to one)
  const int64_t along_a = KT ? ((int64_t)(arows - 1) * g.lda + (ke - kb + 7) / 8 * 8) * 2 : 0;
  const int64_t along_b = KT ? ((int64_t)(brows - 1) * g.ldb + (ke - kb)) * 2 : 0;
  const int arows8 = (arows + 7) / 8 * 8;
  const uint16_t* a_base = AX ? g.a + kb * g.lda + m0 : g.a + m0 * g.lda + kb;
  const uint16_t* b_base = BX ? g.b + kb * g.ldb + n0 : g.b + (int64_t)n0 * g.ldb + kb;
  const __amdgpu_buffer_rsrc_t a_all = make_rsrc(a_base, AX ? 0 : along_a);
  const __amdgpu_buffer_rsrc_t b_all = make_rsrc(b_base, BX ? 0 : along_b);
  const __amdgpu_buffer_rsrc_t u_all = GATED ? make_rsrc(b_base + (int64_t)g.e.N * g.ldb, along_b) : b_all;
  // stage k into half k % 2 of the ring.  Along k, `last` masks the chunks past
  // the end of K (each is whole or absent, or dz's with its zeros);
  // across k, a stage has a descriptor of its own that ends with its last row.
  auto ring = [&](int k) __attribute__((always_inline)) {
    return C::STAGES == 2 ? lds + (k & 1) * C::STAGE : lds + (k % C::STAGES) * C::STAGE;
  };
  auto issue = [&](int k, auto last_tag) __attribute__((always_inline)) {
    constexpr bool LAST = decltype(last_tag)::value;
    char* base = (char*)ring(k);
    const int koff = 2 * kBK * k;
    const int64_t rows = LAST ? klast : kBK;
    const __amdgpu_buffer_rsrc_t ar =
        AX ? make_rsrc(a_base + (int64_t)k * kBK * g.lda, ((rows - 1) * g.lda + arows8) * 2) : a_all;
    const __amdgpu_buffer_rsrc_t br =
        BX ? make_rsrc(b_base + (int64_t)k * kBK * g.ldb, ((rows - 1) * g.ldb + brows) * 2) : b_all;
#pragma unroll
    for (int i = 0; i < C::A_LOADS; ++i)
      load_lds(ar, base + (wave + i * C::NW) * 1024,
               !LAST || AX || sta.chunk * 8 < klast ? sta.off[i] : kPastEnd, AX ? 0 : koff);
#pragma unroll
    for (int i = 0; i < C::B_LOADS; ++i)
      load_lds(GATED && i >= C::B_LOADS / 2 ? u_all : br, base + 2 * C::A_ELEMS + (wave + i * C::NW) * 1024,
               !LAST || BX || stb.chunk * 8 < klast ? stb.off[i] : kPastEnd, BX ? 0 : koff);
  };

  // this wave's weight rows inside the tile (32 a block)
  int prow[C::FN];
#pragma unroll
  for (int i = 0; i < C::FN; ++i) {
    if constexpr (GATED) {
      constexpr int HW = C::WN / 2;
      prow[i] = i < C::FN / 2 ? wave_n * HW + 32 * i : HB + wave_n * HW + 32 * (i - C::FN / 2);
    } else {
      prow[i] = wave_n * C::WN + 32 * i;
    }
  }
  const int lrow = lane & 31, lhalf = lane >> 5, rsw = (lrow / 2) % 8;
  // transposing reads: this lane's row (k) among 16, its place among 32 values
  const int xrow = 8 * lhalf + (lane & 15) / 4;
  const int xcol = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1), xsub = (lane & 1) * 4;
  auto across = [&](int block, auto pitch) __attribute__((always_inline)) {
    constexpr int P = decltype(pitch)::value;
    return xrow * P + (((block / 8) ^ across_swizzle<P>(xrow)) + xcol) * 8 + xsub;
  };

  f32x16 acc[C::FN][C::FM];
#pragma unroll
  for (int i = 0; i < C::FN; ++i)
#pragma unroll
    for (int j = 0; j < C::FM; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  using Mid = std::integral_constant<bool, false>;
  using Last = std::integral_constant<bool, true>;
  // one stage: wait for its loads (a three-stage ring leaves the next stage's in
  // flight) and for every wave's reads of the part refilled next, refill that
  // (next: 0 nothing, 1 a whole stage, 2 the last one), multiply with the
  // operand fetches one MFMA step ahead
  auto step = [&](int k, auto next_tag, auto flying_tag) __attribute__((always_inline)) {
    constexpr int NEXT = decltype(next_tag)::value;
    constexpr int FLYING = decltype(flying_tag)::value ? C::A_LOADS + C::B_LOADS : 0;   // loads that may be outstanding
    static_assert(FLYING < 16, "vector memory counter's low bits");
    __builtin_amdgcn_s_waitcnt(0x70 | FLYING);   // vmcnt(FLYING) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    const uint16_t* sa = ring(k);
    const uint16_t* sb = sa + C::A_ELEMS;
    v8 pw[2][C::FN], px[2][C::FM];
    auto fetch = [&](int kk) __attribute__((always_inline)) {
      const int phys = ((2 * kk + lhalf) ^ rsw) * 8;
#pragma unroll
      for (int i = 0; i < C::FN; ++i) {
        if constexpr (BX) pw[kk & 1][i] = read_across<v8>(sb + 16 * kk * C::BN + across(prow[i], std::integral_constant<int, C::BN>{}), C::BN);
        else pw[kk & 1][i] = *(const v8*)(sb + (prow[i] + lrow) * kBK + phys);
      }
#pragma unroll
      for (int j = 0; j < C::FM; ++j) {
        const int at = wave_m * C::WM + 32 * j;
        if constexpr (AX) px[kk & 1][j] = read_across<v8>(sa + 16 * kk * C::BM + across(at, std::integral_constant<int, C::BM>{}), C::BM);
        else px[kk & 1][j] = *(const v8*)(sa + (at + lrow) * kBK + phys);
      }
    };
    fetch(0);
    if constexpr (NEXT == 1) issue(k + C::STAGES - 1, Mid{});
    if constexpr (NEXT == 2) issue(k + C::STAGES - 1, Last{});
#pragma unroll
    for (int kk = 0; kk < C::KK; ++kk) {
      if (kk + 1 < C::KK) fetch(kk + 1);
#pragma unroll
      for (int i = 0; i < C::FN; ++i)
#pragma unroll
        for (int j = 0; j < C::FM; ++j) acc[i][j] = Elem<F16>::mfma32(pw[kk & 1][i], px[kk & 1][j], acc[i][j]);
    }
    // LDS reads of step 0, the refill, then each step's reads before the
    // previous step's MFMAs
    constexpr int READS = C::FN * (BX ? 2 : 1) + C::FM * (AX ? 2 : 1);
    __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    if constexpr (NEXT != 0) __builtin_amdgcn_sched_group_barrier(0x10, C::A_LOADS + C::B_LOADS, 0);
#pragma unroll
    for (int kk = 0; kk < C::KK; ++kk) {
      if (kk + 1 < C::KK) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
      __builtin_amdgcn_sched_group_barrier(0x8, C::FN * C::FM, 0);
    }
  };
  if (KT > 0) {
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    constexpr int AHEAD = C::STAGES - 1;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (k + 1 < KT) issue(k, Mid{});
      else if (k + 1 == KT) issue(k, Last{});
    }
    using Fly = std::integral_constant<bool, (C::STAGES > 2)>;
    int k = 0;
    for (; k + AHEAD + 1 < KT; ++k) step(k, I1{}, Fly{});
    if (k + AHEAD < KT) step(k++, I2{}, Fly{});
    if constexpr (C::STAGES > 2)
      if (k + 1 < KT) step(k++, I0{}, Fly{});
    step(k, I0{}, Mid{});
  }

  // Epilogue: 32 rows of a wave's columns at a time go through LDS (each wave
  // has its own part of it), so that lanes hold neighbouring columns and every
  // global access covers whole lines.
  __builtin_amdgcn_s_waitcnt(0x70);
  __builtin_amdgcn_s_barrier();   // every wave is done with the operands
  constexpr int FG = C::template staged<GATED>::FG, CW = C::template staged<GATED>::CW;
  constexpr int PITCH = C::template staged<GATED>::PITCH;
  float* stage = (float*)lds + wave * 32 * PITCH;
  const int ncol = n0 + (GATED ? wave_n * (C::WN / 2) : wave_n * C::WN);
  constexpr int LPR = CW / 8, RPP = 64 / LPR;   // lanes a row (8 columns each), rows a pass
  const int er = lane / LPR, ec = (lane % LPR) * 8;
  const int n = ncol + ec;
  // neither activation nor pre: short enough to unroll over the passes
  const bool light = !GATED && !g.e.pre && g.e.act == MOE_ACT_NONE;
  // gradients and most products: 16-bit sums alone, whole 8 columns
  constexpr bool SCALES = F16 && BX;   // gradients' products in fp16 alone
  const float factor = SCALES && g.e.scale ? *g.e.scale : 1.0f;
  const bool plain = light && !g.e.bias && !g.e.res && !g.e.out_f32 && g.e.N % 8 == 0;
  float bz[8], bu[8];
  if constexpr (!PART) load_bias<F16, GATED>(g.e, n, bz, bu);
  auto rows32 = [&](auto jt) __attribute__((always_inline)) {
    constexpr int j = decltype(jt)::value;
#pragma unroll
    for (int i = 0; i < C::FN; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(float4*)(stage + lrow * PITCH + 32 * i + 8 * q + 4 * lhalf) =
            make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
    __builtin_amdgcn_wave_barrier();
    const int64_t mj = m0 + wave_m * C::WM + 32 * j;
    auto staged8 = [&](int r, int col, float (&v)[8]) __attribute__((always_inline)) {
      const float4 a = *(const float4*)(stage + r * PITCH + col), b = *(const float4*)(stage + r * PITCH + col + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    };
    // The residual is read ahead of the stores: the compiler may not move it
    // there, as it may be the output itself (a lane stores what it has read).
    constexpr int PASSES = 32 / RPP;
    if constexpr (PART) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int r = p * RPP + er;
        const int64_t m = mj + r;
        float z[8], u[8];
        staged8(r, ec, z);
        if constexpr (GATED) staged8(r, CW + ec, u);
        if (m < g.e.M && n < g.e.N) {
          float* to = g.part + (split * g.e.M + m) * g.pitch + n;
          store32(to, g.up_col - n, z);
          if constexpr (GATED) store32(to + g.up_col, g.up_col - n, u);
        }
      }
    } else if (plain) {
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int r = p * RPP + er;
        const int64_t m = mj + r;
        float z[8];
        staged8(r, ec, z);
        if constexpr (SCALES) {
#pragma unroll
          for (int c = 0; c < 8; ++c) z[c] *= factor;
        }
        if (m < g.e.M && n < g.e.N) store16<F16, 8, true>((uint16_t*)g.e.out + m * g.e.ldo + n, 8, z);
      }
    } else if (light) {
      float res[PASSES][8];
#pragma unroll
      for (int p = 0; p < PASSES; ++p) load_residual<F16>(g.e, mj + p * RPP + er, n, res[p]);
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int r = p * RPP + er;
        const int64_t m = mj + r;
        float z[8];
        staged8(r, ec, z);
#pragma unroll
        for (int c = 0; c < 8; ++c) z[c] = (SCALES ? z[c] * factor : z[c]) + (bz[c] + res[p][c]);
        if (m < g.e.M && n < g.e.N) store_out<F16>(g.e, m, n, z);
      }
    } else {
      float res[8];
      load_residual<F16>(g.e, mj + er, n, res);
#pragma unroll 1
      for (int r = er; r < 32; r += RPP) {
        const int64_t m = mj + r;
        float z[8], u[8], next[8];
        load_residual<F16>(g.e, r + RPP < 32 ? m + RPP : g.e.M, n, next);
        staged8(r, ec, z);
        if constexpr (GATED) staged8(r, CW + ec, u);
        if (m < g.e.M && n < g.e.N) finish<F16, GATED>(g.e, m, n, z, u, bz, bu, res);
#pragma unroll
        for (int c = 0; c < 8; ++c) res[c] = next[c];
      }
    }
    __builtin_amdgcn_wave_barrier();
  };
  rows32(std::integral_constant<int, 0>{});
  if constexpr (C::FM > 1) rows32(std::integral_constant<int, 1>{});
  if constexpr (C::FM > 2) {
    rows32(std::integral_constant<int, 2>{});
    rows32(std::integral_constant<int, 3>{});
  }
  static_assert(C::FM == 1 || C::FM == 2 || C::FM == 4, "row blocks");
}

// Sums of a split product's partial sums, in split order, and the epilogue.
// Memory bound (8192 x 256 in 4 splits, 42 MB, 8.4 us) or, with little to write,
// bound by the partial sums' latency: four of them are read together and a
// workgroup is one wavefront, so that small outputs spread over the CUs
// (40 x 512 x 4096 in 16 splits 12.0 us with one after the other, 9.3 us so).
template <bool F16, bool GATED>
__global__ __launch_bounds__(64) void join_kernel(ProdArgs g) {
  const int quads = (g.e.N + 3) / 4;
  const int64_t total = g.e.M * quads;
  for (int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 64) {
    const int64_t m = i / quads;
    const int n = (int)(i - m * quads) * 4;
    float z[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) {
      const float* p = g.part + (s * g.e.M + m) * g.pitch + n;
      const float4 x = *(const float4*)p;
      z[0] += x.x; z[1] += x.y; z[2] += x.z; z[3] += x.w;
      if constexpr (GATED) {
        const float4 y = *(const float4*)(p + g.up_col);
        u[0] += y.x; u[1] += y.y; u[2] += y.z; u[3] += y.w;
      }
    }
    if constexpr (F16 && !GATED) {
      if (g.e.scale) {
#pragma unroll
        for (int c = 0; c < 4; ++c) z[c] *= *g.e.scale;
      }
    }
    float bz[4], bu[4], r[4];
    load_bias<F16, GATED>(g.e, n, bz, bu);
    load_residual<F16>(g.e, m, n, r);
    finish<F16, GATED>(g.e, m, n, z, u, bz, bu, r);
  }
}

// --- few rows ---------------------------------------------------------------
//
// Bound by reading the weights: one row through 7168 x 2048 (29 MB) takes 7.6
// us (9.1 with the weights in no cache), of which about 2.5 us any launch takes; 8 K steps' loads in flight a
// wavefront instead of 4, all issued before the first is waited for, took it
// there from 9.6 us.
// A workgroup owns 16 output columns (PART: of one split of K); its wavefronts
// take K in steps of 32 in turn.  Operand lane layout of v_mfma_f32_16x16x32: row (or column) lane % 16,
// k = 8 (lane / 16) .. + 7, so a lane's operand is one 16-byte load; result
// lane: column (token) lane % 16, rows (weight rows) 4 (lane / 16) .. + 3.
constexpr int kFewWaves = 8;

// U K steps have their loads in flight together.
template <int TT, bool F16, bool GATED, bool PART, int U>
__global__ __launch_bounds__(kFewWaves * 64) void few_rows_kernel(ProdArgs g) {
  typedef typename Elem<F16>::v8 v8;
  constexpr int NB = GATED ? 2 : 1;
  __shared__ float4 part[kFewWaves][NB][TT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int n0 = blockIdx.x * 16;
  const int r = lane & 15, kc = (lane >> 4) * 8;
  const int M = (int)g.e.M;
  const int64_t kb = PART ? blockIdx.y * g.kper : 0;
  const int K = (int)(PART ? min(g.K - kb, g.kper) : g.K);   // of this split
  const int brows = min(16, g.e.N - n0);
  const int64_t b_bytes = ((int64_t)(brows - 1) * g.ldb + K) * 2;
  __amdgpu_buffer_rsrc_t b_rsrc[NB];
  b_rsrc[0] = make_rsrc(g.b + (int64_t)n0 * g.ldb + kb, b_bytes);
  if constexpr (GATED) b_rsrc[1] = make_rsrc(g.b + ((int64_t)g.e.N + n0) * g.ldb + kb, b_bytes);
  const __amdgpu_buffer_rsrc_t a_rsrc = make_rsrc(g.a + kb, ((int64_t)(M - 1) * g.lda + K) * 2);
  const uint32_t b_off = r < brows ? 2u * ((uint32_t)r * (uint32_t)g.ldb + kc) : kPastEnd;
  uint32_t a_off[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) a_off[i] = 16 * i + r < M ? 2u * ((uint32_t)(16 * i + r) * (uint32_t)g.lda + kc) : kPastEnd;
  f32x4 acc[NB][TT];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < TT; ++i) acc[b][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave * 32; k0 < K; k0 += kFewWaves * 32 * U) {
    v4u32 wv[U][NB], xv[U][TT];
#pragma unroll
    for (int s = 0; s < U; ++s) {
      const int k = k0 + s * kFewWaves * 32;
      const bool on = k + kc < K;      // a lane's 8 columns are whole or absent
#pragma unroll
      for (int b = 0; b < NB; ++b)
        wv[s][b] = __builtin_amdgcn_raw_buffer_load_b128(b_rsrc[b], (int)(on ? b_off + 2u * k : kPastEnd), 0, 0);
#pragma unroll
      for (int i = 0; i < TT; ++i)
        xv[s][i] = __builtin_amdgcn_raw_buffer_load_b128(a_rsrc, (int)(on && a_off[i] != kPastEnd ? a_off[i] + 2u * k : kPastEnd), 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);   // all of them, before the first is waited for
#pragma unroll
    for (int s = 0; s < U; ++s)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < TT; ++i)
          acc[b][i] = Elem<F16>::mfma16(__builtin_bit_cast(v8, wv[s][b]), __builtin_bit_cast(v8, xv[s][i]), acc[b][i]);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < TT; ++i) part[wave][b][i][lane] = make_float4(acc[b][i][0], acc[b][i][1], acc[b][i][2], acc[b][i][3]);
  __syncthreads();
  for (int i = wave; i < TT; i += kFewWaves) {
    float z[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
      const float4 x = part[w][0][i][lane];
      z[0] += x.x; z[1] += x.y; z[2] += x.z; z[3] += x.w;
      if constexpr (GATED) {
        const float4 y = part[w][NB - 1][i][lane];
        u[0] += y.x; u[1] += y.y; u[2] += y.z; u[3] += y.w;
      }
    }
    const int m = 16 * i + r, n = n0 + (lane >> 4) * 4;
    if (m >= M || n >= g.e.N) continue;
    if constexpr (PART) {
      float* to = g.part + ((int64_t)blockIdx.y * M + m) * g.pitch + n;
      store32(to, 4, z);
      if constexpr (GATED) store32(to + g.up_col, 4, u);
    } else {
      float bz[4], bu[4], res[4];
      load_bias<F16, GATED>(g.e, n, bz, bu);
      load_residual<F16>(g.e, m, n, res);
      finish<F16, GATED>(g.e, m, n, z, u, bz, bu, res);
    }
  }
}

// --- gradients: dz --------------------------------------------------------------

constexpr int kRangeBlocks = 1024;

struct DzArgs {
  const void* d_out;      // [M, N]
  const uint16_t* pre;    // [M, N or 2N]
  uint16_t* dz;           // [M, ldz] or null
  float* sums;            // [ceil(M / 64)][N or 2N] column sums of 64 rows each, or null
  float* range;           // [kRangeBlocks + 1] or null: largest finite |dz| of range_n workgroups; at kRangeBlocks
                          // the inverse of dz's factor
  int64_t M, ldd, ldp, ldz;
  int N, act, d_f32, range_n;
};

// dz of row m, columns n .. n + 7 (and the up columns' in the last half), zeros from `left` on
template <bool F16, int ACT, int HALVES>
__device__ __forceinline__ void form_dz(const DzArgs& a, int64_t m, int n, int left, float (&d)[HALVES][8]) {
  constexpr bool GATED = ACT == MOE_ACT_SWIGLU;
  float g[8] = {}, p[8] = {}, u[8] = {};
  if (left > 0) {
    if (a.d_f32) load32((const float*)a.d_out + m * a.ldd + n, left, g);
    else load16<F16>((const uint16_t*)a.d_out + m * a.ldd + n, left, g);
    if constexpr (ACT != MOE_ACT_NONE) load16<F16>(a.pre + m * a.ldp + n, left, p);
    if constexpr (GATED) load16<F16>(a.pre + m * a.ldp + a.N + n, left, u);
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    if constexpr (GATED) {
      d[0][c] = g[c] * u[c] * slope<MOE_ACT_SILU>(p[c]);
      d[HALVES - 1][c] = g[c] * activate<MOE_ACT_SILU>(p[c]);
    } else {
      d[0][c] = ACT == MOE_ACT_NONE ? g[c] : g[c] * slope<ACT>(p[c]);
    }
  }
}

// the largest of a workgroup's values, to all of its 256 threads
__device__ __forceinline__ float block_max(float v) {
  __shared__ float wave_max[4];
#pragma unroll
  for (int s = 32; s; s >>= 1) v = fmaxf(v, __shfl_xor(v, s));
  if (threadIdx.x % 64 == 0) wave_max[threadIdx.x / 64] = v;
  __syncthreads();
  return fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3]));
}

// The largest finite |dz| of each workgroup's 32 x 64 tiles, before an fp16 dz
// is formed: one more reading of d_out and pre, at HBM's rate (8192 x 2 x 2048 gated
// columns, 134 MB, 37 us of a backward pass's 955; 8192 x 256 from fp32 4.6 of 109).
template <int ACT>
__global__ __launch_bounds__(256) void dz_range_kernel(DzArgs a) {
  constexpr int HALVES = ACT == MOE_ACT_SWIGLU ? 2 : 1;
  const int tid = threadIdx.x, across = (a.N + 63) / 64;
  const int64_t tiles = (a.M + 31) / 32 * across;
  float top = 0.f;
  for (int64_t i = blockIdx.x; i < tiles; i += gridDim.x) {
    const int64_t m = i / across * 32 + tid / 8;
    const int n = (int)(i % across) * 64 + (tid % 8) * 8;
    if (m >= a.M) continue;
    float d[HALVES][8];
    form_dz<true, ACT>(a, m, n, a.N - n, d);
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float v = fabsf(d[h][c]);
        if (v < __builtin_inff()) top = fmaxf(top, v);
      }
  }
  top = block_max(top);
  if (tid == 0) a.range[blockIdx.x] = top;
}

// dz's factor from the workgroups' largest values: a power of two, at most
// 2^126 so that its inverse is a normal number
__device__ __forceinline__ float dz_factor(const DzArgs& a) {
  float top = 0.f;
  for (int i = threadIdx.x; i < a.range_n; i += 256) top = fmaxf(top, a.range[i]);
  top = block_max(top);
  const int e = (int)(__float_as_uint(top) >> 23) - 127;   // top in [2^e, 2^(e + 1)), or below 2^-126
  const int f = min(14 - e, 126);
  return top > 0.f ? __uint_as_float((uint32_t)(f + 127) << 23) : 1.0f;
}

// A thread forms 8 columns of two rows, 8 threads a row of 64 columns, so that
// each access covers whole lines; with SUMS the 64 x 64 columns of a workgroup
// are then added down in row order.  Columns past the last, up to ldz (a
// multiple of 8), become zeros.  Memory bound: 8192 x 2 x 2048
// gated columns, 168 MB, take 36 us, 4.7 TB/s.
template <bool F16, int ACT, bool SUMS>
__global__ __launch_bounds__(256) void dz_kernel(DzArgs a) {
  constexpr bool GATED = ACT == MOE_ACT_SWIGLU;
  constexpr int HALVES = GATED ? 2 : 1;
  __shared__ float tile[SUMS ? HALVES : 1][SUMS ? 32 : 1][SUMS ? 64 : 1];
  const int tid = threadIdx.x;
  const int n = (int)blockIdx.x * 64 + (tid % 8) * 8;
  const int left = a.N - n;
  float factor = 1.0f;
  if constexpr (F16) {
    if (a.range) {
      factor = dz_factor(a);
      if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) a.range[kRangeBlocks] = 1.0f / factor;
    }
  }
  float part[HALVES][8];
#pragma unroll
  for (int h = 0; h < HALVES; ++h)
#pragma unroll
    for (int c = 0; c < 8; ++c) part[h][c] = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = (int64_t)blockIdx.y * 64 + 32 * i + tid / 8;
    if (m >= a.M) continue;
    float d[HALVES][8];
    form_dz<F16, ACT>(a, m, n, left, d);
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        part[h][c] += d[h][c];
        if constexpr (F16) d[h][c] *= factor;
      }
    if (a.dz) {
      // the last half also writes the zeros behind it
      uint16_t* z = a.dz + m * a.ldz + n;
      if constexpr (GATED) {
        if (left > 0) store16<F16>(z, left, d[0]);
        const int room = (int)(a.ldz - a.N) - n;
        if (room > 0) store16<F16>(z + a.N, room, d[HALVES - 1]);
      } else {
        if (n < a.ldz) store16<F16>(z, 8, d[0]);
      }
    }
  }
  if constexpr (SUMS) {
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
#pragma unroll
      for (int c = 0; c < 8; ++c) tile[h][tid / 8][(tid % 8) * 8 + c] = part[h][c];
    __syncthreads();
    const int col = tid % 64, h = tid / 64;
    if (h < HALVES && (int)blockIdx.x * 64 + col < a.N) {
      float s = 0.f;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) s += tile[h][i][col];
      a.sums[blockIdx.y * (int64_t)HALVES * a.N + (int64_t)h * a.N + blockIdx.x * 64 + col] = s;
    }
  }
}

// bias gradient: the partial sums' rows added in a fixed order, four runs of
// them by four threads a column
template <bool F16>
__global__ __launch_bounds__(256) void bias_grad_kernel(const float* sums, int rows, int64_t cols, uint16_t* out) {
  __shared__ float run[4][64];
  const int64_t n = (int64_t)blockIdx.x * 64 + threadIdx.x % 64;
  const int q = threadIdx.x / 64, per = (rows + 3) / 4;
  float s = 0.f;
  if (n < cols) {
#pragma unroll 8
    for (int i = q * per; i < min(rows, (q + 1) * per); ++i) s += sums[i * cols + n];
  }
  run[q][threadIdx.x % 64] = s;
  __syncthreads();
  if (q == 0 && n < cols)
    out[n] = Elem<F16>::bits(run[0][threadIdx.x] + run[1][threadIdx.x] + run[2][threadIdx.x] + run[3][threadIdx.x]);
}

// --- host -------------------------------------------------------------------

int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// How a product is cut: tile 0 = few rows, 1 = 64 x 128, 2 = 128 x 128,
// 3 = 256 x 256, 4 = 128 x 256 (a gated product's columns count twice), and the
// splits of K.
struct Cut {
  int tile, splits;
  int64_t kper;
};

Cut choose_cut(int64_t M, int64_t N, int64_t K, bool gated, bool across) {
  const int64_t NZ = gated ? 2 * N : N;
  // few rows: 64 x 4096 x 4096 takes 22 us that way and 15 us in tiles, 32 rows 13 us either way
  if (M <= 32 && !across) {
    // A CU takes about 30 KB/us from the caches (64 lines in flight), so a few
    // workgroups with long sums are split along K, where that saves more than
    // the join's launch: 20 rows through 256 x 7168 18.1 us whole and 7.5 us in 8
    // splits, one row 10.8 and 6.7 us; 16 rows through 256 x 2048, below that,
    // 5.8 us whole and 6.2 us in 4 splits.
    const int64_t blocks = (N + 15) / 16, bytes = (16 * (gated ? 2 : 1) + M) * K * 2;
    int64_t s = 1;
    while (s < 8 && 2 * s * blocks <= kCus && K / (2 * s) >= 256) s *= 2;
    if ((double)bytes / 30e3 * (1.0 - 1.0 / s) < 3.9) s = 1;
    const int64_t kper = round_up((K + s - 1) / s, kBK);
    return {0, K > 0 ? (int)((K + kper - 1) / kper) : 1, kper};
  }
  // Time of each choice, the smallest wins.  A K step takes a load's latency, or
  // what the multiplications of the workgroups that share a CU take; a round of
  // workgroups adds its fill and epilogue; a split adds its partial sums' round
  // trip and the second launch.  The constants are fitted to times of every
  // choice over 228 products (forward, gated, dx and dw, 33 to 30000 rows,
  // operands not in a cache): the choice costs 1% over the best one on average.
  // Both sides of typical decisions:
  // 8192 x 256 x 7168 takes 49 us as 128 x 256 tiles in 4 splits, 54 us as
  // 128 x 128 in 4, 58 us as 256 x 256 in 8 and 62 us as 64 x 128 in 2;
  // 8192 x 2048 x 7168 takes 196 us as 256 x 256 in one piece and 224 us as
  // 128 x 256; 40 x 512 x 4096 takes 10.2 us as 64 x 128 in 16 splits, 14.5 us in 4.
  static const int bm[5] = {0, 64, 128, 256, 128}, bn[5] = {0, 128, 128, 256, 256};
  static const int per_cu[5] = {0, 3, 2, 1, 1};                       // workgroups of it a CU holds
  static const double latency[5] = {0, 0.564, 0.751, 1.327, 0.831};    // us a step
  static const double shared[5] = {0, 0.353, 0.51, 0, 0};             // ... and workgroup on the CU
  static const double round_us[5] = {0, 4.55, 4.76, 7.9, 5.7};
  static const int pieces[] = {1, 2, 3, 4, 6, 8, 12, 16, 32};
  const int64_t steps = (K + kBK - 1) / kBK;
  Cut best = {1, 1, round_up(K, kBK)};
  double best_us = 1e30;
  for (int t = 1; t <= 4; ++t) {
    int64_t tiles = ((M + bm[t] - 1) / bm[t]) * ((NZ + bn[t] - 1) / bn[t]);
    if (tiles < 1) tiles = 1;   // no rows: nothing to cut
    for (int s : pieces) {
      if (s > 1 && steps < 4 * s) break;
      const int64_t per = (steps + s - 1) / s;
      const int64_t blocks = tiles * s, slots = (int64_t)kCus * per_cu[t];
      const int64_t conc = blocks >= slots ? per_cu[t] : (blocks + kCus - 1) / kCus;
      const double work_us = conc * shared[t];
      const double step_us = work_us > latency[t] ? work_us : latency[t];
      double us = (double)((blocks + kCus * conc - 1) / (kCus * conc)) * (per * step_us + round_us[t]);
      if (s > 1) us += 2.2 + 0.047 * s + (double)s * M * NZ * 8 / 5.58e6;
      if (us < best_us) {
        best_us = us;
        best = {t, s, per * kBK};
      }
    }
  }
  best.splits = K > 0 ? (int)((K + best.kper - 1) / best.kper) : 1;
  return best;
}

size_t part_bytes(const Cut& c, int64_t M, int64_t N, bool gated) {
  return c.splits > 1 ? (size_t)c.splits * M * round_up(N, 4) * (gated ? 2 : 1) * 4 : 0;
}

template <bool F16, int ACT>
void launch_dz_act(const DzArgs& a, const dim3& grid, hipStream_t s) {
  if constexpr (F16)
    if (a.range) hipLaunchKernelGGL((dz_range_kernel<ACT>), dim3((unsigned)a.range_n), dim3(256), 0, s, a);
  if (a.sums) hipLaunchKernelGGL((dz_kernel<F16, ACT, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((dz_kernel<F16, ACT, false>), grid, dim3(256), 0, s, a);
}
template <bool F16>
void launch_dz(const DzArgs& a, hipStream_t s) {
  // the up half's columns may start anywhere, and so end up to 7 past N
  const int cols = a.N + (a.act == MOE_ACT_SWIGLU ? 7 : 0);
  const dim3 grid((unsigned)((cols + 63) / 64), (unsigned)((a.M + 63) / 64));
  switch (a.act) {
    case MOE_ACT_RELU: launch_dz_act<F16, MOE_ACT_RELU>(a, grid, s); break;
    case MOE_ACT_SILU: launch_dz_act<F16, MOE_ACT_SILU>(a, grid, s); break;
    case MOE_ACT_GELU: launch_dz_act<F16, MOE_ACT_GELU>(a, grid, s); break;
    case MOE_ACT_GELU_TANH: launch_dz_act<F16, MOE_ACT_GELU_TANH>(a, grid, s); break;
    case MOE_ACT_SWIGLU: launch_dz_act<F16, MOE_ACT_SWIGLU>(a, grid, s); break;
    default: launch_dz_act<F16, MOE_ACT_NONE>(a, grid, s); break;
  }
}

template <bool F16, bool GATED>
void launch_join(const ProdArgs& g, hipStream_t s) {
  const int64_t blocks = (g.e.M * ((g.e.N + 3) / 4) + 63) / 64;
  hipLaunchKernelGGL((join_kernel<F16, GATED>), dim3((unsigned)(blocks < 32768 ? blocks : 32768)), dim3(64), 0, s, g);
}

template <class C, bool F16, bool GATED, bool AX, bool BX>
void launch_tiles(ProdArgs& g, hipStream_t s) {
  constexpr int HB = GATED ? C::BN / 2 : C::BN;
  g.n_mt = (int)((g.e.M + C::BM - 1) / C::BM);
  g.n_nt = (g.e.N + HB - 1) / HB;
  const unsigned grid = (unsigned)((int64_t)g.n_mt * g.n_nt * g.splits);
  if (g.splits == 1) {
    hipLaunchKernelGGL((product_kernel<C, F16, GATED, false, AX, BX>), dim3(grid), dim3(C::NT), 0, s, g);
    return;
  }
  hipLaunchKernelGGL((product_kernel<C, F16, GATED, true, AX, BX>), dim3(grid), dim3(C::NT), 0, s, g);
  launch_join<F16, GATED>(g, s);
}

template <bool F16, bool GATED, bool AX, bool BX>
hipError_t launch_product(ProdArgs& g, const Cut& c, void* ws, hipStream_t s) {
  if (g.e.M == 0) return hipSuccess;
  g.kper = c.kper;
  g.splits = c.splits;
  g.part = (float*)ws;
  g.up_col = (int)round_up(g.e.N, 4);
  g.pitch = (int64_t)g.up_col * (GATED ? 2 : 1);
  if (c.tile == 0) {
    if constexpr (!AX && !BX) {
      const dim3 grid((unsigned)((g.e.N + 15) / 16), (unsigned)g.splits), block(kFewWaves * 64);
      // More loads in flight for longer sums, as the registers allow (16 K steps'
      // instead of 8: one row, 4096 x 4096 7.6 instead of 8.6 us, 7168 x 2048
      // unchanged and without their masked loads).
      auto go = [&](auto tt, auto part) {
        constexpr int TT = decltype(tt)::value, D = TT + (GATED ? 2 : 1) > 2 ? 2 : 1;
        constexpr bool P = decltype(part)::value;
        if (g.kper > 2048) hipLaunchKernelGGL((few_rows_kernel<TT, F16, GATED, P, 16 / D>), grid, block, 0, s, g);
        else hipLaunchKernelGGL((few_rows_kernel<TT, F16, GATED, P, 8 / D>), grid, block, 0, s, g);
      };
      using One = std::integral_constant<int, 1>;
      using Two = std::integral_constant<int, 2>;
      if (g.splits == 1) {
        if (g.e.M <= 16) go(One{}, std::false_type{});
        else go(Two{}, std::false_type{});
      } else {
        if (g.e.M <= 16) go(One{}, std::true_type{});
        else go(Two{}, std::true_type{});
        launch_join<F16, GATED>(g, s);
      }
    }
  } else if (c.tile == 1) {
    launch_tiles<Tile64, F16, GATED, AX, BX>(g, s);
  } else if (c.tile == 2) {
    launch_tiles<Tile128, F16, GATED, AX, BX>(g, s);
  } else if (c.tile == 4) {
    launch_tiles<TileWide, F16, GATED, AX, BX>(g, s);
  } else {
    launch_tiles<std::conditional_t<GATED, Tile256G, Tile256>, F16, GATED, AX, BX>(g, s);
  }
  return hipGetLastError();
}

bool gated(const moe_linear_desc& d) { return d.act == MOE_ACT_SWIGLU; }

// Workspace of the backward pass, in bytes (pieces 256-byte aligned).
struct BackLayout {
  int64_t NZ, ldz, sums_rows;
  Cut dx, dw;
  bool scaled;   // dz is rounded to fp16 (without an activation a 16-bit d_out is copied at most)
  size_t dz, sums, part, range, total;
};
BackLayout back_layout(const moe_linear_desc& d) {
  BackLayout L;
  L.NZ = (int64_t)d.cols * (gated(d) ? 2 : 1);
  L.ldz = round_up(L.NZ, 8);
  L.sums_rows = (d.rows + 63) / 64;
  L.dx = choose_cut(d.rows, d.depth, L.ldz, false, true);
  L.dw = choose_cut(L.NZ, d.depth, d.rows, false, true);
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off += (size_t)round_up((int64_t)n, 256);
    return at;
  };
  L.dz = take((size_t)d.rows * L.ldz * 2);
  L.sums = take((size_t)L.sums_rows * L.NZ * 4);
  const size_t p1 = part_bytes(L.dx, d.rows, d.depth, false), p2 = part_bytes(L.dw, L.NZ, d.depth, false);
  L.part = take(p1 > p2 ? p1 : p2);
  L.scaled = d.dtype == MOE_F16 && (d.act != MOE_ACT_NONE || d.out_dtype == MOE_F32);
  L.range = take(L.scaled ? (kRangeBlocks + 1) * sizeof(float) : 0);
  L.total = off > 256 ? off : 256;
  return L;
}

}  // namespace

size_t linear_ws_bytes(const moe_linear_desc& d) {
  return part_bytes(choose_cut(d.rows, d.cols, d.depth, gated(d), false), d.rows, d.cols, gated(d));
}

size_t linear_back_ws_bytes(const moe_linear_desc& d) { return back_layout(d).total; }

void linear_cuts(const moe_linear_desc& d, int32_t cuts[6]) {
  const BackLayout L = back_layout(d);
  const Cut all[3] = {choose_cut(d.rows, d.cols, d.depth, gated(d), false), L.dx, L.dw};
  for (int i = 0; i < 3; ++i) {
    cuts[2 * i] = all[i].tile;
    cuts[2 * i + 1] = all[i].splits;
  }
}

hipError_t launch_linear(const moe_linear_desc& d, const LinearBuffers& b, void* ws, hipStream_t s) {
  ProdArgs g;
  g.a = (const uint16_t*)b.x;
  g.b = (const uint16_t*)b.w;
  g.lda = d.ld_x;
  g.ldb = d.ld_w;
  g.K = d.depth;
  Epilogue& e = g.e;
  e.bias = (const uint16_t*)b.bias;
  e.res = b.residual;
  e.pre = (uint16_t*)b.pre;
  e.out = b.out;
  e.M = d.rows; e.N = d.cols;
  e.ldr = d.ld_residual; e.ldp = d.ld_pre; e.ldo = d.ld_out;
  e.act = d.act;
  e.out_f32 = d.out_dtype == MOE_F32;
  e.scale = nullptr;
  const Cut c = choose_cut(d.rows, d.cols, d.depth, gated(d), false);
  if (d.dtype == MOE_F16)
    return gated(d) ? launch_product<true, true, false, false>(g, c, ws, s) : launch_product<true, false, false, false>(g, c, ws, s);
  return gated(d) ? launch_product<false, true, false, false>(g, c, ws, s) : launch_product<false, false, false, false>(g, c, ws, s);
}

hipError_t launch_linear_backward(const moe_linear_desc& d, const LinearGrads& b, void* ws, hipStream_t s) {
  const BackLayout L = back_layout(d);
  char* base = (char*)ws;
  const bool f16 = d.dtype == MOE_F16, f32 = d.out_dtype == MOE_F32;
  uint16_t* dz = (uint16_t*)(base + L.dz);
  // without an activation the incoming gradient can be the operand itself
  const bool direct = d.act == MOE_ACT_NONE && !f32 && d.cols % 8 == 0 && d.ld_out % 8 == 0 && aligned_to(b.d_out, 16);
  const bool want_dz = (b.dx || b.dw) && !direct;
  float* range = L.scaled && want_dz && d.rows > 0 ? (float*)(base + L.range) : nullptr;
  if (d.rows > 0 && (want_dz || b.dbias)) {
    DzArgs a;
    a.d_out = b.d_out;
    a.pre = (const uint16_t*)b.pre;
    a.dz = want_dz ? dz : nullptr;
    a.sums = b.dbias ? (float*)(base + L.sums) : nullptr;
    a.M = d.rows; a.N = d.cols;
    a.ldd = d.ld_out; a.ldp = d.ld_pre; a.ldz = L.ldz;
    a.act = d.act;
    a.d_f32 = f32;
    a.range = range;
    const int64_t tiles = (d.rows + 31) / 32 * ((d.cols + 63) / 64);
    a.range_n = (int)(tiles < kRangeBlocks ? tiles : kRangeBlocks);
    if (f16) launch_dz<true>(a, s);
    else launch_dz<false>(a, s);
  }
  if (b.dbias) {
    const dim3 grid((unsigned)((L.NZ + 63) / 64));
    const float* sums = (const float*)(base + L.sums);
    if (f16) hipLaunchKernelGGL((bias_grad_kernel<true>), grid, dim3(256), 0, s, sums, (int)L.sums_rows, L.NZ, (uint16_t*)b.dbias);
    else hipLaunchKernelGGL((bias_grad_kernel<false>), grid, dim3(256), 0, s, sums, (int)L.sums_rows, L.NZ, (uint16_t*)b.dbias);
  }
  hipError_t rc = hipGetLastError();
  if (rc != hipSuccess) return rc;
  ProdArgs g;
  Epilogue& e = g.e;
  e.bias = nullptr; e.res = nullptr; e.pre = nullptr;
  e.ldr = e.ldp = 0;
  e.act = MOE_ACT_NONE;
  e.out_f32 = 0;
  e.scale = range ? range + kRangeBlocks : nullptr;
  e.N = d.depth;
  g.a = direct ? (const uint16_t*)b.d_out : dz;
  g.lda = direct ? d.ld_out : L.ldz;
  if (b.dx && d.rows > 0) {
    // dx [rows, depth]: dz along its columns, w [n, depth] across them.  dz's
    // zero columns up to a multiple of 8 meet rows past w's end, also zeros.
    g.b = (const uint16_t*)b.w;
    g.ldb = d.ld_w;
    g.K = L.NZ;
    e.M = d.rows;
    e.out = b.dx;
    e.ldo = d.ld_dx;
    rc = f16 ? launch_product<true, false, false, true>(g, L.dx, base + L.part, s)
             : launch_product<false, false, false, true>(g, L.dx, base + L.part, s);
    if (rc != hipSuccess) return rc;
  }
  if (b.dw) {
    // dw [n, depth]: both operands across the rows that are summed over
    g.b = (const uint16_t*)b.x;
    g.ldb = d.ld_x;
    g.K = d.rows;
    e.M = L.NZ;
    e.out = b.dw;
    e.ldo = d.ld_dw;
    rc = f16 ? launch_product<true, false, true, true>(g, L.dw, base + L.part, s)
             : launch_product<false, false, true, true>(g, L.dw, base + L.part, s);
  }
  return rc;
}

}  // namespace moe
