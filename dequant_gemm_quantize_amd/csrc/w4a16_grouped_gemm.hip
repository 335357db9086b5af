// W4A16 product by expert for many rows an expert, bf16 x:
//   y[t, n] = sum_k x[t, k] (q[e, n, k] - zp) s   for the expert e of row t
// on v_mfma_f32_32x32x16_bf16 with float32 accumulation.
//
// bf16 y takes the weight rounded once to bf16, as w4a16_matmul does: that
// adds as much to the error as the rounding of y (2^-9 of the value, in the
// mean over K terms).  float32 y takes it as the sum of two bf16 values, the
// second the first's rounding error, and twice the MFMAs: with fp16 scales
// (4 + 11 significant bits) the two hold the weight exactly.
//
// Workgroup tile BM rows x 128 NJ columns, four waves, each all BM rows of 32 NJ
// columns: no two waves dequantize the same weight, and a wave's accumulators
// (8 x 2 blocks at BM = 256) are reused against 64 KB of LDS reads a K step
// of 64 columns, which is half of what LDS gives in the step's MFMA time.
// x goes from memory to LDS directly, S stages of 64 columns (128-byte
// lines); the packed weights the same way, two stages of 256 columns (again
// 128-byte lines), and from there to registers, where each wave turns its own
// 64 rows into bf16 operands.  Lane (r, h) of an operand holds row r; of the
// step's 64 columns it has the 32 that its half h reads as one 16-byte piece
// of codes, the same permutation of K on both operands.
//
// Bound by the wave's own instructions: 4.9 vector instructions an MFMA leave
// the matrix cores busy 48% of the time, at one wave a SIMD, and no other order
// of conversions and MFMAs did better (372 - 381 us all).  4096 rows of 8
// experts [11008, 4096] 375 us (0.98 PFLOP/s); a large bf16 product of the
// library reaches 1.53.  1024 rows 137 us.
#include <type_traits>

#include "grouped.h"
#include "lds_gemm.h"
#include "w4_common.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int GLine = 128;        // bytes of a row per stage: 64 bf16 or 256 codes

template <typename TS> struct GScale;
template <> struct GScale<_Float16> {
  __device__ static _Float16 load(__amdgpu_buffer_rsrc_t r, uint32_t i) {
    return __builtin_bit_cast(_Float16, (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, 2 * i, 0, 0));
  }
};
template <> struct GScale<float> {
  __device__ static float load(__amdgpu_buffer_rsrc_t r, uint32_t i) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, 4 * i, 0, 0));
  }
};

// 8 codes -> 8 weights in column order, fma(q, s, b) with b = -zp s (exact
// with fp16 scales); hi rounded to bf16, lo the bf16 of what hi lacks.
template <bool SPLIT>
__device__ __forceinline__ void dequant_pairs(uint32_t p, float s, float b, u32x4& hi, u32x4& lo) {
  uint32_t even = p & 0x0f0f0f0fu, odd = (p >> 4) & 0x0f0f0f0fu;
  // opaque to the optimizer, so that each byte converts in place
  asm("" : "+v"(even), "+v"(odd));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float w0 = fmaf((float)((even >> (8 * i)) & 0xffu), s, b);
    const float w1 = fmaf((float)((odd >> (8 * i)) & 0xffu), s, b);
    const uint32_t v = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)w0, (__bf16)w1});
    hi[i] = v;
    if constexpr (SPLIT)
      lo[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)(w0 - bf16_lo(v)), (__bf16)(w1 - bf16_hi(v))});
  }
}

template <int BM, int NJ, int S> constexpr size_t gg_lds() { return (size_t)(S * BM + 2 * 128 * NJ) * GLine; }

}  // namespace

// One tile: rows m0 .. min(m0 + BM, mend) - 1 of y, columns from n0, for the
// expert whose first weight row is ebase.  S: stages of x.  G128: g % 128 == 0, so two steps of
// a stage share a scale.
template <int BM, int NJ, int S, typename TS, typename TY, bool G128>
__device__ __forceinline__ void gg_tile(uint8_t* sgg, int lane, int w, const uint16_t* __restrict__ x, int64_t K,
                                        const uint8_t* __restrict__ packed, const void* __restrict__ scales,
                                        const void* __restrict__ zeros, int64_t N, int g, TY* __restrict__ y, int64_t m0,
                                        int64_t mend, int64_t n0, int64_t ebase) {
  constexpr bool SPLIT = sizeof(TY) == 4;
  constexpr int GBN = 128 * NJ, MI = BM / 32, LA = BM / 32, LW = GBN / 32;
  constexpr int A_STAGE = BM * GLine, W_STAGE = GBN * GLine;
  const uint32_t xrow = (uint32_t)(2 * K), wrow = (uint32_t)(K / 2), ng = (uint32_t)(K / g);
  const uint32_t mrows = (uint32_t)(mend - m0 < BM ? mend - m0 : BM);
  const uint32_t nrows = (uint32_t)(N - n0 < GBN ? N - n0 : GBN);
  // rows past the tile's are past the resource and read as zero
  const __amdgpu_buffer_rsrc_t xr = buf_rsrc_n(uniform_ptr(x + m0 * K), mrows * xrow);
  const __amdgpu_buffer_rsrc_t wr = buf_rsrc_n(uniform_ptr(packed + (ebase + n0) * wrow), nrows * wrow);
  const __amdgpu_buffer_rsrc_t sr =
      buf_rsrc_n(uniform_ptr((const char*)scales + (ebase + n0) * ng * sizeof(TS)), nrows * ng * (uint32_t)sizeof(TS));
  const __amdgpu_buffer_rsrc_t zr =
      buf_rsrc_n(uniform_ptr((const char*)zeros + (ebase + n0) * ng * sizeof(TS)), nrows * ng * (uint32_t)sizeof(TS));

  // memory -> LDS, 8 rows x 128 bytes a load; slot s of row r holds chunk s ^ ((r / 2) % 8)
  const int lrow = lane >> 3, slot = lane & 7;
  uint32_t xo[LA], wo[LW];
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int row = 8 * (w * LA + i) + lrow;
    xo[i] = (uint32_t)row * xrow + 16u * (slot ^ ((row >> 1) & 7));
  }
#pragma unroll
  for (int i = 0; i < LW; ++i) {
    const int row = 8 * (w * LW + i) + lrow;
    wo[i] = (uint32_t)row * wrow + 16u * (slot ^ ((row >> 1) & 7));
  }
  const int nks = (int)(K / 64);
  uint8_t* sw = sgg + S * A_STAGE;
  // steps and stages past the last lie outside the resources
  auto x_issue = [&](int ks) {
    const uint32_t o = ks < nks ? (uint32_t)ks * GLine : kPastEnd;
#pragma unroll
    for (int i = 0; i < LA; ++i) load_lds(xr, sgg + ks % S * A_STAGE + 1024 * (w * LA + i), xo[i] + o);
  };
  auto w_issue = [&](int st) {
    const uint32_t o = 4 * st < nks ? (uint32_t)st * GLine : kPastEnd;
#pragma unroll
    for (int i = 0; i < LW; ++i) load_lds(wr, sw + (st & 1) * W_STAGE + 1024 * (w * LW + i), wo[i] + o);
  };

  // scales of the lane's two weight rows for the four steps of a stage: step
  // u, half h has 32-column block 8 st + 2 u + h
  const int r = lane & 31, h = lane >> 5;
  const int n_lane = 32 * NJ * w + r;
  const uint32_t bpg = (uint32_t)g / 32;
  constexpr int NS = G128 ? 2 : 4;
  TS sv[NJ][NS], zv[NJ][NS], snext[NJ][NS], znext[NJ][NS];
  auto s_issue = [&](int st) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int u = 0; u < NS; ++u) {
        const uint32_t blk = 8u * st + (G128 ? 4u * u : 2u * u + h);
        const uint32_t gi = blk / bpg;  // past the row's last group only for steps that do not run
        const uint32_t at = gi < ng ? (uint32_t)(n_lane + 32 * j) * ng + gi : kPastEnd / sizeof(TS);
        snext[j][u] = GScale<TS>::load(sr, at);
        znext[j][u] = GScale<TS>::load(zr, at);
      }
  };
  auto s_take = [&]() {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int u = 0; u < NS; ++u) sv[j][u] = snext[j][u], zv[j][u] = znext[j][u];
  };

  f32x16 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  const int swz = (r >> 1) & 7;
  int fo[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) fo[t] = r * GLine + 16 * ((4 * h + t) ^ swz);
  // x of K slice t (16 columns: chunk 4 h + t of the line)
  u32x4 xv[2][MI];
  auto x_frag = [&](int ks, auto tc) {
    constexpr int t = decltype(tc)::value;
    const uint8_t* a = sgg + ks % S * A_STAGE + fo[t];
#pragma unroll
    for (int i = 0; i < MI; ++i) xv[t & 1][i] = *(const u32x4*)(a + 32 * GLine * i);
  };
  // the step's codes: chunk 2 u + h of the weight line
  u32x4 cv[NJ], cnext[NJ];
  auto codes = [&](int st, int u) {
    const uint8_t* b = sw + (st & 1) * W_STAGE + (32 * NJ * w + r) * GLine + 16 * ((2 * u + h) ^ swz);
#pragma unroll
    for (int j = 0; j < NJ; ++j) cnext[j] = *(const u32x4*)(b + 32 * GLine * j);
  };
  auto c_take = [&]() {
#pragma unroll
    for (int j = 0; j < NJ; ++j) cv[j] = cnext[j];
  };
  // weights of a slice, in two register sets; slice t of step u
  u32x4 whi[2][NJ], wlo[2][NJ];
  auto dequant = [&](auto tc, auto uc) {
    constexpr int t = decltype(tc)::value, u = decltype(uc)::value;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const float s = (float)sv[j][G128 ? u / 2 : u], b = -(float)zv[j][G128 ? u / 2 : u] * s;
      dequant_pairs<SPLIT>(cv[j][t], s, b, whi[t & 1][j], wlo[t & 1][j]);
    }
  };
  auto mma = [&](auto tc) {
    constexpr int t = decltype(tc)::value;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, whi[t & 1][j]),
                                                            __builtin_bit_cast(bf16x8, xv[t & 1][i]), acc[i][j], 0, 0, 0);
        if constexpr (SPLIT)
          acc[i][j] =
              __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, wlo[t & 1][j]),
                                                      __builtin_bit_cast(bf16x8, xv[t & 1][i]), acc[i][j], 0, 0, 0);
      }
  };
  // an LDS read and some of the next slice's conversions after each MFMA
  auto mix = [&]() {
#pragma unroll
    for (int i = 0; i < MI * NJ; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, SPLIT ? 2 : 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, (SPLIT ? 100 : 52) / (MI * NJ) + 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};
  constexpr std::integral_constant<int, 2> c2{};
  constexpr std::integral_constant<int, 3> c3{};

  s_issue(0);
  w_issue(0);
#pragma unroll
  for (int p = 0; p < S; ++p) x_issue(p);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 1) * LA) : "memory");  // all but the x of the steps behind the first
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  s_take();
  codes(0, 0);
  c_take();
  x_frag(0, c0);
  dequant(c0, c0);

  // One K step of 64 columns, four slices.  A slice's x reads and conversions
  // run under the MFMAs of the one before.  Before the last slice every wave
  // has read all of the step's x and waited for its share of the next step's;
  // behind the barrier that is whole and this step's x stage is free.  The
  // next step's codes are read a slice earlier still: their stage has been
  // whole since the barrier of u = 2.  The wait leaves the x of S - 2 further
  // steps on its way, and behind the barrier of u = 0 also the weights issued
  // there (they are older than what the other waits leave).  A step of 64-row
  // tiles is too short for a load: four stages there took 777 rows of 16
  // experts [2050, 2048], bf16 y, from 39 to 35 us.  Larger tiles wait for their
  // conversions, and more stages would cost the second workgroup of a CU
  // (1024 rows of 8 experts [11008, 4096]: two stages 135 us, three 143, four 162).
  auto step = [&](int ks, auto uc) {
    constexpr int u = decltype(uc)::value;
    x_frag(ks, c1);
    dequant(c1, uc);
    mma(c0);
    mix();
    x_frag(ks, c2);
    codes((ks + 1) / 4, (u + 1) & 3);
    dequant(c2, uc);
    mma(c1);
    mix();
    x_frag(ks, c3);
    dequant(c3, uc);
    mma(c2);
    mix();
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((S - 2) * LA + (u == 1 && S > 2 ? LW : 0)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if constexpr (u == 0) w_issue(ks / 4 + 1);
    if constexpr (u == 1) s_issue(ks / 4 + 1);
    if constexpr (u == 3) s_take();
    x_issue(ks + S);
    c_take();
    x_frag(ks + 1, c0);
    dequant(c0, std::integral_constant<int, (u + 1) & 3>{});
    mma(c3);
    __builtin_amdgcn_sched_barrier(0);
  };
  int ks = 0;
  for (; ks + 4 <= nks; ks += 4) {
    step(ks, c0);
    step(ks + 1, c1);
    step(ks + 2, c2);
    step(ks + 3, c3);
  }
  if (ks < nks) {
    step(ks, c0);
    if (ks + 1 < nks) {
      step(ks + 1, c1);
      if (ks + 2 < nks) step(ks + 2, c2);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may reach LDS after the workgroup has left it
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  constexpr int TURN = turn_bytes<TY, NJ>();
  static_assert(4 * TURN <= (int)gg_lds<BM, NJ, S>(), "the waves' turning places fit in LDS");
  turn_store<TY, MI, NJ>(sgg + w * TURN, lane, acc, y, N, m0, mend, n0 + 32 * NJ * w);
}

// (LDS holds two workgroups of 64-row tiles; registers for three were 4%
// faster than the compiler's larger use of them.)
template <int BM, int NJ, int S, typename TS, typename TY, bool G128>
__global__ __launch_bounds__(256, BM == 256 ? 1 : BM == 64 ? 3 : 2) void k_w4a16_grouped_gemm(
    const uint16_t* __restrict__ x, int64_t T, int64_t K, const int* __restrict__ offsets, int experts,
    const uint8_t* __restrict__ packed, const void* __restrict__ scales, const void* __restrict__ zeros, int64_t N,
    int g, TY* __restrict__ y, uint32_t tiles_n) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t sgg[];  // x stages, then weight stages
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  int64_t m0, mend, n0;
  int64_t ebase;  // the expert's first weight row
  int half;
  {
    const uint32_t total = (uint32_t)grouped_tiles(offsets, experts, (int)T, BM, lane) * tiles_n;
    uint32_t t;
    if (!xcd_tile<32, BM == 256>(total, t, half)) return;
    GroupTile gt;
    if (!find_group_tile(offsets, experts, (int)T, BM, tiles_n, t, lane, gt)) return;
    uint32_t tm, tn;
    band(gt.tile, (uint32_t)(gt.rows + BM - 1) / BM, tiles_n, tm, tn);
    m0 = gt.row0 + (int64_t)BM * tm;
    n0 = (int64_t)128 * NJ * tn;
    mend = gt.row0 + gt.rows;
    ebase = (int64_t)gt.expert * N;
  }
  if (half == 0 && mend > m0 + BM / 2) mend = m0 + BM / 2;
  if (half == 1) {
    m0 += BM / 2;
    if (m0 >= mend) return;
  }
  // half a tile, or one with rows in its upper half only, takes half the time
  if constexpr (BM > 64) {
    if (half >= 0 || mend - m0 <= BM / 2) {
      gg_tile<BM / 2, NJ, S, TS, TY, G128>(sgg, lane, w, x, K, packed, scales, zeros, N, g, y, m0, mend, n0, ebase);
      return;
    }
  }
  gg_tile<BM, NJ, S, TS, TY, G128>(sgg, lane, w, x, K, packed, scales, zeros, N, g, y, m0, mend, n0, ebase);
}

// K % 64 == 0: whole steps; 256 rows of K bf16 stay below 2^31 bytes.
bool w4a16_grouped_gemm_fits(int64_t k) { return k % 64 == 0 && k <= ((int64_t)1 << 21); }

template <int BM, int NJ, int S, typename TS, typename TY, bool G128>
static hipError_t gg_go(const uint16_t* x, int64_t t, int64_t k, const int* offsets, int experts,
                        const uint8_t* packed, const void* scales, const void* zeros, int64_t n, int g, void* y,
                        hipStream_t st) {
  static std::atomic<uint64_t> attr_done{0};  // LDS above the 64 KB default
  const hipError_t e = once_per_device(attr_done, [] {
    return hipFuncSetAttribute((const void*)k_w4a16_grouped_gemm<BM, NJ, S, TS, TY, G128>,
                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)gg_lds<BM, NJ, S>());
  });
  if (e != hipSuccess) return e;
  const int64_t tiles_n = (n + 128 * NJ - 1) / (128 * NJ);
  const int64_t grid = xcd_grid<32, BM == 256>(grouped_max_tiles(t, experts, BM) * tiles_n);
  k_w4a16_grouped_gemm<BM, NJ, S, TS, TY, G128><<<dim3((unsigned)grid), 256, gg_lds<BM, NJ, S>(), st>>>(
      x, t, k, offsets, experts, packed, scales, zeros, n, g, (TY*)y, (uint32_t)tiles_n);
  return hipGetLastError();
}

template <typename TS, typename TY, bool G128>
static hipError_t gg_size(const uint16_t* x, int64_t t, int64_t k, const int* offsets, int experts,
                          const uint8_t* packed, const void* scales, const void* zeros, int64_t n, int g, void* y,
                          hipStream_t st) {
  // Experts [11008, 4096], 8 of them, us with 256 x 256 / 128 x 128 / 64 x 128
  // tiles (each with two stages of x): 2048 rows 205 / 235 / 271, 1024 rows 198 /
  // 136 / 162, 512 rows 180 / 112 / 100, 256 rows 179 / 99 / 74.  (A launch has fewer than 2^32 threads,
  // which the smallest tiles of the largest calls could exceed.)
  if (t > 192 * (int64_t)experts)
    return gg_go<256, 2, 2, TS, TY, G128>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  const bool too_many = grouped_max_tiles(t, experts, 64) * ((n + 127) / 128) >= (1 << 24) - 8;
  if (t > 80 * (int64_t)experts || too_many)
    return gg_go<128, 1, 2, TS, TY, G128>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  return gg_go<64, 1, 4, TS, TY, G128>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
}

template <typename TS, typename TY>
static hipError_t gg_pick(const uint16_t* x, int64_t t, int64_t k, const int* offsets, int experts,
                          const uint8_t* packed, const void* scales, const void* zeros, int64_t n, int g, void* y,
                          hipStream_t st) {
  if (g % 128 == 0) return gg_size<TS, TY, true>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  return gg_size<TS, TY, false>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
}

hipError_t launch_w4a16_grouped_gemm(const void* x, int64_t t, int64_t k, const int* offsets, int experts,
                                     const uint8_t* packed, const void* scales, const void* zeros, int sz_dtype,
                                     int64_t n, int g, void* y, int y_dtype, hipStream_t st) {
  const uint16_t* xb = (const uint16_t*)x;
  if (sz_dtype == W4_F16) {
    if (y_dtype == W4_F32)
      return gg_pick<_Float16, float>(xb, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
    return gg_pick<_Float16, __bf16>(xb, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  }
  if (y_dtype == W4_F32)
    return gg_pick<float, float>(xb, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  return gg_pick<float, __bf16>(xb, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
}

}  // namespace w4
