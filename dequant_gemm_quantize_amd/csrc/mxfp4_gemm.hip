// MXFP4 product for many rows, dense or by expert:
//   y[m, n] = sum over blocks b of 2^(xs + ws - 254) * sum_{k in b} xv wv
// on v_mfma_scale_f32_32x32x64_f8f6f4: lane (r = lane % 32, h = lane / 32) holds
// 16 bytes (one block of 32 columns) of row r of each operand and that
// block's scale byte, so the scales cost no instruction of their own.
//
// Bound by three things that lie close together.  The operands of an FP4 MFMA
// (2 KB, 32 cycles) take LDS twice as long as a CU's four MFMAs if each is read
// for one alone, so a wave has a large block of outputs (128 x 128 of the
// workgroup's 256 x 256, 256 accumulators a lane): LDS is then busy half of the
// MFMAs' time.  The matrix cores on real data are held back by power (a loop
// of nothing but these MFMAs reaches 6.6 - 7.2 PFLOP/s on random codes and over
// 9 on zeros).  And the tiles come from L2, 64 KB a K step and CU, which takes
// about a step's time and has to be asked for one and a half steps ahead.  y
// is a third of the bytes at K = 4096.
// Measured, kernel time: 512 x 28672 x 8192 64 us (3.7 PFLOP/s), 2048 x 11008 x
// 4096 57 us (3.2); 4096 rows by expert, 8 of [11008, 4096], 130 us (2.8: the
// experts' last tiles); 4096 x 8192 x 8192 136 us a call in a replayed graph (4.1).
// Matrix cores are busy a third of that time.
#include <type_traits>

#include "grouped.h"
#include "lds_gemm.h"
#include "w4_common.h"
#include "w4_internal.h"

namespace w4 {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStepBytes = 128;  // a K step: 256 columns, one 128-byte line of a row

__device__ __forceinline__ i32x8 mx_operand(u32x4 v) {
  return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

template <int J>
__device__ __forceinline__ f32x16 mx_mfma(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, J, (int)sa, J, (int)sb);
}

// Workgroup tile BM x BN of WR x WC waves, each 32 MI x 32 NJ outputs.
template <int BM_, int BN_, int WR_, int WC_, int S_> struct MxTile {
  static constexpr int BM = BM_, BN = BN_, WR = WR_, WC = WC_, S = S_;
  static constexpr int NW = WR * WC, NT = 64 * NW;
  static constexpr int MI = BM / (32 * WR), NJ = BN / (32 * WC);
  static constexpr int LA = BM / (8 * NW), LB = BN / (8 * NW);  // 1 KB loads per wave and step
  static constexpr int A_STAGE = BM * kStepBytes, B_STAGE = BN * kStepBytes, STAGE = A_STAGE + B_STAGE;
  static constexpr size_t lds = (size_t)S * STAGE;
  typedef MxTile<BM / 2, BN, WR, WC, S> Half;
  static constexpr uint32_t SLOTS = 2 * lds <= 163840 ? 64 : 32;  // workgroups an XCD holds (160 KB of LDS a CU)
  // Halves of small tiles cost more than they give: with few rows the second
  // one is often empty and the weights are read twice (256 rows of 8 experts
  // [11008, 4096] 46 us without, 51 with).
  static constexpr bool SPLIT = BM == 256;
};

}  // namespace

// One tile: rows m0 .. min(m0 + BM, mend) - 1 of y, columns from n0.
template <typename T, typename TY>
__device__ __forceinline__ void mx_tile(uint8_t* smx, int lane, int w, const uint8_t* __restrict__ xq,
                                        const uint8_t* __restrict__ xs, int64_t K, const uint8_t* __restrict__ wp,
                                        const uint8_t* __restrict__ sp, int64_t N, TY* __restrict__ y, int64_t m0,
                                        int64_t mend, int64_t n0) {
  constexpr int MI = T::MI, NJ = T::NJ, LA = T::LA, LB = T::LB, S = T::S;
  const int wm = w / T::WC, wn = w % T::WC;
  const uint32_t half = (uint32_t)(K / 2), kb = (uint32_t)(K / 32);
  const int mrows = (int)(mend - m0 < T::BM ? mend - m0 : T::BM);
  const int nrows = (int)(N - n0 < T::BN ? N - n0 : T::BN);

  // Rows past the tile's are past the resource and read as zero.
  const __amdgpu_buffer_rsrc_t ar = buf_rsrc_n(uniform_ptr(xq + m0 * half), mrows * half);
  const __amdgpu_buffer_rsrc_t br = buf_rsrc_n(uniform_ptr(wp + n0 * half), nrows * half);
  const __amdgpu_buffer_rsrc_t asr = buf_rsrc_n(uniform_ptr(xs + m0 * kb), mrows * kb);
  const __amdgpu_buffer_rsrc_t bsr = buf_rsrc_n(uniform_ptr(sp + n0 * kb), nrows * kb);

  // ---- memory -> LDS, 8 rows x 128 bytes per load.  Lane l writes the 16
  // bytes at 16 l: row l / 8, slot l % 8.  Slot s of row r holds chunk
  // s ^ ((r / 2) % 8) of the row's eight, so that the 16 rows a fragment read
  // touches at once lie in 16 different places of 256 bytes.
  const int lrow = lane >> 3, slot = lane & 7;
  uint32_t ao[LA], bo[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int row = 8 * (w * LA + i) + lrow;
    ao[i] = (uint32_t)row * half + 16u * (slot ^ ((row >> 1) & 7));
  }
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int row = 8 * (w * LB + i) + lrow;
    bo[i] = (uint32_t)row * half + 16u * (slot ^ ((row >> 1) & 7));
  }
  const int nks = (int)((half + kStepBytes - 1) / kStepBytes);
  // The step is part of the checked offset, so nothing past the tile's rows is
  // read.  K % 256 == 128: the last step's second half is the next row's; its
  // scales, both operands', read as 2^-127, and the products, below 2^-240,
  // add nothing.  Steps past the last one lie outside the resource.
  auto issue = [&](int ks, int stage) {
    uint8_t* base = smx + stage * T::STAGE;
    const uint32_t o = ks < nks ? (uint32_t)ks * kStepBytes : kPastEnd;
#pragma unroll
    for (int i = 0; i < LA; ++i)
      load_lds(ar, base + 1024 * (w * LA + i), ao[i] + o);
#pragma unroll
    for (int i = 0; i < LB; ++i)
      load_lds(br, base + T::A_STAGE + 1024 * (w * LB + i), bo[i] + o);
  };

  // ---- scales: lane (r, h) of fragment f loads 16 of the 32 scale bytes of
  // row r for four K steps; two exchanges between the wave's halves leave it
  // with one word a step, the scales of blocks 4 h .. 4 h + 3 of that step.
  const int r = lane & 31, h = lane >> 5;
  auto scale_load = [&](const __amdgpu_buffer_rsrc_t& rs, uint32_t row, int chunk) -> u32x4 {
    const uint32_t o = 32u * chunk + 16u * h;
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, row * kb + o, 0, 0));
  };
  // Words past the row's end (the next row's, or zero past the resource, whose
  // end is checked word by word) become zero, which is 2^-127.
  auto scale_mask = [&](u32x4 v, int chunk) -> u32x4 {
    const int left = (int)kb - 32 * chunk - 16 * h;  // scale bytes of the row from the lane's first on
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 4 * i < left ? v[i] : 0u;
    return v;
  };
  auto exchange = [&](u32x4 v) -> u32x4 {
    const auto p = __builtin_amdgcn_permlane32_swap(v.x, v.y, false, false);
    const auto q = __builtin_amdgcn_permlane32_swap(v.z, v.w, false, false);
    return u32x4{p[0], q[0], p[1], q[1]};  // steps 0, 1, 2, 3
  };
  u32x4 sa[MI], sb[NJ], na[MI], nb[NJ];
  auto scales_issue = [&](int chunk) {
#pragma unroll
    for (int i = 0; i < MI; ++i) na[i] = scale_load(asr, 32 * (wm * MI + i) + r, chunk);
#pragma unroll
    for (int j = 0; j < NJ; ++j) nb[j] = scale_load(bsr, 32 * (wn * NJ + j) + r, chunk);
  };

  f32x16 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // fragment addresses: chunk 4 h + J of row r
  const int x = (r >> 1) & 7;
  const uint8_t* af = smx + (32 * MI * wm + r) * kStepBytes;
  const uint8_t* bf = smx + T::A_STAGE + (32 * NJ * wn + r) * kStepBytes;
  int fo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) fo[j] = 16 * ((4 * h + j) ^ x);
  // Fragments of the four quarters of a K step.
  u32x4 av[4][MI], bv[4][NJ];
  auto frag = [&](int stage, auto jc) {
    constexpr int J = decltype(jc)::value;
    const uint8_t* a = af + stage * T::STAGE + fo[J];
    const uint8_t* b = bf + stage * T::STAGE + fo[J];
#pragma unroll
    for (int i = 0; i < MI; ++i) av[J][i] = *(const u32x4*)(a + 32 * kStepBytes * i);
#pragma unroll
    for (int j = 0; j < NJ; ++j) bv[J][j] = *(const u32x4*)(b + 32 * kStepBytes * j);
  };
  // rows i0 .. i1 - 1 of the wave's block, quarter J of a step
  auto mma = [&](auto jc, auto uc, int i0, int i1) {
    constexpr int J = decltype(jc)::value, U = decltype(uc)::value;
#pragma unroll
    for (int i = i0; i < i1; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = mx_mfma<J>(bv[J][j], av[J][i], acc[i][j], sb[j][U], sa[i][U]);
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};
  constexpr std::integral_constant<int, 2> c2{};
  constexpr std::integral_constant<int, 3> c3{};

  scales_issue(0);
#pragma unroll
  for (int p = 0; p < S; ++p) issue(p, p);
#pragma unroll
  for (int i = 0; i < MI; ++i) na[i] = exchange(scale_mask(na[i], 0));
#pragma unroll
  for (int j = 0; j < NJ; ++j) nb[j] = exchange(scale_mask(nb[j], 0));
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 1) * (LA + LB)) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  frag(0, c0);

  // One K step, with two barriers.  Every wave reads all of the stage into
  // registers under the MFMAs of the first quarter and a half; behind the
  // first barrier the stage is free and the step S further on is loaded into
  // it.  Before the last MFMAs each wave waits for its own share of the next
  // stage, which the second barrier makes whole, and reads its first quarter.
  // So a load has almost one and a half steps to arrive (with one barrier it
  // had one, and the step took as long as the load).  Nothing here is
  // conditional: a branch around MFMAs would make the compiler move 256
  // accumulators where it joins.
  auto step = [&](int ks, auto u) {
    constexpr int U = decltype(u)::value;
    const int stage = ks % S;
    if constexpr (U == 0) {
#pragma unroll
      for (int i = 0; i < MI; ++i) sa[i] = na[i];
#pragma unroll
      for (int j = 0; j < NJ; ++j) sb[j] = nb[j];
    }
    frag(stage, c1);
    frag(stage, c2);
    mma(c0, u, 0, MI);
    interleave<MI * NJ, 2 * (MI + NJ)>();
    __builtin_amdgcn_sched_barrier(0);
    frag(stage, c3);
    mma(c1, u, 0, MI / 2);
    interleave<MI * NJ / 2, MI + NJ>();
    __builtin_amdgcn_sched_barrier(0);
    mma(c1, u, MI / 2, MI);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if constexpr (U == 0) {
      scales_issue(ks / 4 + 1);
      __builtin_amdgcn_sched_barrier(0);  // before the stage's loads, which the second wait leaves outstanding
    }
    issue(ks + S, stage);
    mma(c2, u, 0, MI);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (U == 3) {
#pragma unroll
      for (int i = 0; i < MI; ++i) na[i] = exchange(scale_mask(na[i], ks / 4 + 1));
#pragma unroll
      for (int j = 0; j < NJ; ++j) nb[j] = exchange(scale_mask(nb[j], ks / 4 + 1));
    }
    mma(c3, u, 0, MI / 2);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 1) * (LA + LB)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    frag((ks + 1) % S, c0);
    mma(c3, u, MI / 2, MI);
    interleave<MI * NJ / 2, MI + NJ>();
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
  __builtin_amdgcn_s_barrier();  // every wave is done with its fragments
  asm volatile("" ::: "memory");
  constexpr int TURN = turn_bytes<TY, NJ>();
  static_assert(T::NW * TURN <= (int)T::lds, "the waves' turning places fit in LDS");
  turn_store<TY, MI, NJ>(smx + w * TURN, lane, acc, y, N, m0 + 32 * MI * wm, mend, n0 + 32 * NJ * wn);
}

template <typename T, typename TY, bool GROUPED>
__global__ __launch_bounds__(T::NT, 1) void k_mx_gemm(const uint8_t* __restrict__ xq, const uint8_t* __restrict__ xs,
                                                      int64_t M, int64_t K, const uint8_t* __restrict__ packed,
                                                      const uint8_t* __restrict__ scales, int64_t N,
                                                      void* __restrict__ y, const int* __restrict__ offsets,
                                                      int experts, uint32_t tiles_m, uint32_t tiles_n) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smx[];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // ---- tile: the list goes through bands of 8 M tiles, in a band N tile by N
  // tile: the 32 tiles that an XCD has at a time read 8 + 4 operand tiles
  int64_t m0, mend, n0;
  const uint8_t* wp = packed;
  const uint8_t* sp = scales;
  uint32_t t;
  int half;
  {
    uint32_t total = tiles_m * tiles_n;
    if constexpr (GROUPED) total = (uint32_t)grouped_tiles(offsets, experts, (int)M, T::BM, lane) * tiles_n;
    if (!xcd_tile<T::SLOTS, T::SPLIT>(total, t, half)) return;
    if constexpr (GROUPED) {
      GroupTile g;
      if (!find_group_tile(offsets, experts, (int)M, T::BM, tiles_n, t, lane, g)) return;
      const uint32_t own = (uint32_t)(g.rows + T::BM - 1) / T::BM;
      uint32_t tm, tn;
      band(g.tile, own, tiles_n, tm, tn);
      m0 = g.row0 + (int64_t)T::BM * tm;
      n0 = (int64_t)T::BN * tn;
      mend = g.row0 + g.rows;
      wp += (int64_t)g.expert * N * (K / 2);
      sp += (int64_t)g.expert * N * (K / 32);
    } else {
      uint32_t tm, tn;
      band(t, tiles_m, tiles_n, tm, tn);
      m0 = (int64_t)T::BM * tm;
      n0 = (int64_t)T::BN * tn;
      mend = M;
    }
  }
  if (half == 0 && mend > m0 + T::BM / 2) mend = m0 + T::BM / 2;
  if (half == 1) {
    m0 += T::BM / 2;
    if (m0 >= mend) return;
  }
  // half a tile, or one with rows in its upper half only, takes half the time
  if (half >= 0 || mend - m0 <= T::BM / 2)
    mx_tile<typename T::Half, TY>(smx, lane, w, xq, xs, K, wp, sp, N, (TY*)y, m0, mend, n0);
  else
    mx_tile<T, TY>(smx, lane, w, xq, xs, K, wp, sp, N, (TY*)y, m0, mend, n0);
}

bool mx_gemm_fits(int64_t k) { return k % 128 == 0; }

template <typename T, typename TY, bool GROUPED>
static hipError_t mx_gemm_go(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                             const uint8_t* scales, int64_t n, void* y, const int* offsets, int experts,
                             hipStream_t st) {
  static std::atomic<uint64_t> attr_done{0};  // LDS above the 64 KB default
  const hipError_t e = once_per_device(attr_done, [] {
    return hipFuncSetAttribute((const void*)k_mx_gemm<T, TY, GROUPED>, hipFuncAttributeMaxDynamicSharedMemorySize,
                               (int)T::lds);
  });
  if (e != hipSuccess) return e;
  const int64_t tiles_m = GROUPED ? grouped_max_tiles(m, experts, T::BM) : (m + T::BM - 1) / T::BM;
  const int64_t tiles_n = (n + T::BN - 1) / T::BN;
  const int64_t grid = xcd_grid<T::SLOTS, T::SPLIT>(tiles_m * tiles_n);
  k_mx_gemm<T, TY, GROUPED><<<dim3((unsigned)grid), T::NT, T::lds, st>>>(xq, xs, m, k, packed, scales, n, y, offsets,
                                                                       experts, (uint32_t)tiles_m, (uint32_t)tiles_n);
  return hipGetLastError();
}

// Workgroup tiles.  The first two have a CU to themselves (128 and 112 KB of
// LDS), of the third two share one.
typedef MxTile<256, 256, 2, 2, 2> MxLarge;
typedef MxTile<256, 192, 2, 2, 2> MxNarrow;
typedef MxTile<128, 128, 2, 2, 2> MxSmall;

// Time of all tiles in rounds of a large tile a CU.  Measured, K = 4096 to
// 16384: a round of narrow tiles takes 0.88 of a round of large ones, a round of
// halves of either about 0.6 of it, a round of small ones with two a CU 0.68,
// with one a CU 0.45 ([11008, 4096], 128 rows: 15 us against 31).

template <typename TY, bool GROUPED>
static hipError_t mx_gemm_pick(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                               const uint8_t* scales, int64_t n, void* y, const int* offsets, int experts,
                               hipStream_t st) {
  // by expert each one's last tile is half full on average, and each has one
  const int64_t some = experts < m ? experts : m;
  auto tiles = [&](int bm, int bn) {
    const int64_t half = m / bm + (some + 1) / 2;
    const int64_t tm = !GROUPED ? (m + bm - 1) / bm : half > some ? half : some;
    return tm * ((n + bn - 1) / bn);
  };
  const int64_t small = tiles(128, 128);
  const double large_t = xcd_rounds<32>(tiles(256, 256), 0.6), narrow_t = 0.88 * xcd_rounds<32>(tiles(256, 192), 0.6),
               small_t = small <= 256 ? 0.45 : 0.68 * (double)((small + 511) / 512);
  if (small_t <= large_t && small_t <= narrow_t)
    return mx_gemm_go<MxSmall, TY, GROUPED>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  if (narrow_t < large_t)
    return mx_gemm_go<MxNarrow, TY, GROUPED>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  return mx_gemm_go<MxLarge, TY, GROUPED>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
}

template <typename TY>
static hipError_t mx_gemm_form(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                               const uint8_t* scales, int64_t n, void* y, const int* offsets, int experts,
                               hipStream_t st) {
  if (offsets != nullptr) return mx_gemm_pick<TY, true>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  return mx_gemm_pick<TY, false>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
}

hipError_t launch_mx_gemm(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                          const uint8_t* scales, int64_t n, void* y, int y_dtype, const int* offsets, int experts,
                          hipStream_t st) {
  if (y_dtype == W4_F32) return mx_gemm_form<float>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  return mx_gemm_form<__bf16>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
}

}  // namespace w4
