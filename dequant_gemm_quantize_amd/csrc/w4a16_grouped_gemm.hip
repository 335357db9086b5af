// W4A16 product by expert for many rows an expert, bf16 x:
//   y[t, n] = sum over groups j of s (sum_{k in j} x q - zp sum_{k in j} x)
// for the expert of row t, on v_mfma_f32_32x32x16_bf16 with float32 accumulation.
//
// A code 0..15 is an exact bf16, so no weight is rounded: a unit of 128 (64, 32:
// what divides the group) columns is summed by itself, and the float32 sums
// take the scale in one fma each.  The zero-points' part is a product of its
// own with one column a unit, s zp times the unit's sum of x, each the sum of
// three bf16 values (8 of the 9 products, the ninth below 2^-32): one MFMA for
// two units.  The sums of x come from an MFMA against ones, 16 rows a wave.
// (Weights rounded to bf16 before the product took 390 us where this takes 440
// to 465, and left an error against 64 bits of 2.3e-3 where the rounding of bf16 y
// alone leaves 1.7e-3; as the sum of two bf16 values they took 650.)
//
// Workgroup tile 128 x 128 or 64 x 128 of four waves, each all the rows of 32
// columns: a lane holds one weight row, so its scale and zero-point are one
// register each, and no two waves convert the same code.  Two or three
// workgroups a CU, so that one's conversions and sums run beside another's
// MFMAs.  x goes from memory to LDS directly, two stages of 64 columns
// (128-byte lines); the packed weights the same way, two stages of 256 columns
// (again 128-byte lines), and from there to registers, where a wave turns its
// own 32 rows into operands.
//
// Bound by the matrix cores and the vector instructions (6 an MFMA with units
// of 128 columns, more with shorter ones), which are busy half of the time each
// and wait for each other.  Experts [11008, 4096], 8 of them, bf16 y, fp16 scales:
// 4096 rows 440 - 465 us (0.8 PFLOP/s; a large bf16 product of the library reaches
// 1.53), with groups of 64 540, of 32 715; 1200 rows 176 / 219 / 306, 256 rows 71 /
// 97 / 136.
#include <type_traits>

#include "grouped.h"
#include "lds_gemm.h"
#include "w4_common.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int GLine = 128;  // bytes of a row per stage: 64 bf16 or 256 codes

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

template <typename TS> struct Pair {
  typedef TS type __attribute__((ext_vector_type(2)));
};

// 8 codes -> 8 bf16 in column order, exactly.  A byte of 0..15 read as OCP
// E4M3 is that number times 2^-9 (subnormals, then the first binade), so the
// conversion at scale 2^9 gives the code itself, two at a time.
__device__ __forceinline__ u32x4 codes_bf16(uint32_t p) {
  const uint32_t even = p & 0x0f0f0f0fu, odd = (p >> 4) & 0x0f0f0f0fu;
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u);  // columns 0 1 2 3, a byte each
  const uint32_t hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);
  u32x4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
  return r;
}

// v as the sum of three bf16 values, each the upper half of what is left (exact).
__device__ __forceinline__ void three_parts(float v, uint32_t (&p)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    p[i] = __float_as_uint(v) >> 16;
    v -= __uint_as_float(p[i] << 16);
  }
}

constexpr int GBN = 128;  // columns of a workgroup's tile: 32 for each of four waves

// Workgroup tile of BM = 32 MI rows; two stages of 64 columns of x, two of 256
// columns of codes, and the parts of the sums of x of two units, twice.
template <int BM_, int WAVES_> struct GTile {
  static constexpr int BM = BM_, MI = BM / 32;
  static constexpr int WAVES = WAVES_;                     // waves of a SIMD that the registers are cut for
  static constexpr int LA = BM / 32, LW = GBN / 32;        // 1 KB loads per wave and stage
  static constexpr int A_STAGE = BM * GLine, W_STAGE = GBN * GLine;
  static constexpr int SUMS = 2 * (A_STAGE + W_STAGE);     // where the sums of x are
  static constexpr size_t lds = SUMS + 4 * 16 * (size_t)BM;
};

}  // namespace

// One tile: rows m0 .. min(m0 + BM, mend) - 1 of y, columns from n0, for the
// expert whose first weight row is ebase.  F: K slices of 16 columns that are
// summed before the scale is applied, a unit (8, 4 or 2: the largest whose
// columns divide the group).
template <typename T, int F, typename TS, typename TY>
__device__ __forceinline__ void gg_tile(uint8_t* sgg, int lane, int w, const uint16_t* __restrict__ x, int64_t K,
                                        const uint8_t* __restrict__ packed, const void* __restrict__ scales,
                                        const void* __restrict__ zeros, int64_t N, int g, TY* __restrict__ y, int64_t m0,
                                        int64_t mend, int64_t n0, int64_t ebase) {
  constexpr int MI = T::MI, LA = T::LA, LW = T::LW, BM = T::BM;
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
  uint8_t* sw = sgg + 2 * T::A_STAGE;
  // steps and stages past the last lie outside the resources
  auto x_issue = [&](int ks, int stage) {
    const uint32_t o = ks < nks ? (uint32_t)ks * GLine : kPastEnd;
#pragma unroll
    for (int i = 0; i < LA; ++i) load_lds(xr, sgg + stage * T::A_STAGE + 1024 * (w * LA + i), xo[i] + o);
  };
  auto w_issue = [&](int st) {
    const uint32_t o = 4 * st < nks ? (uint32_t)st * GLine : kPastEnd;
#pragma unroll
    for (int i = 0; i < LW; ++i) load_lds(wr, sw + (st & 1) * T::W_STAGE + 1024 * (w * LW + i), wo[i] + o);
  };

  // Scales of the lane's weight row for the units of a stage, and zero-points
  // of every second one: half h takes those of units 2 p + h.
  const int r = lane & 31, h = lane >> 5;
  const uint32_t n_lane = 32 * w + r;
  constexpr int NP = 8 / F;  // pairs of units of a stage
  struct Scales {
    typename Pair<TS>::type s[NP];  // two to a register where they fit
    TS z[NP];
  };
  // unit / (units of a group) by a product: exact below 2^16 units, K <= 2^21
  const uint32_t upg = (uint32_t)g / (16 * F), inv = 0xffffffffu / upg + 1;
  auto s_load = [&](int st) {
    Scales v;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      uint32_t gi[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t unit = 2 * (NP * (uint32_t)st + p) + q;
        gi[q] = upg == 1 ? unit : __umulhi(unit, inv);
      }
      // past the row's last group only for units that do not exist: zero
      auto at = [&](uint32_t i) { return i < ng ? n_lane * ng + i : kPastEnd / (uint32_t)sizeof(TS); };
      v.s[p].x = GScale<TS>::load(sr, at(gi[0]));
      v.s[p].y = GScale<TS>::load(sr, at(gi[1]));
      v.z[p] = GScale<TS>::load(zr, at(h ? gi[1] : gi[0]));
    }
    return v;
  };
  Scales now, next;

  // acc: the scaled sums; d: the running unit's, which `sfold` will scale
  f32x16 acc[MI][1], d[MI], none;
  float sfold = 0.0f;
#pragma unroll
  for (int e = 0; e < 16; ++e) none[e] = 0.0f;
#pragma unroll
  for (int i = 0; i < MI; ++i) acc[i][0] = d[i] = none;
  auto fold = [&](int i) {
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[i][0][e] = fmaf(sfold, d[i][e], acc[i][0][e]);
    asm("" : "+v"(acc[i][0]));  // no instruction: keeps the 16 sums in the registers they came from
  };

  // Slice t of a step: half h has columns 8 c .. 8 c + 7, c = 4 (t / 2) + 2 h + t % 2,
  // so a slice stays within a block of 32 columns and the two words of
  // codes that a lane takes of a block are neighbours.  (A stage of x goes by the
  // step's number within a stage of codes, so that LDS addresses have fixed offsets.)
  const int swz = (r >> 1) & 7;
  int fo[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) fo[t] = r * GLine + 16 * ((4 * (t >> 1) + 2 * h + (t & 1)) ^ swz);
  u32x4 xv[2][MI];
  auto x_frag = [&](int stage, auto tc) {
    constexpr int t = decltype(tc)::value;
    const uint8_t* a = sgg + stage * T::A_STAGE + fo[t];
#pragma unroll
    for (int i = 0; i < MI; ++i) xv[t & 1][i] = *(const u32x4*)(a + 32 * GLine * i);
  };
  u32x4 cv, cnext;
  auto codes = [&](int st, int u) {
    const uint8_t* b = sw + (st & 1) * T::W_STAGE + n_lane * GLine + 8 * h;
    const u32x2 c0 = *(const u32x2*)(b + 16 * ((2 * u) ^ swz)), c1 = *(const u32x2*)(b + 16 * ((2 * u + 1) ^ swz));
    cnext = u32x4{c0.x, c0.y, c1.x, c1.y};
  };
  u32x4 wv[2];
  auto convert = [&](auto tc) {
    constexpr int t = decltype(tc)::value;
    wv[t & 1] = codes_bf16(cv[t]);
  };
  // slice t of step u; where it begins a unit, the unit before is scaled and added first
  auto mma = [&](auto tc, auto uc) {
    constexpr int t = decltype(tc)::value, u = decltype(uc)::value, unit = (4 * u + t) / F;
    constexpr bool begins = (4 * u + t) % F == 0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if constexpr (begins) {
        fold(i);
        __builtin_amdgcn_sched_barrier(0);  // d's registers are free: no second set of them
      }
      d[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, xv[t & 1][i]),
                                                     __builtin_bit_cast(bf16x8, wv[t & 1]), begins ? none : d[i], 0, 0,
                                                     0);
    }
    if constexpr (begins) sfold = (float)now.s[unit / 2][unit & 1];
  };

  // Sums of x over the columns of a unit: 16 rows a wave by an MFMA against
  // ones, split into three bf16 parts and left in LDS as an operand of 8
  // values, hi mid lo hi mid lo hi mid, at [pair of units % 2][unit % 2][row].
  constexpr int SR = BM > 64 ? BM / 64 : 1;  // blocks of 16 rows a wave sums
  const int l16 = lane & 15, h4 = lane >> 4;
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
  const int srow = 16 * (SR * w % (BM / 16));  // (with fewer blocks than waves, several waves write the same values)
  f32x4 xsum[SR];
  u32x4 xs[SR][2];
  auto sum_frag = [&](int stage) {
#pragma unroll
    for (int q = 0; q < SR; ++q)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int row = srow + 16 * q + l16;
        xs[q][b] = *(const u32x4*)(sgg + stage * T::A_STAGE + row * GLine + 16 * ((4 * b + h4) ^ ((row >> 1) & 7)));
      }
  };
  auto sum_put = [&](int q, int unit) {
    // register e of a lane holds row 4 h4 + e, whatever l16: lanes l16 % 4 == e write it
    const f32x4 v = xsum[q];
    const int e = l16 & 3;
    uint32_t p[3];
    three_parts(e < 2 ? (e == 0 ? v[0] : v[1]) : (e == 2 ? v[2] : v[3]), p);
    const u32x4 op = {p[0] | p[1] << 16, p[2] | p[0] << 16, p[1] | p[2] << 16, p[0] | p[1] << 16};
    *(u32x4*)(sgg + T::SUMS + 16 * ((unit & 3) * BM + srow + 16 * q + 4 * h4 + e)) = op;
  };
  auto sums = [&](int ks, auto uc) {
    constexpr int u = decltype(uc)::value;
#pragma unroll
    for (int q = 0; q < SR; ++q) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        constexpr f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
        const bool begins = (2 * u + b) * 2 % F == 0;
        xsum[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xs[q][b]), ones,
                                                          begins ? zero : xsum[q], 0, 0, 0);
        if ((2 * u + b + 1) * 2 % F == 0) sum_put(q, (4 * ks + 2 * b) / F);
      }
    }
  };
  // The zero-points of a pair, p of the stage: acc -= s zp (sum of x), a product
  // of K = 16 whose lower half is the first unit's parts, the upper the second's.
  u32x4 xc[MI], wc;
  auto zero_frag = [&](int pair, int p) {
    const uint8_t* a = sgg + T::SUMS + 16 * (((2 * pair & 3) + h) * BM + r);
#pragma unroll
    for (int i = 0; i < MI; ++i) xc[i] = *(const u32x4*)(a + 32 * 16 * i);
    uint32_t c[3];
    three_parts(-(float)(h ? now.s[p].y : now.s[p].x) * (float)now.z[p], c);
    wc = u32x4{c[0] | c[0] << 16, c[0] | c[1] << 16, c[1] | c[1] << 16, c[2] | c[2] << 16};
  };
  auto zero_mma = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
      acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, xc[i]),
                                                          __builtin_bit_cast(bf16x8, wc), acc[i][0], 0, 0, 0);
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};
  constexpr std::integral_constant<int, 2> c2{};
  constexpr std::integral_constant<int, 3> c3{};

  now = s_load(0);
  w_issue(0);
  x_issue(0, 0);
  x_issue(1, 1);
  // a unit that does not exist has the zero-point term 0 times what its place holds: a number
  for (int i = threadIdx.x; i < 4 * BM; i += 256) *(u32x4*)(sgg + T::SUMS + 16 * i) = u32x4{0, 0, 0, 0};
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LA) : "memory");  // all but the second step's x
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  codes(0, 0);
  cv = cnext;
  x_frag(0, c0);
  convert(c0);

  // One K step of 64 columns, four slices.  A slice's x reads and conversions
  // run under the MFMAs of the one before.  Before the last slice every wave
  // has read all of the step's x and waited for its share of the next step's;
  // behind the barrier that is whole and this step's x stage is free.  The
  // next step's codes are read a slice earlier still: their stage has been
  // whole since the barrier of u = 1.  The sums of x that the step ends are
  // whole behind its barrier too, and their places are written again two pairs
  // of units, so at least one barrier, later.
  auto step = [&](int ks, auto uc) {
    constexpr int u = decltype(uc)::value;
    constexpr bool pair_ends = (4 * u + 4) % (2 * F) == 0;
    sum_frag(u % 2);
    x_frag(u % 2, c1);
    convert(c1);
    mma(c0, uc);
    __builtin_amdgcn_sched_barrier(0);
    sums(ks, uc);
    x_frag(u % 2, c2);
    codes((ks + 1) / 4, (u + 1) & 3);
    convert(c2);
    mma(c1, uc);
    __builtin_amdgcn_sched_barrier(0);
    x_frag(u % 2, c3);
    convert(c3);
    mma(c2, uc);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if constexpr (u == 0) w_issue(ks / 4 + 1);
    if constexpr (u == 1) next = s_load(ks / 4 + 1);
    x_issue(ks + 2, u % 2);
    cv = cnext;
    x_frag((u + 1) % 2, c0);
    if constexpr (pair_ends) zero_frag(2 * ks / F, 2 * u / F);
    convert(c0);
    mma(c3, uc);
    if constexpr (pair_ends) zero_mma();
    if constexpr (u == 3) now = next;
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
#pragma unroll
  for (int i = 0; i < MI; ++i) fold(i);
  if (4 * nks % (2 * F) != 0) {  // the last unit has no second one
    if (F == 4 && nks % 4 == 3) now.s[0] = now.s[NP - 1], now.z[0] = now.z[NP - 1];
    zero_frag(2 * (nks - 1) / F, 0);
    zero_mma();
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");  // no load may reach LDS after the workgroup has left it
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  constexpr int TURN = turn_bytes<TY, 1>();
  static_assert(4 * TURN <= (int)T::lds, "the waves' turning places fit in LDS");
  turn_store<TY, MI, 1, false>(sgg + w * TURN, lane, acc, y, N, m0, mend, n0 + 32 * w);
}

template <typename T, typename H, int F, typename TS, typename TY>
__global__ __launch_bounds__(256, T::WAVES) void k_w4a16_grouped_gemm(
    const uint16_t* __restrict__ x, int64_t rows, int64_t K, const int* __restrict__ offsets, int experts,
    const uint8_t* __restrict__ packed, const void* __restrict__ scales, const void* __restrict__ zeros, int64_t N,
    int g, TY* __restrict__ y, uint32_t tiles_n) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t sgg[];  // x stages, weight stages, sums of x
  constexpr int BM = T::BM;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  int64_t m0, mend, n0;
  int64_t ebase;  // the expert's first weight row
  int half;
  {
    const uint32_t total = (uint32_t)grouped_tiles(offsets, experts, (int)rows, BM, lane) * tiles_n;
    uint32_t t;
    if (!xcd_tile<32, false>(total, t, half)) return;
    GroupTile gt;
    if (!find_group_tile(offsets, experts, (int)rows, BM, tiles_n, t, lane, gt)) return;
    uint32_t tm, tn;
    band(gt.tile, (uint32_t)(gt.rows + BM - 1) / BM, tiles_n, tm, tn);
    m0 = gt.row0 + (int64_t)BM * tm;
    n0 = (int64_t)GBN * tn;
    mend = gt.row0 + gt.rows;
    ebase = (int64_t)gt.expert * N;
  }
  // a tile with rows in its upper half only takes half the time
  if (mend - m0 <= BM / 2) {
    gg_tile<H, F, TS, TY>(sgg, lane, w, x, K, packed, scales, zeros, N, g, y, m0, mend, n0, ebase);
    return;
  }
  gg_tile<T, F, TS, TY>(sgg, lane, w, x, K, packed, scales, zeros, N, g, y, m0, mend, n0, ebase);
}

// K % 64 == 0: whole steps; 128 rows of K bf16 stay below 2^31 bytes.
bool w4a16_grouped_gemm_fits(int64_t k) { return k % 64 == 0 && k <= ((int64_t)1 << 21); }

template <typename T, typename H, int F, typename TS, typename TY>
static hipError_t gg_go(const uint16_t* x, int64_t t, int64_t k, const int* offsets, int experts,
                        const uint8_t* packed, const void* scales, const void* zeros, int64_t n, int g, void* y,
                        hipStream_t st) {
  static std::atomic<uint64_t> attr_done{0};  // LDS above the 64 KB default
  const hipError_t e = once_per_device(attr_done, [] {
    return hipFuncSetAttribute((const void*)k_w4a16_grouped_gemm<T, H, F, TS, TY>,
                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)T::lds);
  });
  if (e != hipSuccess) return e;
  const int64_t tiles_n = (n + GBN - 1) / GBN;
  const int64_t grid = xcd_grid<32, false>(grouped_max_tiles(t, experts, T::BM) * tiles_n);
  k_w4a16_grouped_gemm<T, H, F, TS, TY><<<dim3((unsigned)grid), 256, T::lds, st>>>(
      x, t, k, offsets, experts, packed, scales, zeros, n, g, (TY*)y, (uint32_t)tiles_n);
  return hipGetLastError();
}

// 72 KB of LDS, two workgroups a CU; 52 KB, three.
typedef GTile<128, 2> GLarge;
typedef GTile<64, 2> GLargeHalf;
typedef GTile<64, 3> GSmall;
typedef GTile<32, 3> GSmallHalf;

template <int F, typename TS, typename TY>
static hipError_t gg_size(const uint16_t* x, int64_t t, int64_t k, const int* offsets, int experts,
                          const uint8_t* packed, const void* scales, const void* zeros, int64_t n, int g, void* y,
                          hipStream_t st) {
  // us with 128 / 64 rows a tile, groups of 128, 64 and 32: 16 experts [2050, 2048], 2600 rows 48 / 56, 54 / 64,
  // 73 / 87; 8 of [11008, 4096], 1200 rows 176 / 175, 212 / 214, 293 / 297; 16 of [2048, 2048], 2048 rows
  // 39 / 35, 47 / 43, 66 / 64.
  // (A launch has fewer than 2^32 threads, which the smaller tiles of the largest calls could exceed.)
  const bool too_many = grouped_max_tiles(t, experts, 64) * ((n + GBN - 1) / GBN) >= (1 << 24) - 8;
  if (t > 144 * (int64_t)experts || too_many)
    return gg_go<GLarge, GLargeHalf, F, TS, TY>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  return gg_go<GSmall, GSmallHalf, F, TS, TY>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
}

template <typename TS, typename TY>
static hipError_t gg_pick(const uint16_t* x, int64_t t, int64_t k, const int* offsets, int experts,
                          const uint8_t* packed, const void* scales, const void* zeros, int64_t n, int g, void* y,
                          hipStream_t st) {
  if (g % 128 == 0) return gg_size<8, TS, TY>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  if (g % 64 == 0) return gg_size<4, TS, TY>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  return gg_size<2, TS, TY>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
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
