// Transposed W4A16 product of many rows of bf16 dy, with low-rank adapters:
//   dx[m, k] = sum_n dy[m, n] (q[n, k] - zp[n, j]) s[n, j]  (+ sum_r low[m, r] A[l(m), r, k])
// on v_mfma_f32_32x32x16_bf16 with float32 accumulation; j is the group of column k.
//
// Workgroup tile 64 MI x 128, 64 weight rows a step.  Four waves multiply, each 32 MI x 64
// of the tile, and four load and convert, one of each on every SIMD.  dy, codes,
// scales and zero-points go from memory to LDS directly; the converting waves turn codes into weights,
// once a workgroup, in the operand tile [128 columns of dx][64 weight rows].
// A word of codes holds eight columns of one weight row while the sum runs over rows: a
// thread takes the same eight columns of four rows and stores four rows of each column
// as one 8-byte piece.  The pairs that a conversion to bf16 makes are two rows of one
// column, so turning costs no instruction of its own.
//
// A weight is the sum of PW bf16 parts, each an operand tile of its own: two with fp16 scales (15 bits with
// whole zero-points, so exact) and for a bf16 result (16 bits, off by 2^-16 of itself at most, beside the 2^-8 of the
// result's rounding), three for a float32 result of float32 scales (24 bits).  (One, a weight rounded to bf16,
// took 169 us for 2048 rows of [11008, 4096] where two take 260, and left an error against 64 bits of 2.3e-3 where the
// rounding of a bf16 result alone leaves 1.7e-3.)
//
// Bound by the matrix cores, which have twice the weights' products: 2048 rows of [11008, 4096] 260 us (370 GFLOP of them,
// 1.42 PFLOP/s; busy 73% of the time), 333 rows of [4096, 11008] 80 to 98.
#pragma once

#include <type_traits>

#include "lds_gemm.h"
#include "lora.h"
#include "w4_common.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int kTileK = 128;  // columns of dx a tile
constexpr int kTileN = 64;   // weight rows a step

// SUBS: groups of an operand tile's columns, 1 (groups of a multiple of 128) or 4.
template <int MI_, int PW_, int SUBS_> struct TilePlan {
  static constexpr int MI = MI_, PW = PW_, SUBS = SUBS_;
  static constexpr int BM = 64 * MI;  // four multiplying waves, two by two of 32 MI x 64
  static constexpr int AS = MI * PW <= 4 ? 3 : 2;  // stages of dy: what fits in 160 KB
  // bytes of a stage: dy (AS of them), weights (two), codes, and scales with zero-points (three)
  static constexpr int A_STAGE = BM * 128, B_PART = kTileK * 128, B_STAGE = PW * B_PART;
  static constexpr int RAW_STAGE = kTileN * kTileK / 2, TAB_HALF = SUBS * 256;
  static constexpr int TAB_STAGE = 2 * TAB_HALF;
  static constexpr int B_AT = AS * A_STAGE, RAW_AT = B_AT + 2 * B_STAGE, TAB_AT = RAW_AT + 3 * RAW_STAGE;
  static constexpr size_t lds = TAB_AT + 3 * TAB_STAGE;
  static_assert(lds <= 160 * 1024, "LDS of a CU");
};

// Slot (16 bytes) of chunk c (0 .. 3) of row n of a stage of codes: the 16 lanes
// that read one chunk of rows 4 b + i, b = 0 .. 15, meet every bank twice, the least there is.
__device__ __forceinline__ int raw_row(int slot) {  // the row that a slot has
  const int p = slot >> 2;
  return (p & ~7) | ((p & 1) << 2) | ((p >> 1) & 3);
}
__device__ __forceinline__ int raw_slot(int n, int c) {
  const int p = (n & ~7) | ((n >> 2) & 1) | ((n & 3) << 1);
  return 4 * p + (c ^ ((n >> 3) & 3));
}

// acc += low out for the wave's 32 MI rows from m0 (those before mend) and 64
// columns from c0, segment by segment: rows of other segments are zero in the operand, and
// keep their sums, since zero times an adapter that is not finite would be NaN.  (Loads of a block
// of ranks all issued ahead need registers that the sums have: forward, 1024 rows of [11008, 4096], 16 ranks, 126 -> 162 us.)
template <int MI>
__device__ __forceinline__ void add_adapters(const Adapters& ad, int lane, f32x16 (&acc)[MI][2], int64_t K, int64_t m0,
                                             int64_t mend, int64_t k0) {
  const int r = lane & 31, h = lane >> 5;
  const int64_t top = mend < m0 + 32 * MI ? mend : m0 + 32 * MI;
  for (int s = segments_before(ad.offsets, ad.segments, m0, lane); s < ad.segments; ++s) {
    const int64_t lo = ad.offsets[s] > m0 ? ad.offsets[s] : m0, hi = ad.offsets[s + 1] < top ? ad.offsets[s + 1] : top;
    if (lo >= top) break;
    const int l = ad.which[s];
    if (l < 0 || l >= ad.count || lo >= hi) continue;
    for (int r0 = 0; r0 < ad.rank; r0 += 16) {
      const bool in = r0 + 8 * h < ad.rank;
      bf16x8 w[2][3];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t k = k0 + 32 * j + r, at = ((int64_t)l * ad.rank + r0 + 8 * h) * K + k;
        const bool real = in && k < K;
        w[j][0] = w[j][1] = w[j][2] = zero8();
        if (ad.wide) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = real ? ((const float*)ad.out)[at + i * K] : 0.0f;
          pack8(v, w[j]);
        } else {
          uint16_t v[8];
          bf16x8 one[1];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = real ? ((const uint16_t*)ad.out)[at + i * K] : (uint16_t)0;
          pack8(v, one);
          w[j][0] = one[0];
        }
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int64_t m = m0 + 32 * i + r;
        if (m0 + 32 * i >= hi || m0 + 32 * i + 32 <= lo) continue;  // the same in every lane
        const bool own = m >= lo && m < hi;  // a lane's sums are all of row m
        bf16x8 a[3] = {zero8(), zero8(), zero8()};
        if (in && own) load8(ad.low + m * ad.rank + r0 + 8 * h, a);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f32x16 sum = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int p = 2; p >= 0; --p) {
            sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j][0], a[p], sum, 0, 0, 0);
            if (ad.wide) {
#pragma unroll
              for (int q = 1; q + p < 3; ++q) sum = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j][q], a[p], sum, 0, 0, 0);
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][j][e] += own ? sum[e] : 0.0f;
        }
      }
    }
  }
}

// The order of a slice's instructions: the next slice's reads under the first MFMAs.
template <typename T>
__device__ __forceinline__ void slice_order() {
  constexpr int M = 2 * T::MI * T::PW, R = T::MI + 2 * T::PW;
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (i < R) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace

// Steps first .. first + steps - 1 of 64 weight rows are part blockIdx.y's; with
// parts its float32 sums go to dx + blockIdx.y * M * K (TY float), without adapters, else the result to dx.
template <typename T, typename TS, typename TY>
__global__ __launch_bounds__(512, 2) void k_w4a16_tiles(
    const uint16_t* __restrict__ dy, int64_t M, const uint8_t* __restrict__ packed, const void* __restrict__ scales,
    const void* __restrict__ zeros, int64_t N, int64_t K, int g, int64_t row, int steps, Adapters ad, TY* __restrict__ dx,
    uint32_t tiles_m, uint32_t tiles_k) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t sm[];
  constexpr int MI = T::MI, BM = T::BM, PW = T::PW, SUBS = T::SUBS;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t t, tm, tk;
  int whole;
  if (!xcd_tile<32, false>(tiles_m * tiles_k, t, whole)) return;
  band(t, tiles_m, tiles_k, tm, tk);
  const int64_t m0 = (int64_t)BM * tm, k0 = (int64_t)kTileK * tk;
  const uint32_t half = (uint32_t)(K / 2), ng = (uint32_t)(K / g), drow = (uint32_t)(2 * row);
  const int all = (int)((N + kTileN - 1) / kTileN), first = (int)blockIdx.y * steps;
  const int nst = all - first < steps ? all - first : steps;  // steps of this part

  constexpr std::integral_constant<int, 0> n0{};
  constexpr std::integral_constant<int, 1> n1{};
  constexpr std::integral_constant<int, 2> n2{};
  constexpr std::integral_constant<int, 3> n3{};
  constexpr std::integral_constant<int, 4> n4{};
  constexpr std::integral_constant<int, 5> n5{};
  auto barrier = [&]() {
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // step(number) for every step, the numbers counted modulo 6, the period of two and three stages
  auto all_steps = [&](auto step) {
    for (int st = 0;;) {
      step(st, n0);
      if (++st >= nst) break;
      step(st, n1);
      if (++st >= nst) break;
      step(st, n2);
      if (++st >= nst) break;
      step(st, n3);
      if (++st >= nst) break;
      step(st, n4);
      if (++st >= nst) break;
      step(st, n5);
      if (++st >= nst) break;
    }
  };

  // Waves 4 to 7 load and convert, waves 0 to 3 multiply.  Barrier t, before which
  // the operands of step t have all been read, and those of t + 1 are whole, is passed by all.
  if (w >= 4) {
    const int pw = w - 4;
    // dy -> LDS: 8 rows x 128 bytes a load; slot s of row r holds chunk s ^ ((r / 2) % 8)
    constexpr int LA = BM / 32;
    const uint32_t mrows = (uint32_t)(M - m0 < BM ? M - m0 : BM);
    const __amdgpu_buffer_rsrc_t ar = buf_rsrc_n(uniform_ptr(dy + m0 * row), mrows * drow);
    uint32_t ao[LA];
    const int lrow = lane >> 3, slot = lane & 7;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int r = 8 * (pw * LA + i) + lrow;
      ao[i] = (uint32_t)r * drow + 16u * (slot ^ ((r >> 1) & 7));
    }
    auto a_issue = [&](int st, int stage, int i) {  // load i of a step
      const uint32_t n0 = st < nst ? (uint32_t)(first + st) * kTileN : (uint32_t)N, left = (uint32_t)N - n0;
      const int r = 8 * (pw * LA + i) + lrow;  // chunks past the last weight row read as zero
      load_lds_at(ar, sm + stage * T::A_STAGE + 1024 * (pw * LA + i),
                  8u * (slot ^ ((r >> 1) & 7)) < left ? ao[i] : kPastEnd, 2 * n0);
    };
    // Codes, scales and zero-points -> LDS.  Codes: 16 bytes a lane.  Scales: for
    // each weight row the 4 bytes that hold the value of a group (with fp16 two values,
    // of which the value's number in the array, odd or even, says which; the
    // array has an even number, so no word lies across its end).  SUBS 1: the first of these waves loads
    // scales, the second zero-points; SUBS 4: wave i those of columns 32 i .. 32 i + 31.
    const int sub0 = SUBS > 1 ? pw : 0;
    const int64_t kc = k0 + 32 * sub0;
    const uint32_t gi = (uint32_t)((kc < K ? kc : K - 1) / g);
    const int rs = 64 * pw + lane;  // the lane's slot of a load of codes by all four waves
    const int rn = raw_row(rs), rc = (rs & 3) ^ ((rn >> 3) & 3);
    const uint32_t ro = k0 / 2 + 16 * rc < half ? (uint32_t)rn * half + (uint32_t)(k0 / 2) + 16u * rc : kPastEnd;
    auto r_issue = [&](int st, int stage) {
      uint8_t* dst = sm + T::RAW_AT + stage * T::RAW_STAGE + 1024 * pw;
      const int64_t n0 = (int64_t)(first + st) * kTileN;
      const int64_t have = st < nst ? (N - n0 < kTileN ? N - n0 : kTileN) : 0;
      load_lds(buf_rsrc_n(uniform_ptr(packed + (st < nst ? n0 : 0) * half), (uint32_t)have * half), dst, ro);
    };
    auto s_issue = [&](int st, int stage) {
      uint8_t* tab = sm + T::TAB_AT + stage * T::TAB_STAGE;
      const int64_t n0 = (int64_t)(first + st) * kTileN;
      const int64_t have = st < nst ? (N - n0 < kTileN ? N - n0 : kTileN) : 0;
      const uint32_t bytes = (uint32_t)have * ng * (uint32_t)sizeof(TS);
      const int64_t byte = (st < nst ? n0 : 0) * ng * (int64_t)sizeof(TS);
      const uint32_t so = ((uint32_t)lane * ng + gi) * (uint32_t)sizeof(TS) & ~3u;
      if (SUBS > 1 || pw == 0)
        load_lds4(buf_rsrc_n(uniform_ptr((const char*)scales + byte), bytes), tab + 256 * sub0, so);
      if (SUBS > 1 || pw == 1)
        load_lds4(buf_rsrc_n(uniform_ptr((const char*)zeros + byte), bytes), tab + T::TAB_HALF + 256 * sub0, so);
    };

    // 4 floats -> two words of bf16, in PW parts: each the upper half of what is left, the second of two rounded to nearest
    auto put4 = [&](uint8_t* at, float (&v)[4]) {
      u32x2 d;
#pragma unroll
      for (int q = 0; q < PW; ++q) {
        if (PW == 2 && q == 1) {
          d.x = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[0], (__bf16)v[1]});
          d.y = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2], (__bf16)v[3]});
        } else {
          d.x = __builtin_amdgcn_perm(__float_as_uint(v[1]), __float_as_uint(v[0]), 0x07060302u);
          d.y = __builtin_amdgcn_perm(__float_as_uint(v[3]), __float_as_uint(v[2]), 0x07060302u);
        }
        *(u32x2*)(at + q * T::B_PART) = d;
        if (q + 1 < PW) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] -= __uint_as_float(__float_as_uint(v[i]) & 0xffff0000u);
        }
      }
    };
    auto value = [&](uint32_t word, uint32_t odd) {
      if constexpr (sizeof(TS) == 2) return (float)__builtin_bit_cast(_Float16, (uint16_t)(word >> (16 * odd)));
      else return __uint_as_float(word);
    };
    // one code with s and z: -zp s in two parts (exact with fp16 scales, 11 bits times 11), zp in three
    auto weight = [&](uint32_t byte, float s, float z) {
      const float q = (float)(uint8_t)byte;
      return PW == 2 ? fmaf(q, s, z) : (q - z) * s;
    };

    // The thread's piece is columns 8 kb .. 8 kb + 7 of weight rows 4 b .. 4 b + 3.
    const int b = lane & 15, kb = 4 * pw + (lane >> 4);
    int rawo[4], bo[4];
    uint32_t odd[4];  // whether the scale is the upper half of its word
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rawo[i] = T::RAW_AT + 16 * raw_slot(4 * b + i, pw) + 4 * (kb & 3);
      odd[i] = (gi + i * ng) & 1;
      // row r of the operand tile has its chunk of weight rows 8 (b / 2) .. at slot (b / 2) ^ ((r / 2) % 8)
      bo[i] = T::B_AT + 128 * (8 * kb + 2 * i) + 16 * ((b >> 1) ^ ((4 * kb + i) & 7)) + 8 * (b & 1);
    }
    // The weights of a step, from codes and scales of stages rs_ and ss to operands of stage bs.  `load` is
    // called between the eight parts of the work.
    auto convert = [&](int rs_, int ss, int bs, auto load) {
      uint8_t* out = sm + bs * T::B_STAGE;
      const uint8_t* tb = sm + T::TAB_AT + ss * T::TAB_STAGE;
      const u32x4 sw = *(const u32x4*)(tb + 256 * sub0 + 16 * b),
                  zw = *(const u32x4*)(tb + T::TAB_HALF + 256 * sub0 + 16 * b);
      uint32_t lo[4], hi[4];
      float s[4], z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t p = *(const uint32_t*)(sm + rawo[i] + rs_ * T::RAW_STAGE);
        s[i] = value(sw[i], odd[i]), z[i] = value(zw[i], odd[i]);
        if constexpr (PW == 2) z[i] *= -s[i];
        lo[i] = p & 0x0f0f0f0fu;
        hi[i] = (p >> 4) & 0x0f0f0f0fu;
        asm("" : "+v"(lo[i]), "+v"(hi[i]));  // no instruction: bytes are converted in place, not masked again one by one
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        load(j);
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = weight((j & 1 ? hi[i] : lo[i]) >> (8 * (j >> 1)), s[i], z[i]);
        put4(out + bo[j >> 1] + 128 * (j & 1), v);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

#pragma unroll
    for (int i = 0; i < 3; ++i) r_issue(i, i), s_issue(i, i);
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      a_issue(0, 0, i);
      if constexpr (T::AS == 3) a_issue(1, 1, i);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    barrier();  // all four waves' codes and scales of step 0 are there
    convert(0, 0, 0, [](int) {});
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    barrier();
    // In step t the loads of dy of t + 2 (t + 1 with two stages), of scales and of codes of t + 3 are issued, into
    // the places that step t - 1 has left, and the weights of t + 1 made.  Loads come in from the L2 cache
    // 1000 to 2000 cycles after their issue: with three stages they have two steps.  The loads of dy are
    // spread over the conversion; issued together they held it up (2048 rows of
    // [11008, 4096]: 185 us against 169).
    all_steps([&](int st, auto number) {
      constexpr int k = decltype(number)::value;
      r_issue(st + 3, k % 3);
      s_issue(st + 3, k % 3);
      convert((k + 1) % 3, (k + 1) % 3, (k + 1) % 2, [&](int j) {
        if (j % (8 / LA) == 0) a_issue(st + T::AS - 1, (k + T::AS - 1) % T::AS, j / (8 / LA));
      });
      // all but this step's loads; with two stages of dy, those too
      constexpr int scales_n = SUBS > 1 ? 2 : 1;
      if constexpr (T::AS == 2) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      else if (SUBS == 1 && pw > 1) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LA + 1) : "memory");
      else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LA + 1 + scales_n) : "memory");
      barrier();
    });
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may reach LDS when the sums are turned there
    barrier();
    return;
  }

  f32x16 acc[MI][2];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  const int r = lane & 31, h = lane >> 5, swz = (r >> 1) & 7;
  const int wm = w >> 1, wn = w & 1;
  // Slice q of a step: 16 weight rows, 8 a half.  The operands of a slice are read
  // under the MFMAs of the one before, those of a step's first behind the barrier before the last slice.
  int fa[4], fb[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    fa[q] = 128 * (32 * MI * wm + r) + 16 * ((2 * q + h) ^ swz);
    fb[q] = T::B_AT + 128 * (64 * wn + r) + 16 * ((2 * q + h) ^ swz);
  }
  bf16x8 av[2][MI], bv[2][PW][2];
  auto frag = [&](int as, int bs, auto qc) {
    constexpr int q = decltype(qc)::value;
    const uint8_t* a = sm + fa[q] + as * T::A_STAGE;
    const uint8_t* bt = sm + fb[q] + bs * T::B_STAGE;
#pragma unroll
    for (int p = 0; p < PW; ++p)
#pragma unroll
      for (int j = 0; j < 2; ++j) bv[q & 1][p][j] = *(const bf16x8*)(bt + p * T::B_PART + 128 * 32 * j);
#pragma unroll
    for (int i = 0; i < MI; ++i) av[q & 1][i] = *(const bf16x8*)(a + 128 * 32 * i);
  };
  auto mma = [&](auto qc) {
    constexpr int q = decltype(qc)::value;
#pragma unroll
    for (int p = 0; p < PW; ++p)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bv[q & 1][p][j], av[q & 1][i], acc[i][j], 0, 0, 0);
  };
  barrier();
  barrier();
  frag(0, 0, n0);
  all_steps([&](int st, auto number) {
    constexpr int k = decltype(number)::value, a = k % T::AS, e = k % 2;
    frag(a, e, n1);
    mma(n0);
    slice_order<T>();
    frag(a, e, n2);
    mma(n1);
    slice_order<T>();
    frag(a, e, n3);
    mma(n2);
    slice_order<T>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    barrier();
    frag((a + 1) % T::AS, 1 - e, n0);
    mma(n3);
    slice_order<T>();
  });
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  barrier();
  const int64_t mw = m0 + 32 * MI * wm, kw = k0 + 64 * wn;
  if (ad.count > 0) add_adapters<MI>(ad, lane, acc, K, mw, M, kw);
  constexpr int TURN = turn_bytes<TY, 2>();
  static_assert(4 * TURN <= (int)T::lds, "the waves' turning places fit in LDS");
  turn_store<TY, MI, 2, true>(sm + w * TURN, lane, acc, dx + (int64_t)blockIdx.y * M * K, K, mw, M, kw);
}

template <int MI, int PW, int SUBS, typename TS, typename TY>
static hipError_t tiles_go(const TilesArgs& a, const Adapters& ad, hipStream_t st) {
  typedef TilePlan<MI, PW, SUBS> T;
  static std::atomic<uint64_t> attr_done{0};  // LDS above the 64 KB default
  const hipError_t e = once_per_device(attr_done, [] {
    return hipFuncSetAttribute((const void*)k_w4a16_tiles<T, TS, TY>, hipFuncAttributeMaxDynamicSharedMemorySize,
                               (int)T::lds);
  });
  if (e != hipSuccess) return e;
  const int64_t tiles_m = (a.m + T::BM - 1) / T::BM, tiles_k = (a.k + kTileK - 1) / kTileK;
  const dim3 grid((unsigned)xcd_grid<32, false>(tiles_m * tiles_k), (unsigned)a.parts);
  k_w4a16_tiles<T, TS, TY><<<grid, 512, T::lds, st>>>((const uint16_t*)a.x, a.m, a.packed, a.scales, a.zeros, a.n, a.k,
                                                     a.g, a.row, a.steps, ad, (TY*)a.y, (uint32_t)tiles_m, (uint32_t)tiles_k);
  return hipGetLastError();
}

}  // namespace w4
