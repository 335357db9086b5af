// W4A16 product by expert for few rows an expert (decode), bf16 x, and for any
// number of rows, float32 x:
//   y[t, n] = sum over groups j of s (sum_{k in j} x (16 + q) - (16 + zp) sum_{k in j} x)
// on v_mfma_f32_16x16x32_bf16 (16 token rows, 16 weight rows).  16 + q is an
// exact bfloat16 whose mantissa bits 3..6 are the code: a shift and an and-or
// make a pair of operands, codes i and i + 4 of a word (x is put into that
// order once a slice).  The sums of x come from the same instruction against
// ones.  Nothing is rounded below float32; 16 rather than 128 + q keeps the
// part that cancels small.  float32 x is the sum of three bf16 values (8 bits of
// its 24 each), which take three MFMAs to a pair of codes converted once.
//
// Bound by the weight bytes, and close behind by the vector unit that turns
// codes into operands.  A workgroup goes through RB blocks of 16 weight rows of
// one expert, all of K, for up to 16 token rows (one block a workgroup was
// slower: starting the waves, about 13 cycles each on every XCD, then takes
// longer than reading the weights).  Its waves have a slice of K each, 512
// columns with G128 (or take such slices in turn): a wave keeps x of its slice,
// and its sums, in registers for all the blocks, and the codes and scales of
// the next block are in flight while one is computed.  The waves add
// their sums through LDS at the end.  A call's share of a replayed graph of
// calls, weights rotated: two rows of two experts [11008, 4096] 14.6 us (3.1 TB/s; the
// kernel alone 13.6), 16 rows of 64 experts [2048, 2048] 11.1 us; float32 x 17.8
// and 15.7 us (multiply-adds of the vector unit, a weight row a lane, took 129
// and 83).  Groups of 32, 16 rows of 64 experts: 17.4 us.
//
// The codes are loaded as 256-byte runs of a row (128 without G128) and
// regrouped through the wave's own place in LDS, row t's 16-byte piece c at slot
// c ^ t (c ^ (t / 2 % 8)), free of bank conflicts; LDS operations of a wave
// complete in order.  G128 (groups of a multiple of 128): lane (l16, h) has
// piece 4 j + h of row l16, a 32-column block of each 128 columns, and x's
// columns to match.  Otherwise a group may end at any 32-column block, so an
// MFMA takes one block, of which lane (l16, h) has 8 columns.
#include <type_traits>

#include "grouped.h"
#include "lds_gemm.h"
#include "w4_common.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int kGRowsGrid = 1 << 20;  // workgroups; more tiles than that loop

// mask and magic of the conversion, kept in registers (w4_common.h, NibConst)
struct Nib16 {
  uint32_t mask, magic;
  __device__ static Nib16 make() {
    Nib16 k{0x00780078u, 0x41804180u};
    asm("" : "+v"(k.mask), "+v"(k.magic));
    return k;
  }
};

// 8 codes -> 16 + q as bf16 in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 codes16(uint32_t p, const Nib16& nk) {
  u32x4 r;
  r.x = ((p << 3) & nk.mask) | nk.magic;
  r.y = ((p >> 1) & nk.mask) | nk.magic;
  r.z = ((p >> 5) & nk.mask) | nk.magic;
  r.w = ((p >> 9) & nk.mask) | nk.magic;
  return __builtin_bit_cast(bf16x8, r);
}

// 8 consecutive bf16 into that order.
__device__ __forceinline__ bf16x8 order_as_codes(u32x4 v) {
  u32x4 r;
  r.x = __builtin_amdgcn_perm(v.z, v.x, 0x05040100u);  // 0 4
  r.y = __builtin_amdgcn_perm(v.z, v.x, 0x07060302u);  // 1 5
  r.z = __builtin_amdgcn_perm(v.w, v.y, 0x05040100u);  // 2 6
  r.w = __builtin_amdgcn_perm(v.w, v.y, 0x07060302u);  // 3 7
  return __builtin_bit_cast(bf16x8, r);
}

// 8 consecutive float32 as hi + mid + lo, each bf16 in that order: the upper
// halves of the words, of what they lack, and of what that lacks, which is exact.
__device__ __forceinline__ void split_as_codes(u32x4 v0, u32x4 v1, bf16x8 (&out)[3]) {
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = __builtin_amdgcn_perm(v1[i], v0[i], 0x07060302u);
      if (p < 2) {
        v0[i] = __float_as_uint(__uint_as_float(v0[i]) - __uint_as_float(v0[i] & 0xffff0000u));
        v1[i] = __float_as_uint(__uint_as_float(v1[i]) - __uint_as_float(v1[i] & 0xffff0000u));
      }
    }
    out[p] = __builtin_bit_cast(bf16x8, r);
  }
}

// The value that each of the wave's four rows of 16 lanes holds, in every row.
__device__ __forceinline__ void spread4(uint32_t v, uint32_t (&out)[4]) {
  const auto half = __builtin_amdgcn_permlane32_swap(v, v, false, false);  // rows 0 1 0 1 and 2 3 2 3
  const auto lo = __builtin_amdgcn_permlane16_swap(half[0], half[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(half[1], half[1], false, false);
  out[0] = lo[0], out[1] = lo[1], out[2] = hi[0], out[3] = hi[1];
}

template <typename TS>
__device__ __forceinline__ float scale_value(uint32_t v) {
  if constexpr (sizeof(TS) == 2) return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
  else return __uint_as_float(v);
}

}  // namespace

// SL: 32-column blocks of a wave's slice, 16 or 8.
template <typename TX, typename TS, typename TY, bool G128, int SL, int RB>
__global__ __launch_bounds__(512, 2) void k_w4a16_grouped_rows(
    const TX* __restrict__ x, int64_t T, int64_t K, const int* __restrict__ offsets, int experts,
    const uint8_t* __restrict__ packed, const void* __restrict__ scales, const void* __restrict__ zeros, int64_t N,
    int g, TY* __restrict__ y, uint32_t tiles_n, int64_t tiles) {
  // [waves][16 tokens][16 RB rows] sums; before them 256 SL bytes a wave to regroup weights
  extern __shared__ __attribute__((aligned(16))) float part[];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6;
  const int l16 = lane & 15, h = lane >> 4;
  constexpr int RPL = 64 / SL, NC = 16 / RPL;  // rows a load covers, loads a block
  const int lp = lane % SL, lr = lane / SL;    // the lane's piece and row of them
  const uint32_t ng = (uint32_t)(K / g), half = (uint32_t)(K / 2), xrow = (uint32_t)(sizeof(TX) * K);
  const int blocks32 = (int)(K / 32), slices = (blocks32 + SL - 1) / SL;
  const uint32_t bpg = (uint32_t)g / 32;
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
  const Nib16 nk = Nib16::make();
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int NS = G128 ? SL / 4 : SL;  // scales of a row in a slice
  // blocks whose codes are held at a time (with three the sums of six blocks
  // left no registers: 16.5 us against 14.6 for two rows of [11008, 4096])
  constexpr int D = RB < 2 ? 1 : 2;
  constexpr int NX = sizeof(TX) == 4 ? 3 : 1, WX = sizeof(TX) / 2;  // bf16 parts of x; 16-byte loads of 8 columns
  constexpr int NL = 2 * NS / 4;    // loads of them, a scale or zero-point a lane
  typedef typename std::conditional<sizeof(TS) == 2, uint16_t, uint32_t>::type Raw;
  u32x4* place = (u32x4*)part + 16 * SL * w;

  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    GroupTile gt;
    if (!find_group_tile(offsets, experts, (int)T, 16, tiles_n, tile, lane, gt)) break;
    const int64_t n0 = (int64_t)16 * RB * (gt.tile % tiles_n), r0 = gt.row0 + (int64_t)16 * (gt.tile / tiles_n);
    const int tokens = (int)(gt.row0 + gt.rows - r0 < 16 ? gt.row0 + gt.rows - r0 : 16);
    const int rows = (int)(N - n0 < 16 * RB ? N - n0 : 16 * RB);
    const int64_t first = (int64_t)gt.expert * N + n0;
    // weight rows past the end are past the resource and read as zero; their
    // scales repeat the last row's
    const __amdgpu_buffer_rsrc_t wr = buf_rsrc_n(uniform_ptr(packed + first * half), (uint32_t)rows * half);
    const __amdgpu_buffer_rsrc_t xr = buf_rsrc_n(uniform_ptr(x + r0 * K), (uint32_t)tokens * xrow);
    f32x4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = zero;

    for (int s = w; s < slices; s += nw) {
      const int b0 = SL * s;                                   // the slice's first 32-column block
      const int nb = blocks32 - b0 < SL ? blocks32 - b0 : SL;  // its blocks; those past K read x as zero
      u32x4 cv[D][NC];
      Raw sz[D][NL];
      const uint32_t wo = (uint32_t)lr * half + 16u * lp + (uint32_t)s * (16 * SL);
      // Scale or zero-point 4 i + h of the slice's 2 NS for row l16 (the scales
      // first).  One value a lane, spread over the lanes afterwards: these
      // gathers cost the address unit 64 lanes each whatever they fetch, and
      // with one load for every value they took longer than the codes.
      const Raw* sp[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int which = 4 * i + h, blk = (G128 ? 4 : 1) * (which % NS);
        sp[i] = (const Raw*)(which < NS ? scales : zeros) + first * ng + (uint32_t)(b0 + (blk < nb ? blk : 0)) / bpg;
      }
      auto load = [&](int b) {
        const int u = b % D;
#pragma unroll
        for (int i = 0; i < NC; ++i)
          cv[u][i] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, wo + (uint32_t)(16 * b + RPL * i) * half, 0, 2));
        const uint32_t row = 16 * b + l16 < rows ? 16 * b + l16 : rows - 1;
#pragma unroll
        for (int i = 0; i < NL; ++i) sz[u][i] = sp[i][row * ng];
      };
#pragma unroll
      for (int b = 0; b < D; ++b) load(b);
      // G128: columns 8 q .. 8 q + 7 of block 4 j + h at 4 j + q; otherwise 8 h .. 8 h + 7 of block i
      u32x4 xq[SL][WX];
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        const int blk = G128 ? (i & ~3) + h : i;
        const uint32_t col = 32u * (uint32_t)(b0 + blk) + (G128 ? 8u * (i & 3) : 8u * h);
        const uint32_t off = blk < nb ? (uint32_t)l16 * xrow + (uint32_t)sizeof(TX) * col : kPastEnd;
#pragma unroll
        for (int j = 0; j < WX; ++j)
          xq[i][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, off + 16 * j, 0, 0));
      }
      // every load of the slice is on its way before anything waits for one
      // (the compiler would sink the codes' loads to their use behind this)
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      bf16x8 xv[SL][NX];
#pragma unroll
      for (int i = 0; i < SL; ++i)
        if constexpr (NX == 1) xv[i][0] = order_as_codes(xq[i][0]);
        else split_as_codes(xq[i][0], xq[i][1], xv[i]);
      f32x4 xs[NS];
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        f32x4 low = zero;
        xs[i] = zero;
#pragma unroll
        for (int q = 0; q < SL / NS; ++q) {
          const bf16x8(&v)[NX] = xv[SL / NS * i + q];
          xs[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], ones, xs[i], 0, 0, 0);
#pragma unroll
          for (int p = 1; p < NX; ++p) low = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[p], ones, low, 0, 0, 0);
        }
        if constexpr (NX > 1) xs[i] += low;
      }
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int u = b % D;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int t = RPL * i + lr;
          place[SL * t + (lp ^ (SL == 16 ? t : (t >> 1) & 7))] = cv[u][i];
        }
        __builtin_amdgcn_wave_barrier();
        uint32_t words[SL];
        const int sw = SL == 16 ? l16 : (l16 >> 1) & 7;
        if constexpr (G128) {
#pragma unroll
          for (int j = 0; j < SL / 4; ++j) {
            const u32x4 v = place[SL * l16 + ((4 * j + h) ^ sw)];
#pragma unroll
            for (int q = 0; q < 4; ++q) words[4 * j + q] = v[q];
          }
        } else {
#pragma unroll
          for (int c = 0; c < SL; ++c) words[c] = ((const uint32_t*)(place + SL * l16 + (c ^ sw)))[h];
        }
        __builtin_amdgcn_wave_barrier();
        float val[2 * NS];  // scales, then zero-points
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          uint32_t v[4];
          spread4(sz[u][i], v);
#pragma unroll
          for (int k = 0; k < 4; ++k) val[4 * i + k] = scale_value<TS>(v[k]);
        }
        // the lower parts' sums are small and rounded finely; added once, they
        // cost the upper part's one rounding
        f32x4 d[NS], low[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) d[i] = low[i] = zero;
#pragma unroll
        for (int q = 0; q < SL / NS; ++q)
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const bf16x8 c = codes16(words[SL / NS * i + q], nk);
            const bf16x8(&v)[NX] = xv[SL / NS * i + q];
            d[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[0], c, d[i], 0, 0, 0);
#pragma unroll
            for (int p = 1; p < NX; ++p) low[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[p], c, low[i], 0, 0, 0);
          }
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          if constexpr (NX > 1) d[i] += low[i];
          const float sc = val[i], nz = -sc * (16.0f + val[NS + i]);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[b][r] = fmaf(sc, d[i][r], fmaf(nz, xs[i][r], acc[b][r]));
        }
        if (b + D < RB) {
          load(b + D);
          asm volatile("" ::: "memory");
        }
      }
    }

    // lane holds tokens 4 h + r (r = 0..3) of weight row 16 b + l16
    __syncthreads();  // the regrouping places overlap the sums'
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (4 * h + r < tokens) {
#pragma unroll
        for (int b = 0; b < RB; ++b) part[((w * 16 + 4 * h + r) * RB + b) * 16 + l16] = acc[b][r];
      }
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * RB * tokens; o += blockDim.x) {
      float v = 0.0f;
#pragma unroll 8
      for (int i = 0; i < nw; ++i) v += part[i * 256 * RB + o];
      const int64_t n = n0 + o % (16 * RB), m = r0 + o / (16 * RB);
      if (n < N) {
        if constexpr (sizeof(TY) == 4) y[m * N + n] = v;
        else y[m * N + n] = (TY)f32_to_bf16_bits(v);
      }
    }
    if (tile + gridDim.x < tiles) __syncthreads();  // the next tile writes part again
  }
}

// At most 8 waves, each taking the same number of slices of sl blocks.
static int grouped_rows_waves(int64_t k, int sl) {
  const int64_t slices = (k / 32 + sl - 1) / sl;
  const int64_t per = (slices + 7) / 8;
  return (int)((slices + per - 1) / per);
}

template <typename TX, typename TS, typename TY, bool G128, int SL, int RB>
static hipError_t gr_rb(const TX* x, int64_t t, int64_t k, const int* offsets, int experts, const uint8_t* packed,
                        const void* scales, const void* zeros, int64_t n, int g, void* y, hipStream_t st) {
  const int64_t tiles_n = (n + 16 * RB - 1) / (16 * RB), tiles = grouped_max_tiles(t, experts, 16) * tiles_n;
  const int nw = grouped_rows_waves(k, SL);
  const size_t sums = (size_t)nw * 1024 * RB, places = (size_t)nw * 256 * SL;
  const dim3 grid((unsigned)(tiles < kGRowsGrid ? tiles : kGRowsGrid));
  k_w4a16_grouped_rows<TX, TS, TY, G128, SL, RB><<<grid, 64 * nw, sums > places ? sums : places, st>>>(
      x, t, k, offsets, experts, packed, scales, zeros, n, g, (TY*)y, (uint32_t)tiles_n, tiles);
  return hipGetLastError();
}

template <typename TX, typename TS, typename TY, bool G128>
static hipError_t gr_size(const TX* x, int64_t t, int64_t k, const int* offsets, int experts, const uint8_t* packed,
                          const void* scales, const void* zeros, int64_t n, int g, void* y, hipStream_t st) {
  // The three parts of float32 x take the registers of twice the columns, and
  // so do the scales and sums of groups that end at any block, which leave none
  // for six blocks of rows, and with float32 x for one only (four: 8 rows of 8
  // experts [11008, 4096] 155 us against 131).  (Groups of 64: one block a workgroup and 16 waves
  // took 8 rows of 8 experts [11008, 4096] 100 us, one and 8 waves 61, up to
  // four 56; groups of 32, 16 rows of 64 experts [2048, 2048] 22 and 17.)
  constexpr int SL = G128 && sizeof(TX) == 2 ? 16 : 8, MAX = G128 ? 6 : sizeof(TX) == 2 ? 4 : 1;
  if constexpr (MAX > 1) {
    switch (rows_per_group<MAX>(grouped_max_tiles(t, experts, 16), (n + 15) / 16)) {
      case 1: break;
      case 2: return gr_rb<TX, TS, TY, G128, SL, 2>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
      case 4: return gr_rb<TX, TS, TY, G128, SL, 4>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
      default:
        if constexpr (MAX == 6) return gr_rb<TX, TS, TY, G128, SL, 6>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
    }
  }
  return gr_rb<TX, TS, TY, G128, SL, 1>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
}

template <typename TX, typename TS, typename TY>
static hipError_t gr_pick(const void* xv, int64_t t, int64_t k, const int* offsets, int experts, const uint8_t* packed,
                          const void* scales, const void* zeros, int64_t n, int g, void* y, hipStream_t st) {
  const TX* x = (const TX*)xv;
  if (g % 128 == 0) return gr_size<TX, TS, TY, true>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  return gr_size<TX, TS, TY, false>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
}

template <typename TX>
static hipError_t gr_types(const void* x, int64_t t, int64_t k, const int* offsets, int experts, const uint8_t* packed,
                           const void* scales, const void* zeros, int sz_dtype, int64_t n, int g, void* y, int y_dtype,
                           hipStream_t st) {
  if (sz_dtype == W4_F16) {
    if (y_dtype == W4_F32)
      return gr_pick<TX, _Float16, float>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
    return gr_pick<TX, _Float16, uint16_t>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  }
  if (y_dtype == W4_F32)
    return gr_pick<TX, float, float>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  return gr_pick<TX, float, uint16_t>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
}

hipError_t launch_w4a16_grouped_rows(const void* x, int x_dtype, int64_t t, int64_t k, const int* offsets, int experts,
                                     const uint8_t* packed, const void* scales, const void* zeros, int sz_dtype,
                                     int64_t n, int g, void* y, int y_dtype, hipStream_t st) {
  if (x_dtype == W4_F32)
    return gr_types<float>(x, t, k, offsets, experts, packed, scales, zeros, sz_dtype, n, g, y, y_dtype, st);
  return gr_types<uint16_t>(x, t, k, offsets, experts, packed, scales, zeros, sz_dtype, n, g, y, y_dtype, st);
}

}  // namespace w4
