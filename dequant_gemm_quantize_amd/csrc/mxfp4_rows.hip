// MXFP4 product for few rows per weight matrix (decode), dense or by expert:
//   y[m, n] = sum over blocks b of 2^(xs + ws - 254) * sum_{k in b} xv wv
// on v_mfma_scale_f32_16x16x128_f8f6f4, whose lane (l16, h) holds one block of
// 32 columns (16 bytes) of row l16 of each operand and that block's scale, so
// the scales are applied inside the instruction and the sums stay in float32.
//
// Bound by the weight bytes.  A workgroup goes through RB blocks of 16 weight
// rows, all of K, for up to 16 MT token rows.  Its waves have a 512-column slice
// of K each (or take such slices in turn), keep x of it in registers for all
// the blocks, and add their sums through LDS at the end.  The weights of the
// next block are in flight while one is computed.  One block a workgroup
// was slower: the launch then has so many waves that starting them (about 13
// cycles a wave on each XCD) takes longer than reading the weights.
//
// Measured (a call's share of a replayed graph of calls, weights rotated; the
// kernel alone takes 1 - 2 us less): one row times [11008, 4096] 7.4 - 8.0 us (3.1
// TB/s), [28672, 8192] 26.2 us (4.8 TB/s), [8192, 28672] 23.3 us (5.4 TB/s), 16 rows
// of 64 experts [2048, 2048] 8.9 us of which the bytes of the experts with rows
// take 6.2.  More token
// rows cost time of their own, since every workgroup reads x of its slices
// (64 rows times [4096, 11008] 19 us against 6.6 for one).  16 waves in place of 8
// where a workgroup has one block: 7.2 us against 6.6 for [4096, 11008].
//
// Any K that is a multiple of 32: the last, partial slice is loaded block by
// block, and blocks past K count as zero.
#include "grouped.h"
#include "w4_common.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int kMxSlice = 512;   // columns of K per wave and turn
constexpr int kMxMaxGrid = 1 << 20;  // workgroups; more tiles than that loop

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef u32x4 u32x4_u __attribute__((aligned(1)));  // scale rows start at any byte

__device__ __forceinline__ i32x8 fp4_operand(u32x4 v) {
  return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

}  // namespace

template <typename TY, bool GROUPED, int MT, int RB>
__global__ __launch_bounds__(512, 2) void k_mx_rows(const uint8_t* __restrict__ xq, const uint8_t* __restrict__ xs,
                                                    int64_t M, int64_t K, const uint8_t* __restrict__ packed,
                                                    const uint8_t* __restrict__ scales, int64_t N,
                                                    void* __restrict__ y, const int* __restrict__ offsets, int experts,
                                                    uint32_t tiles_n, int64_t tiles) {
  // [waves][16 MT tokens][16 RB rows] sums; before them 4 KB a wave to regroup weights
  extern __shared__ __attribute__((aligned(16))) float part[];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6;
  const int l16 = lane & 15, h = lane >> 4;
  const int64_t kb = K / 32, half = K / 2;
  const int full = (int)(K / kMxSlice), slices = (int)((K + kMxSlice - 1) / kMxSlice);
  // blocks whose weights are held at a time (three or four were slower: one row
  // times [28672, 8192] 26.2, 27.2 and 28.4 us)
  constexpr int D = RB < 2 ? 1 : 2;

  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    int64_t r0, rend, n0;  // token rows r0 .. rend - 1 at most 16 MT of them, weight rows from n0
    const uint8_t* wp = packed;
    const uint8_t* sp = scales;
    if constexpr (GROUPED) {
      GroupTile g;
      if (!find_group_tile(offsets, experts, (int)M, 16 * MT, tiles_n, tile, lane, g)) break;
      n0 = (int64_t)16 * RB * (g.tile % tiles_n);
      r0 = g.row0 + (int64_t)16 * MT * (g.tile / tiles_n);
      rend = g.row0 + g.rows;
      wp += (int64_t)g.expert * N * half;
      sp += (int64_t)g.expert * N * kb;
    } else {
      n0 = (tile % tiles_n) * (16 * RB);
      r0 = (tile / tiles_n) * (16 * MT);
      rend = M;
    }
    if (rend > r0 + 16 * MT) rend = r0 + 16 * MT;
    const int blocks = (int)((rend - r0 + 15) / 16);  // token blocks with a row
    const int rows = (int)(N - n0 < 16 * RB ? N - n0 : 16 * RB);
    wp += n0 * half;
    sp += n0 * kb;

    // rows past the end repeat the last one and are never stored
    const uint8_t* xl[MT];
    const uint8_t* xsl[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t row = r0 + 16 * t + l16 < rend ? r0 + 16 * t + l16 : rend - 1;
      xl[t] = xq + row * half + 16 * h;
      xsl[t] = xs + row * kb;
    }
    f32x4 acc[RB][MT];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[b][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int sl = w; sl < full; sl += nw) {
      u32x4 wv[D][4], wsv[D];
      auto load = [&](int b) {
        const uint8_t* base = wp + (int64_t)sl * 256 + 16 * l16;  // 256-byte runs of rows 16 b + 4 j + h
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 16 * b + 4 * j + h < rows ? 16 * b + 4 * j + h : rows - 1;
          wv[b % D][j] = ldg_nt((const u32x4*)(base + t * half));
        }
        wsv[b % D] = *(const u32x4_u*)(sp + (16 * b + l16 < rows ? 16 * b + l16 : rows - 1) * kb + 16 * sl);
      };
#pragma unroll
      for (int b = 0; b < D; ++b) load(b);
      u32x4 xv[MT][4], xsv[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (t > 0 && t >= blocks) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[t][j] = *(const u32x4*)(xl[t] + (int64_t)sl * 256 + 64 * j);
        xsv[t] = *(const u32x4_u*)(xsl[t] + 16 * sl);
      }
      // every load of the slice is on its way before anything waits for one
      asm volatile("" ::: "memory");
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        __builtin_amdgcn_sched_barrier(0);
        u32x4(&v)[4] = wv[b % D];
        const u32x4 vs = wsv[b % D];
        regroup_runs((u32x4*)part + 256 * w, lane, v);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (t > 0 && t >= blocks) break;
#pragma unroll
          for (int j = 0; j < 4; ++j)  // block 4 j + h: byte h of scale word j
            acc[b][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                fp4_operand(xv[t][j]), fp4_operand(v[j]), acc[b][t], 4, 4, 0, (int)(xsv[t][j] >> (8 * h)), 0,
                (int)(vs[j] >> (8 * h)));
        }
        if (b + D < RB) {
          load(b + D);
          asm volatile("" ::: "memory");
        }
      }
    }
    if (full < slices && w == full % nw) {  // the partial slice
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t blk = (int64_t)16 * full + 4 * j + h;
        if ((int64_t)16 * full + 4 * j >= kb) break;  // the same in every lane
        const bool in = blk < kb;
        u32x4 wv[RB];
        uint32_t wsv[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          wv[b] = u32x4{0, 0, 0, 0};
          wsv[b] = 0;
          if (in) {
            const int row = 16 * b + l16 < rows ? 16 * b + l16 : rows - 1;
            wv[b] = *(const u32x4*)(wp + row * half + (int64_t)full * 256 + 64 * j + 16 * h);
            wsv[b] = sp[row * kb + blk];
          }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (t > 0 && t >= blocks) break;
          u32x4 xv = {0, 0, 0, 0};
          uint32_t xsv = 0;
          if (in) {
            xv = *(const u32x4*)(xl[t] + (int64_t)full * 256 + 64 * j);
            xsv = xsl[t][blk];
          }
#pragma unroll
          for (int b = 0; b < RB; ++b)
            acc[b][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(xv), fp4_operand(wv[b]), acc[b][t], 4,
                                                                        4, 0, (int)xsv, 0, (int)wsv[b]);
        }
      }
    }

    // lane holds tokens 16 t + 4 h + r (r = 0..3) of weight row 16 b + l16
    __syncthreads();  // the regrouping places overlap the sums'
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + 16 * t + 4 * h + r < rend) {
#pragma unroll
          for (int b = 0; b < RB; ++b)
            part[((w * 16 * MT + 16 * t + 4 * h + r) * RB + b) * 16 + l16] = acc[b][t][r];
        }
    __syncthreads();
    const int outs = 16 * RB * (int)(rend - r0);
    for (int o = threadIdx.x; o < outs; o += blockDim.x) {
      float s = 0.0f;
#pragma unroll 8
      for (int v = 0; v < nw; ++v) s += part[v * 256 * MT * RB + o];
      const int64_t n = n0 + o % (16 * RB), m = r0 + o / (16 * RB);
      if (n < N) {
        if constexpr (sizeof(TY) == 4)
          ((float*)y)[m * N + n] = s;
        else
          ((uint16_t*)y)[m * N + n] = (uint16_t)f32_to_bf16_bits(s);
      }
    }
    if (tile + gridDim.x < tiles) __syncthreads();  // the next tile writes part again
  }
}

// At most 8 waves, each taking the same number of slices.
static int mx_rows_waves(int64_t k) {
  const int64_t slices = (k + kMxSlice - 1) / kMxSlice;
  const int64_t per = (slices + 7) / 8;
  return (int)((slices + per - 1) / per);
}

template <typename TY, bool GROUPED, int MT, int RB>
static void mx_rows_go(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                       const uint8_t* scales, int64_t n, void* y, const int* offsets, int experts, hipStream_t st) {
  const int64_t tiles_n = (n + 16 * RB - 1) / (16 * RB);
  const int64_t tiles_m = GROUPED ? grouped_max_tiles(m, experts, 16 * MT) : (m + 16 * MT - 1) / (16 * MT);
  const int64_t tiles = tiles_m * tiles_n;
  const int nw = mx_rows_waves(k);
  const size_t sums = (size_t)nw * 256 * MT * RB * sizeof(float), places = (size_t)nw * 4096;
  const dim3 grid((unsigned)(tiles < kMxMaxGrid ? tiles : kMxMaxGrid));
  k_mx_rows<TY, GROUPED, MT, RB><<<grid, 64 * nw, sums > places ? sums : places, st>>>(
      xq, xs, m, k, packed, scales, n, y, offsets, experts, (uint32_t)tiles_n, tiles);
}

// Blocks of 16 weight rows a workgroup, by the rounds of workgroups on 256 CUs:
// a workgroup's start, first loads and sums cost about as much as three blocks.
template <typename TY, bool GROUPED, int MT>
static void mx_rows_rb(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                       const uint8_t* scales, int64_t n, void* y, const int* offsets, int experts, hipStream_t st) {
  const int64_t tiles_m = GROUPED ? grouped_max_tiles(m, experts, 16 * MT) : (m + 16 * MT - 1) / (16 * MT);
  switch (rows_per_group<MT == 4 ? 2 : MT == 2 ? 4 : 6>(tiles_m, (n + 15) / 16)) {
    case 1: return mx_rows_go<TY, GROUPED, MT, 1>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
    case 2: return mx_rows_go<TY, GROUPED, MT, 2>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
    case 4:
      if constexpr (MT < 4) return mx_rows_go<TY, GROUPED, MT, 4>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
      return;
    default:
      if constexpr (MT == 1) return mx_rows_go<TY, GROUPED, MT, 6>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  }
}

template <typename TY>
static hipError_t mx_rows_pick(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                               const uint8_t* scales, int64_t n, void* y, const int* offsets, int experts,
                               hipStream_t st) {
  if (offsets != nullptr) {
    if (m <= 8 * (int64_t)experts) mx_rows_rb<TY, true, 1>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
    else mx_rows_rb<TY, true, 4>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  } else if (m <= 16) mx_rows_rb<TY, false, 1>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  else if (m <= 32) mx_rows_rb<TY, false, 2>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  else mx_rows_rb<TY, false, 4>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  return hipGetLastError();
}

hipError_t launch_mx_rows(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                          const uint8_t* scales, int64_t n, void* y, int y_dtype, const int* offsets, int experts,
                          hipStream_t st) {
  if (y_dtype == W4_F32) return mx_rows_pick<float>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  return mx_rows_pick<__bf16>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
}

}  // namespace w4
