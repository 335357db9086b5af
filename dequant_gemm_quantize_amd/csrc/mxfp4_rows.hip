// MXFP4 product for few rows per weight matrix (decode), dense or by expert:
//   y[m, n] = sum over blocks b of 2^(xs + ws - 254) * sum_{k in b} xv wv
// on v_mfma_scale_f32_16x16x128_f8f6f4, whose lane (l16, h) holds one block of
// 32 columns (16 bytes) of row l16 of each operand and that block's scale, so
// the scales are applied inside the instruction and the sums stay in float32.
//
// Bound by the weight bytes.  A workgroup owns 16 weight rows and up to 16 MT
// token rows over all of K; its waves take 512-column slices of K in turn
// (slice w, w + waves, ...) and add their sums through LDS at the end.  The
// weights go from memory to the operand registers directly: a load covers 64
// contiguous bytes of each of 16 rows, four loads a whole slice.
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

template <typename TY, bool GROUPED, int MT>
__global__ __launch_bounds__(512) void k_mx_rows(const uint8_t* __restrict__ xq, const uint8_t* __restrict__ xs,
                                                 int64_t M, int64_t K, const uint8_t* __restrict__ packed,
                                                 const uint8_t* __restrict__ scales, int64_t N,
                                                 void* __restrict__ y, const int* __restrict__ offsets, int experts,
                                                 uint32_t tiles_n, int64_t tiles) {
  extern __shared__ __attribute__((aligned(16))) float part[];  // [waves][16 MT tokens][16 rows]
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6;
  const int l16 = lane & 15, h = lane >> 4;
  const int64_t kb = K / 32, half = K / 2;
  const int full = (int)(K / kMxSlice), slices = (int)((K + kMxSlice - 1) / kMxSlice);

  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    int64_t r0, rend, n0;  // token rows r0 .. rend - 1 at most 16 MT of them, weight rows from n0
    const uint8_t* wp = packed;
    const uint8_t* sp = scales;
    if constexpr (GROUPED) {
      GroupTile g;
      if (!find_group_tile(offsets, experts, (int)M, 16 * MT, tiles_n, tile, lane, g)) break;
      const uint32_t tm = g.tile / tiles_n;
      n0 = (int64_t)16 * (g.tile % tiles_n);
      r0 = g.row0 + (int64_t)16 * MT * tm;
      rend = g.row0 + g.rows;
      wp += (int64_t)g.expert * N * half;
      sp += (int64_t)g.expert * N * kb;
    } else {
      n0 = (tile % tiles_n) * 16;
      r0 = (tile / tiles_n) * (16 * MT);
      rend = M;
    }
    if (rend > r0 + 16 * MT) rend = r0 + 16 * MT;
    const int blocks = (int)((rend - r0 + 15) / 16);  // token blocks with a row

    // rows past the end repeat the last one and are never stored
    const int64_t wrow = n0 + l16 < N ? n0 + l16 : N - 1;
    const uint8_t* wl = wp + wrow * half + 16 * h;
    const uint8_t* ws = sp + wrow * kb;
    const uint8_t* xl[MT];
    const uint8_t* xsl[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t row = r0 + 16 * t + l16 < rend ? r0 + 16 * t + l16 : rend - 1;
      xl[t] = xq + row * half + 16 * h;
      xsl[t] = xs + row * kb;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int sl = w; sl < full; sl += nw) {
      u32x4 wv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) wv[j] = ldg_nt((const u32x4*)(wl + (int64_t)sl * 256 + 64 * j));
      const u32x4 wsv = *(const u32x4_u*)(ws + 16 * sl);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (t > 0 && t >= blocks) break;
        u32x4 xv[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[j] = *(const u32x4*)(xl[t] + (int64_t)sl * 256 + 64 * j);
        const u32x4 xsv = *(const u32x4_u*)(xsl[t] + 16 * sl);
#pragma unroll
        for (int j = 0; j < 4; ++j)  // block 4 j + h: byte h of scale word j
          acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(xv[j]), fp4_operand(wv[j]), acc[t], 4, 4,
                                                                   0, (int)(xsv[j] >> (8 * h)), 0,
                                                                   (int)(wsv[j] >> (8 * h)));
      }
    }
    if (full < slices && w == full % nw) {  // the partial slice
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t b = (int64_t)16 * full + 4 * j + h;
        if ((int64_t)16 * full + 4 * j >= kb) break;  // the same in every lane
        const bool in = b < kb;
        u32x4 wv = {0, 0, 0, 0};
        uint32_t wsv = 0;
        if (in) {
          wv = *(const u32x4*)(wl + (int64_t)full * 256 + 64 * j);
          wsv = ws[b];
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (t > 0 && t >= blocks) break;
          u32x4 xv = {0, 0, 0, 0};
          uint32_t xsv = 0;
          if (in) {
            xv = *(const u32x4*)(xl[t] + (int64_t)full * 256 + 64 * j);
            xsv = xsl[t][b];
          }
          acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(xv), fp4_operand(wv), acc[t], 4, 4, 0,
                                                                   (int)xsv, 0, (int)wsv);
        }
      }
    }

    // lane holds tokens 16 t + 4 h + r (r = 0..3) of weight row l16
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[(w * 16 * MT + 16 * t + 4 * h + r) * 16 + l16] = acc[t][r];
    __syncthreads();
    const int outs = 16 * (int)(rend - r0);
    for (int o = threadIdx.x; o < outs; o += blockDim.x) {
      float s = 0.0f;
      for (int v = 0; v < nw; ++v) s += part[v * 256 * MT + o];
      const int64_t n = n0 + (o & 15), m = r0 + (o >> 4);
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

template <typename TY, bool GROUPED, int MT>
static void mx_rows_go(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                       const uint8_t* scales, int64_t n, void* y, const int* offsets, int experts, hipStream_t st) {
  const int64_t tiles_n = (n + 15) / 16;
  const int64_t tiles_m = GROUPED ? grouped_max_tiles(m, experts, 16 * MT) : (m + 16 * MT - 1) / (16 * MT);
  const int64_t tiles = tiles_m * tiles_n;
  const int nw = mx_rows_waves(k);
  const dim3 grid((unsigned)(tiles < kMxMaxGrid ? tiles : kMxMaxGrid));
  k_mx_rows<TY, GROUPED, MT><<<grid, 64 * nw, (size_t)nw * 256 * MT * sizeof(float), st>>>(
      xq, xs, m, k, packed, scales, n, y, offsets, experts, (uint32_t)tiles_n, tiles);
}

template <typename TY>
static hipError_t mx_rows_pick(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                               const uint8_t* scales, int64_t n, void* y, const int* offsets, int experts,
                               hipStream_t st) {
  if (offsets != nullptr) mx_rows_go<TY, true, 4>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  else if (m <= 16) mx_rows_go<TY, false, 1>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  else if (m <= 32) mx_rows_go<TY, false, 2>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  else mx_rows_go<TY, false, 4>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  return hipGetLastError();
}

hipError_t launch_mx_rows(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                          const uint8_t* scales, int64_t n, void* y, int y_dtype, const int* offsets, int experts,
                          hipStream_t st) {
  if (y_dtype == W4_F32) return mx_rows_pick<float>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
  return mx_rows_pick<__bf16>(xq, xs, m, k, packed, scales, n, y, offsets, experts, st);
}

}  // namespace w4
