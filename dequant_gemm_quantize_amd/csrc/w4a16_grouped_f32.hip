// W4A16 product by expert with float32 x (small layers and checks): rows of x
// grouped by expert, group-wise INT4 weights of each expert,
//   y[t, n] = sum over groups j of s[e, n, j] * sum_{k in j} x[t, k] (q[e, n, k] - zp[e, n, j])
// for the expert e that owns row t, in float32 multiply-adds.
//
// A wave has 64 weight rows, one a lane, and 4 token rows, whose x is the same
// address in every lane; each lane reads its row in 16-byte pieces of 32
// codes, which lie in one group.  q - zp is an exact small integer, and the
// group's scale multiplies the float32 sum of 32 columns.
#include "grouped.h"
#include "w4_common.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int kF32Grid = 1 << 20;  // workgroups; more tiles than that loop

}  // namespace

template <typename TS, typename TY>
__global__ __launch_bounds__(256) void k_w4a16_grouped_f32(const float* __restrict__ x, int64_t T, int64_t K,
                                                           const int* __restrict__ offsets, int experts,
                                                           const uint8_t* __restrict__ packed,
                                                           const void* __restrict__ scales,
                                                           const void* __restrict__ zeros, int64_t N, int g,
                                                           TY* __restrict__ y, uint32_t tiles_n, int64_t tiles) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t ng = K / g;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    GroupTile gt;
    if (!find_group_tile(offsets, experts, (int)T, 16, tiles_n, tile, lane, gt)) break;
    const int64_t n = (int64_t)64 * (gt.tile % tiles_n) + lane;
    const int64_t r0 = gt.row0 + (int64_t)16 * (gt.tile / tiles_n) + 4 * w;
    const int64_t rend = gt.row0 + gt.rows;
    if (r0 >= rend) continue;
    const int64_t row = (int64_t)gt.expert * N + (n < N ? n : N - 1);
    const u32x4* wp = (const u32x4*)(packed + row * (K / 2));
    const float* xp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xp[i] = x + (r0 + i < rend ? r0 + i : rend - 1) * K;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t b = 0; b < K / 32; ++b) {
      const u32x4 p = wp[b];
      const int64_t gi = row * ng + b / (g / 32);
      const float s = ScaleT<TS>::load(scales, gi), z = ScaleT<TS>::load(zeros, gi);
      float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float q = (float)((p[j >> 3] >> (4 * (j & 7))) & 15u) - z;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = fmaf(xp[i][32 * b + j], q, sum[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(s, sum[i], acc[i]);
    }
    if (n < N) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r0 + i < rend) {
          if constexpr (sizeof(TY) == 4) y[(r0 + i) * N + n] = acc[i];
          else y[(r0 + i) * N + n] = (TY)f32_to_bf16_bits(acc[i]);
        }
    }
  }
}

template <typename TS, typename TY>
static hipError_t f32_go(const void* x, int64_t t, int64_t k, const int* offsets, int experts, const uint8_t* packed,
                         const void* scales, const void* zeros, int64_t n, int g, void* y, hipStream_t st) {
  const int64_t tiles_n = (n + 63) / 64, tiles = grouped_max_tiles(t, experts, 16) * tiles_n;
  const dim3 grid((unsigned)(tiles < kF32Grid ? tiles : kF32Grid));
  k_w4a16_grouped_f32<TS, TY><<<grid, 256, 0, st>>>((const float*)x, t, k, offsets, experts, packed, scales, zeros, n, g,
                                                   (TY*)y, (uint32_t)tiles_n, tiles);
  return hipGetLastError();
}

hipError_t launch_w4a16_grouped_f32(const void* x, int64_t t, int64_t k, const int* offsets, int experts,
                                    const uint8_t* packed, const void* scales, const void* zeros, int sz_dtype,
                                    int64_t n, int g, void* y, int y_dtype, hipStream_t st) {
  if (sz_dtype == W4_F16) {
    if (y_dtype == W4_F32)
      return f32_go<_Float16, float>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
    return f32_go<_Float16, uint16_t>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  }
  if (y_dtype == W4_F32) return f32_go<float, float>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
  return f32_go<float, uint16_t>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, st);
}

}  // namespace w4
