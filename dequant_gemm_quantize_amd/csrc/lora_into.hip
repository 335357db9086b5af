// Into the low rank: for the rows of a segment with adapter l,
//   low[m, r] = scaling[l] sum_d x[m, d] W[l, r, d]     (x into A [L, R, K]), or
//   low[m, r] = scaling[l] sum_d x[m, d] W[l, d, r]     (dy into B [L, N, R]),
// float32, on v_mfma_f32_16x16x32_bf16: bf16 values as they are, float32 ones as the
// exact sum of three bf16 values.  Rows of no adapter are left as they were.
//
// A workgroup has 16 MT rows of one segment and RT ranks; its waves go through D in
// turn, 128 values at a time, and add their sums through LDS.  Few rows take
// four ranks a workgroup, so that more CUs read the adapter's rows.
#include "lora.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int kIntoWaves = 8;
constexpr int64_t kIntoGrid = 1 << 20;  // workgroups; more tiles than that loop

// The adapter's values at rank r, 8 of them along D from d on.  DOWN: [R, D] (D % 32 == 0), otherwise [D, R].
template <bool DOWN, typename TW>
__device__ __forceinline__ void adapter8(const TW* w, int64_t d, int64_t D, int r, int R, bool real,
                                         bf16x8 (&out)[Parts<TW>::n]) {
  if constexpr (DOWN) {
    if (real && d < D) {
      load8(w + (int64_t)r * D + d, out);
      return;
    }
#pragma unroll
    for (int p = 0; p < Parts<TW>::n; ++p) out[p] = zero8();
  } else {
    TW v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = real && d + i < D ? w[(d + i) * R + r] : (TW)0;
    pack8(v, out);
  }
}

}  // namespace

template <bool DOWN, int MT, int RT, typename TX, typename TW>
__global__ __launch_bounds__(64 * kIntoWaves) void k_lora_into(
    const TX* __restrict__ x, int64_t M, int64_t D, const TW* __restrict__ weights, int count, int R,
    const float* __restrict__ scaling, const int* __restrict__ offsets, const int* __restrict__ which, int segments,
    float* __restrict__ low, uint32_t rblocks, int64_t tiles, int wide) {
  __shared__ float part[kIntoWaves][16 * MT][RT];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, h = lane >> 4;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    GroupTile gt;
    if (!find_group_tile(offsets, segments, (int)M, 16 * MT, rblocks, tile, lane, gt)) return;
    const int ad = which[gt.expert];
    if (ad < 0 || ad >= count) continue;
    const int rb = (int)(gt.tile % rblocks) * RT;
    const int64_t m0 = gt.row0 + (int64_t)16 * MT * (gt.tile / rblocks);
    const int64_t left = gt.row0 + gt.rows - m0;
    const int rows = (int)(left < 16 * MT ? left : 16 * MT);
    const TW* wl = weights + (int64_t)ad * R * D;
    const int r = rb + l16;
    const bool rank = l16 < RT && r < R;

    f32x4 acc[MT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t][0] = acc[t][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t d0 = 128 * w; d0 < D; d0 += 128 * kIntoWaves) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t d = d0 + 32 * q + 8 * h;
        bf16x8 b[Parts<TW>::n];
        adapter8<DOWN>(wl, d, D, r, R, rank, b);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          bf16x8 a[Parts<TX>::n];
          const int row = 16 * t + l16;
          row8(x + (m0 + (row < rows ? row : 0)) * D, d, D, row < rows, wide, a);
          mfma_parts(a, b, acc[t]);
        }
      }
    }
    // lane holds rows 4 h + e of rank l16
    if (l16 < RT) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[w][16 * t + 4 * h + e][l16] = acc[t][0][e] + acc[t][1][e];
    }
    __syncthreads();
    const float c = scaling[ad];
    for (int o = threadIdx.x; o < rows * RT; o += 64 * kIntoWaves) {
      const int row = o / RT, q = o % RT;
      if (rb + q >= R) continue;
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kIntoWaves; ++i) v += part[i][row][q];
      low[(m0 + row) * R + rb + q] = c * v;
    }
    __syncthreads();  // the next tile writes part again
  }
}

template <bool DOWN, int MT, int RT, typename TX, typename TW>
static hipError_t into_go(const LoraInto& a, hipStream_t st) {
  const int64_t rblocks = (a.rank + RT - 1) / RT;
  const int64_t tiles = grouped_max_tiles(a.m, a.segments, 16 * MT) * rblocks;
  k_lora_into<DOWN, MT, RT><<<dim3((unsigned)(tiles < kIntoGrid ? tiles : kIntoGrid)), 64 * kIntoWaves, 0, st>>>(
      (const TX*)a.x, a.m, a.d, (const TW*)a.weights, (int)a.count, a.rank, a.scaling, a.offsets, a.which,
      (int)a.segments, a.low, (uint32_t)rblocks, tiles, a.d * (int64_t)sizeof(TX) % 16 == 0);
  return hipGetLastError();
}

template <bool DOWN, typename TX, typename TW>
static hipError_t into_size(const LoraInto& a, hipStream_t st) {
  if (a.m <= 16 * a.segments) return into_go<DOWN, 1, 4, TX, TW>(a, st);
  return into_go<DOWN, 1, 16, TX, TW>(a, st);
}

template <bool DOWN>
static hipError_t into_types(const LoraInto& a, hipStream_t st) {
  if (a.x_dtype == W4_F32)
    return a.w_dtype == W4_F32 ? into_size<DOWN, float, float>(a, st) : into_size<DOWN, float, uint16_t>(a, st);
  return a.w_dtype == W4_F32 ? into_size<DOWN, uint16_t, float>(a, st) : into_size<DOWN, uint16_t, uint16_t>(a, st);
}

hipError_t launch_lora_into(const LoraInto& a, hipStream_t st) {
  return a.down ? into_types<true>(a, st) : into_types<false>(a, st);
}

}  // namespace w4
