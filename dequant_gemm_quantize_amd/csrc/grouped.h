// Rows grouped by expert: which rows and which expert a workgroup's tile has.
//
// offsets[0 .. E] (device memory, int32) bound the experts' rows: expert e
// owns rows offsets[e] .. offsets[e + 1] - 1.  The host does not know them,
// so a launch covers the most tiles that any offsets can need and each
// workgroup finds its own tile from the offsets.  Every value read is clamped
// to [0, T] and a falling pair owns no row, so no offsets lead out of bounds.
#pragma once

#include "w4_common.h"

namespace w4 {

// The most tiles of bm rows that T rows of E experts can need: every expert
// with rows adds at most one partial tile.
inline int64_t grouped_max_tiles(int64_t t, int64_t experts, int bm) {
  const int64_t some = experts < t ? experts : t;
  return (t + some * (bm - 1)) / bm;
}

struct GroupTile {
  int expert;
  int64_t row0;  // the expert's first row
  int rows;      // the expert's rows
  uint32_t tile;  // the tile's number within the expert
};

// Rows of experts base .. base + 63, one a lane (0 past the last expert).
__device__ __forceinline__ int group_rows(const int* offsets, int experts, int t, int base, int lane,
                                          int& row0) {
  row0 = 0;
  if (base + lane >= experts) return 0;
  int a = offsets[base + lane], b = offsets[base + lane + 1];
  a = a < 0 ? 0 : a > t ? t : a;
  b = b < 0 ? 0 : b > t ? t : b;
  row0 = a;
  return b > a ? b - a : 0;
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t u = __shfl_up(v, o, kWave);
    if (lane >= o) v += u;
  }
  return v;
}

// Tiles of bm rows that the offsets need; the same in every lane.
__device__ __forceinline__ int64_t grouped_tiles(const int* offsets, int experts, int t, int bm, int lane) {
  int64_t total = 0;
  for (int base = 0; base < experts; base += kWave) {
    int row0;
    const int rows = group_rows(offsets, experts, t, base, lane, row0);
    int64_t n = (rows + bm - 1) / bm;
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) n += __shfl_xor(n, o, kWave);
    total += n;
  }
  return total;
}

// Finds tile `want` of the list in which every expert has its tiles of bm
// rows times `width` tiles; tile is then the number within the expert's
// tiles x width.  False when the list is shorter.  All 64 lanes call it.
__device__ __forceinline__ bool find_group_tile(const int* offsets, int experts, int t, int bm, int64_t width,
                                                int64_t want, int lane, GroupTile& g) {
  int64_t before = 0;
  for (int base = 0; base < experts; base += kWave) {
    int row0;
    const int rows = group_rows(offsets, experts, t, base, lane, row0);
    const int64_t mine = (int64_t)((rows + bm - 1) / bm) * width;
    const int64_t upto = before + wave_scan(mine, lane);
    const uint64_t past = __ballot(upto > want);
    if (past != 0) {
      const int f = __builtin_ctzll(past);
      g.expert = __builtin_amdgcn_readfirstlane(base + f);
      g.row0 = __builtin_amdgcn_readfirstlane(__shfl(row0, f, kWave));
      g.rows = __builtin_amdgcn_readfirstlane(__shfl(rows, f, kWave));
      // the launch has fewer than 2^31 tiles, and want is one of them
      g.tile = (uint32_t)__builtin_amdgcn_readfirstlane((int)(want - __shfl(upto - mine, f, kWave)));
      return true;
    }
    before = __shfl(upto, kWave - 1, kWave);
  }
  return false;
}

}  // namespace w4
