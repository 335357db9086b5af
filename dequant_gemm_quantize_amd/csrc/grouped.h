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

// Blocks of 16 weight rows that a workgroup of the few-row products goes
// through (1, 2, 4 or 6, at most MAX), for tiles_m row tiles of `blocks` such
// blocks: the fewest rounds of workgroups on 256 CUs, where a workgroup's
// start, first loads and final sums cost about as much as three blocks.
template <int MAX>
inline int rows_per_group(int64_t tiles_m, int64_t blocks) {
  int best = 1;
  int64_t least = 0;
  for (int rb = 1; rb <= MAX; rb += rb == 1 ? 1 : 2) {
    const int64_t groups = tiles_m * ((blocks + rb - 1) / rb), t = (groups + 255) / 256 * (rb + 3);
    if (rb == 1 || t < least) best = rb, least = t;
  }
  return best;
}

struct GroupTile {
  int expert;
  int64_t row0;  // the expert's first row
  int rows;      // the expert's rows
  uint32_t tile;  // the tile's number within the expert's tiles x width
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

// Inclusive sum over the lanes of a wave: shifts within rows of 16 lanes, then
// the rows' last lanes into the rows behind them (register moves of the vector
// unit, no trip through LDS).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast 15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast 31 into rows 2 and 3
  return v;
}

// Tiles of bm rows that the offsets need; the same in every lane.
__device__ __forceinline__ int64_t grouped_tiles(const int* offsets, int experts, int t, int bm, int lane) {
  int64_t total = 0;
  for (int base = 0; base < experts; base += kWave) {
    int row0;
    const int rows = group_rows(offsets, experts, t, base, lane, row0);
    total += __builtin_amdgcn_readlane(wave_scan((rows + bm - 1) / bm), kWave - 1);
  }
  return total;
}

// Finds tile `want` of the list in which every expert has its tiles of bm
// rows times `width` tiles.  False when the list is shorter.  All 64 lanes
// call it, with the same want.  (Rows are at most 2^24 and bm at least 16, so
// 64 experts' tiles fit 32 bits whatever the offsets hold; the launch has
// fewer than 2^31 tiles, and want is one of them.)
__device__ __forceinline__ bool find_group_tile(const int* offsets, int experts, int t, int bm, uint32_t width,
                                                int64_t want, int lane, GroupTile& g) {
  int64_t before = 0;
  for (int base = 0; base < experts; base += kWave) {
    int row0;
    const int rows = group_rows(offsets, experts, t, base, lane, row0);
    const int mine = (rows + bm - 1) / bm;
    const int upto = wave_scan(mine);
    const uint64_t past = __ballot((before + upto) * width > want);
    if (past != 0) {
      const int f = __builtin_ctzll(past);
      g.expert = base + f;
      g.row0 = __builtin_amdgcn_readlane(row0, f);
      g.rows = __builtin_amdgcn_readlane(rows, f);
      g.tile = (uint32_t)(want - (before + __builtin_amdgcn_readlane(upto - mine, f)) * width);
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  return false;
}

}  // namespace w4
