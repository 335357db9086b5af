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
#include "w4a16_grouped_rows.h"

namespace w4 {

template <typename TX>
static hipError_t gr_types(const void* x, int64_t t, int64_t k, const int* offsets, int experts, const uint8_t* packed,
                           const void* scales, const void* zeros, int sz_dtype, int64_t n, int g, void* y, int y_dtype,
                           hipStream_t st) {
  if (sz_dtype == W4_F16) {
    if (y_dtype == W4_F32)
      return gr_pick<TX, _Float16, float>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, NoAdapters{}, st);
    return gr_pick<TX, _Float16, uint16_t>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, NoAdapters{}, st);
  }
  if (y_dtype == W4_F32)
    return gr_pick<TX, float, float>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, NoAdapters{}, st);
  return gr_pick<TX, float, uint16_t>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, NoAdapters{}, st);
}

hipError_t launch_w4a16_grouped_rows(const void* x, int x_dtype, int64_t t, int64_t k, const int* offsets, int experts,
                                     const uint8_t* packed, const void* scales, const void* zeros, int sz_dtype,
                                     int64_t n, int g, void* y, int y_dtype, hipStream_t st) {
  if (x_dtype == W4_F32)
    return gr_types<float>(x, t, k, offsets, experts, packed, scales, zeros, sz_dtype, n, g, y, y_dtype, st);
  return gr_types<uint16_t>(x, t, k, offsets, experts, packed, scales, zeros, sz_dtype, n, g, y, y_dtype, st);
}

}  // namespace w4
