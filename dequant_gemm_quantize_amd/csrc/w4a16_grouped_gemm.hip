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
#include "w4a16_grouped_gemm.h"

namespace w4 {

// K % 64 == 0: whole steps; 128 rows of K bf16 stay below 2^31 bytes.
bool w4a16_grouped_gemm_fits(int64_t k) { return k % 64 == 0 && k <= ((int64_t)1 << 21); }

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
    return gg_go<GLarge, GLargeHalf, F, TS, TY>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, 1, 0, NoAdapters{}, st);
  return gg_go<GSmall, GSmallHalf, F, TS, TY>(x, t, k, offsets, experts, packed, scales, zeros, n, g, y, 1, 0, NoAdapters{}, st);
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
