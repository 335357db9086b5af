// W4A16 product with the adapters of its rows' requests, for many rows of bf16 x:
//   y[m, n] = sum over groups j of s (sum_{k in j} x q - zp sum_{k in j} x) + sum_r low[m, r] B[l(m), n, r]
// The kernel is the many-row product's by expert, with one expert, so no weight is
// rounded whatever the types.  The low-rank part joins the sums of the first part before they are stored,
// request by request.  One part where the tiles fill the CUs; otherwise the sum over K
// is split, and k_w4a16_sum (w4a16_lora.hip) adds the parts.
//
// Bound by the matrix cores and the vector instructions of conversions and scales, which wait for each other (matrix
// cores busy 41% of the time): 2048 rows of [11008, 4096], rank 64, 250 us, of which
// the low-rank part takes about 25; [4096, 4096], rank 16, 86; 128 rows of [4096, 11008] in nine parts 23 and their sum 6.
// (Tiles with weights rounded to bf16 took 236, 72 and 31, with two bf16 parts a weight for a float32 result 360.)
#include "w4a16_grouped_gemm.h"

namespace w4 {

template <int F, typename TS, typename TY>
static hipError_t lg_size(const TilesArgs& a, const Adapters& ad, hipStream_t st) {
  const uint16_t* x = (const uint16_t*)a.x;
  if (a.mi == 4)
    return gg_go<GLarge, GLargeHalf, F, TS, TY>(x, a.m, a.k, nullptr, 1, a.packed, a.scales, a.zeros, a.n, a.g, a.y,
                                                a.parts, a.steps, ad, st);
  return gg_go<GSmall, GSmallHalf, F, TS, TY>(x, a.m, a.k, nullptr, 1, a.packed, a.scales, a.zeros, a.n, a.g, a.y,
                                              a.parts, a.steps, ad, st);
}

template <typename TS, typename TY>
static hipError_t lg_pick(const TilesArgs& a, const Adapters& ad, hipStream_t st) {
  if (a.g % 128 == 0) return lg_size<8, TS, TY>(a, ad, st);
  if (a.g % 64 == 0) return lg_size<4, TS, TY>(a, ad, st);
  return lg_size<2, TS, TY>(a, ad, st);
}

hipError_t launch_w4a16_lora_gemm(const TilesArgs& a, const LoraOut& lo, hipStream_t st) {
  const Adapters ad = adapters_of(lo);
  if (a.sz_dtype == W4_F16)
    return a.y_dtype == W4_F32 ? lg_pick<_Float16, float>(a, ad, st) : lg_pick<_Float16, __bf16>(a, ad, st);
  return a.y_dtype == W4_F32 ? lg_pick<float, float>(a, ad, st) : lg_pick<float, __bf16>(a, ad, st);
}

}  // namespace w4
