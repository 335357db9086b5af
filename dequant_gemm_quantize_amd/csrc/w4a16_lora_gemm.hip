// W4A16 product with the adapters of its rows' requests, for many rows of bf16 x:
//   y[m, n] = sum over groups j of s (sum_{k in j} x q - zp sum_{k in j} x) + sum_r low[m, r] B[l(m), n, r]
// The kernel is the many-row product's by expert, with one expert, so no weight is
// rounded whatever the types.  The low-rank part joins the sums before they are stored.
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
  const Adapters ad{lo.low,           lo.out,        lo.offsets, lo.which, (int)lo.segments,
                    (int)lo.count, lo.rank, lo.dtype == W4_F32, lo.parts, lo.whole};
  if (a.sz_dtype == W4_F16)
    return a.y_dtype == W4_F32 ? lg_pick<_Float16, float>(a, ad, st) : lg_pick<_Float16, __bf16>(a, ad, st);
  return a.y_dtype == W4_F32 ? lg_pick<float, float>(a, ad, st) : lg_pick<float, __bf16>(a, ad, st);
}

}  // namespace w4
