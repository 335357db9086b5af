// Transposed W4A16 product of many rows: which kernel of w4a16_tiles.h a call takes.
#include "w4a16_tiles.h"

namespace w4 {

template <int MI, int PW, typename TS, typename TY>
static hipError_t tiles_subs(const TilesArgs& a, const Adapters& ad, hipStream_t st) {
  if (a.g % 128 == 0) return tiles_go<MI, PW, 1, TS, TY>(a, ad, st);
  return tiles_go<MI, PW, 4, TS, TY>(a, ad, st);
}

template <int MI, typename TS>
static hipError_t tiles_types(const TilesArgs& a, const Adapters& ad, hipStream_t st) {
  if (a.y_dtype == W4_F32) return tiles_subs<MI, 2, TS, float>(a, ad, st);
  return tiles_subs<MI, 2, TS, __bf16>(a, ad, st);
}

hipError_t launch_w4a16_tiles(const TilesArgs& a, const LoraOut& lo, hipStream_t st) {
  const Adapters ad = adapters_of(lo);
  if (a.pw == 3) return tiles_subs<2, 3, float, float>(a, ad, st);
  if (a.sz_dtype == W4_F16) return a.mi == 2 ? tiles_types<2, _Float16>(a, ad, st) : tiles_types<4, _Float16>(a, ad, st);
  return a.mi == 2 ? tiles_types<2, float>(a, ad, st) : tiles_types<4, float>(a, ad, st);
}

}  // namespace w4
