// Transposed W4A16 product for many rows: which kernel of w4a16_t_gemm.h a call takes.
#include "w4a16_t_gemm.h"

namespace w4 {

template <int MI, int PW, typename TS, typename TY>
static hipError_t tg_subs(const void* dy, int64_t m, int64_t k, const uint8_t* packed, const void* scales,
                          const void* zeros, int64_t n, int g, int parts, int steps, const Adapters& ad, void* dx,
                          hipStream_t st) {
  const uint16_t* d = (const uint16_t*)dy;
  if (g % 128 == 0)
    return tg_go<MI, PW, 1, TS, TY>(d, m, k, packed, scales, zeros, n, g, parts, steps, ad, (TY*)dx, st);
  return tg_go<MI, PW, 4, TS, TY>(d, m, k, packed, scales, zeros, n, g, parts, steps, ad, (TY*)dx, st);
}

template <typename TS>
static hipError_t tg_types(const void* dy, int64_t m, int64_t k, const uint8_t* packed, const void* scales,
                           const void* zeros, int64_t n, int g, void* dx, int dx_dtype, int mi, int pw, int parts,
                           int steps, const Adapters& ad, hipStream_t st) {
  if (pw == 1) {
    if (dx_dtype == W4_F32)
      return mi == 2 ? tg_subs<2, 1, TS, float>(dy, m, k, packed, scales, zeros, n, g, parts, steps, ad, dx, st)
                     : tg_subs<4, 1, TS, float>(dy, m, k, packed, scales, zeros, n, g, parts, steps, ad, dx, st);
    return mi == 2 ? tg_subs<2, 1, TS, __bf16>(dy, m, k, packed, scales, zeros, n, g, parts, steps, ad, dx, st)
                   : tg_subs<4, 1, TS, __bf16>(dy, m, k, packed, scales, zeros, n, g, parts, steps, ad, dx, st);
  }
  if constexpr (sizeof(TS) == 2)
    return mi == 2 ? tg_subs<2, 2, TS, float>(dy, m, k, packed, scales, zeros, n, g, parts, steps, ad, dx, st)
                   : tg_subs<4, 2, TS, float>(dy, m, k, packed, scales, zeros, n, g, parts, steps, ad, dx, st);
  else
    return tg_subs<2, 3, TS, float>(dy, m, k, packed, scales, zeros, n, g, parts, steps, ad, dx, st);
}

hipError_t launch_w4a16_t_gemm(const void* dy, int64_t m, int64_t k, const uint8_t* packed, const void* scales,
                               const void* zeros, int sz_dtype, int64_t n, int g, void* dx, int dx_dtype,
                               const LoraOut& lo, int mi, int pw, int parts, int steps, hipStream_t st) {
  const Adapters ad{lo.low,           lo.out,        lo.offsets, lo.which, (int)lo.segments,
                    (int)lo.count, lo.rank, lo.dtype == W4_F32};
  if (sz_dtype == W4_F16)
    return tg_types<_Float16>(dy, m, k, packed, scales, zeros, n, g, dx, dx_dtype, mi, pw, parts, steps, ad, st);
  return tg_types<float>(dy, m, k, packed, scales, zeros, n, g, dx, dx_dtype, mi, pw, parts, steps, ad, st);
}

}  // namespace w4
