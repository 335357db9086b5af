// W4A16 product with the adapters of its rows' requests, for many rows of bf16 x:
//   y[m, n] = sum_k x[m, k] (q[n, k] - zp) s + sum_r low[m, r] B[l(m), n, r]
// The kernel is the many-row product's by expert, with one expert.  The low-rank
// part goes to the same sums as a product of its own after the last K step: 16
// ranks an MFMA, three bf16 parts of the float32 low-rank values.
#include "w4a16_grouped_gemm.h"

namespace w4 {

hipError_t launch_w4a16_lora_gemm(const void* x, int64_t m, int64_t k, const uint8_t* packed, const void* scales,
                                  const void* zeros, int sz_dtype, int64_t n, int g, void* y, int y_dtype,
                                  const LoraOut& lo, hipStream_t st) {
  const Adapters ad{lo.low,           lo.out,        lo.offsets, lo.which, (int)lo.segments,
                    (int)lo.count, lo.rank, lo.dtype == W4_F32};
  const uint16_t* xb = (const uint16_t*)x;
  if (sz_dtype == W4_F16) {
    if (y_dtype == W4_F32) return gg_pick<_Float16, float>(xb, m, k, nullptr, 1, packed, scales, zeros, n, g, y, ad, st);
    return gg_pick<_Float16, __bf16>(xb, m, k, nullptr, 1, packed, scales, zeros, n, g, y, ad, st);
  }
  if (y_dtype == W4_F32) return gg_pick<float, float>(xb, m, k, nullptr, 1, packed, scales, zeros, n, g, y, ad, st);
  return gg_pick<float, __bf16>(xb, m, k, nullptr, 1, packed, scales, zeros, n, g, y, ad, st);
}

}  // namespace w4
