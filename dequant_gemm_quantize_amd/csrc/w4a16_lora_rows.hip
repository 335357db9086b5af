// W4A16 product with the adapters of its rows' requests, for few rows of bf16 x
// and any number of rows of float32 x:
//   y[m, n] = sum_k x[m, k] (q[n, k] - zp) s + sum_r low[m, r] B[l(m), n, r]
// The kernel is the few-row product's by expert, with one expert.  The low-rank
// part, 2 R operations an output, is a float32 dot product of the thread that adds the waves' sums.
#include "w4a16_grouped_rows.h"

namespace w4 {

template <typename TX>
static hipError_t lr_types(const void* x, int64_t m, int64_t k, const uint8_t* packed, const void* scales,
                           const void* zeros, int sz_dtype, int64_t n, int g, void* y, int y_dtype, const Adapters& ad,
                           hipStream_t st) {
  if (sz_dtype == W4_F16) {
    if (y_dtype == W4_F32)
      return gr_pick<TX, _Float16, float>(x, m, k, nullptr, 1, packed, scales, zeros, n, g, y, ad, st);
    return gr_pick<TX, _Float16, uint16_t>(x, m, k, nullptr, 1, packed, scales, zeros, n, g, y, ad, st);
  }
  if (y_dtype == W4_F32) return gr_pick<TX, float, float>(x, m, k, nullptr, 1, packed, scales, zeros, n, g, y, ad, st);
  return gr_pick<TX, float, uint16_t>(x, m, k, nullptr, 1, packed, scales, zeros, n, g, y, ad, st);
}

hipError_t launch_w4a16_lora_rows(const void* x, int x_dtype, int64_t m, int64_t k, const uint8_t* packed,
                                  const void* scales, const void* zeros, int sz_dtype, int64_t n, int g, void* y,
                                  int y_dtype, const LoraOut& lo, hipStream_t st) {
  const Adapters ad = adapters_of(lo);
  if (x_dtype == W4_F32) return lr_types<float>(x, m, k, packed, scales, zeros, sz_dtype, n, g, y, y_dtype, ad, st);
  return lr_types<uint16_t>(x, m, k, packed, scales, zeros, sz_dtype, n, g, y, y_dtype, ad, st);
}

}  // namespace w4
