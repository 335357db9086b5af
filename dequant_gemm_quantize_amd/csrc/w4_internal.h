// Internal launcher interface between the C ABI (api.cpp) and the kernels.
// Launchers assume validated arguments and enqueue on the given stream.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include <atomic>

#include "../../include/w4.h"

namespace w4 {

// Runs set() (an idempotent per-device setting such as a kernel's dynamic-LDS
// limit) once for the current device and remembers success in `done`, one bit
// per device.  Concurrent first calls may both run set(); that is harmless.
// Devices past 63 are set on every call.
template <typename F>
hipError_t once_per_device(std::atomic<uint64_t>& done, F set) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return hipSuccess;
  e = set();
  if (e == hipSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

hipError_t launch_quantize_pack(const void* w, int w_dtype, int64_t n, int64_t k, int g,
                                uint8_t* packed, void* scales, void* zeros, int sz_dtype,
                                bool symmetric, hipStream_t st);
// Calibrated symmetric quantize + pack: mode 0 = percentile (param = p in
// (0, 100]), mode 1 = MSE search (param = candidates, >= 2); g <= 1024.
bool quantize_cal_fits(int g);
hipError_t launch_quantize_pack_cal(const void* w, int w_dtype, int64_t n, int64_t k, int g, int mode,
                                    double param, uint8_t* packed, void* scales, void* zeros,
                                    int sz_dtype, hipStream_t st);
// GPTQ ([P4] Step 3): Hessian, inverse Cholesky factor, column sweep.
bool gptq_group_ok(int g);
hipError_t launch_gptq_hessian(const float* x, int64_t t, int k, double* h, hipStream_t st);
hipError_t launch_gptq_inverse_cholesky(double* h, int k, double* u, int* info, hipStream_t st);
hipError_t launch_gptq_quantize_pack(float* w, const double* u, int64_t n, int k, int g, bool symmetric,
                                     uint8_t* packed, void* scales, void* zeros, int sz_dtype,
                                     hipStream_t st);
hipError_t launch_dequant(const uint8_t* packed, const void* scales, const void* zeros,
                          int sz_dtype, int64_t n, int64_t k, int g, void* out, int out_dtype,
                          hipStream_t st);
hipError_t launch_act_quant(const void* x, int x_dtype, int64_t m, int64_t k, int8_t* xq,
                            float* x_scale, hipStream_t st);
hipError_t launch_w4a16_generic(const void* x, int x_dtype, int64_t m, int64_t k,
                                const uint8_t* packed, const void* scales, const void* zeros,
                                int sz_dtype, int64_t n, int g, void* y, int y_dtype,
                                hipStream_t st);
hipError_t launch_w4a16_decode(const void* x, int64_t m, int64_t k, const uint8_t* packed,
                               const void* scales, const void* zeros, int sz_dtype, int64_t n,
                               int g, void* y, int y_dtype, hipStream_t st);
bool decode_lds_fits(int64_t m, int64_t k);
hipError_t launch_w4a16_dot2(const void* x, int64_t m, int64_t k, const uint8_t* packed,
                             const void* scales, const void* zeros, int sz_dtype, int64_t n,
                             int g, void* y, int y_dtype, hipStream_t st);
bool dot2_fits(int64_t m, int64_t k, int g);
hipError_t launch_w4a16_gemv(const void* x, int64_t m, int64_t k, const uint8_t* packed,
                             const void* scales, const void* zeros, int sz_dtype, int64_t n,
                             int g, void* y, int y_dtype, hipStream_t st);
bool gemv_mfma_fits(int64_t m, int64_t k, int g);
// 2 <= M <= 4 tokens on the 4x4x4 matrix-core shape: K = 4096, g % 32 == 0.
hipError_t launch_w4a16_quad(const void* x, int64_t m, int64_t k, const uint8_t* packed,
                             const void* scales, const void* zeros, int sz_dtype, int64_t n,
                             int g, void* y, int y_dtype, hipStream_t st);
bool quad_fits(int64_t m, int64_t k, int g);
// ws: optional float32 workspace for split K (nullptr or too small: no split).
hipError_t launch_w4a16_gemm(const void* x, int64_t m, int64_t k, const uint8_t* packed,
                             const void* scales, const void* zeros, int sz_dtype, int64_t n,
                             int g, void* y, int y_dtype, void* ws, size_t ws_bytes, hipStream_t st);
bool gemm_fits(int64_t m, int64_t k, int g);
// Bytes of workspace the GEMM uses for split K on this shape (0: it does not
// split); never above kSplitKMaxBytes.
constexpr size_t kSplitKMaxBytes = (size_t)32 << 20;
size_t gemm_workspace_bytes(int64_t m, int64_t k, int64_t n, int g);
// Device address (current device) of the library's static scratch of
// kSplitKMaxBytes, for callers that cannot allocate.
hipError_t scratch_address(void** out);
hipError_t launch_w4a8_gemv(const int8_t* xq, const float* xs, int64_t m, int64_t k,
                            const uint8_t* packed, const void* scales, const void* zeros,
                            int sz_dtype, int64_t n, int g, void* y, int y_dtype, hipStream_t st);
bool w4a8_gemv_fits(int64_t m, int64_t k, int g);
hipError_t launch_w4a8_gemv_mfma(const int8_t* xq, const float* xs, int64_t m, int64_t k,
                                 const uint8_t* packed, const void* scales, const void* zeros,
                                 int sz_dtype, int64_t n, int g, void* y, int y_dtype,
                                 hipStream_t st);
bool w4a8_gemv_mfma_fits(int64_t m, int64_t k, int g);
// ws: optional float32 workspace for split K (nullptr or too small: no split).
hipError_t launch_w4a8_gemm(const int8_t* xq, const float* xs, int64_t m, int64_t k,
                            const uint8_t* packed, const void* scales, const void* zeros,
                            int sz_dtype, int64_t n, int g, void* y, int y_dtype, void* ws,
                            size_t ws_bytes, hipStream_t st);
bool w4a8_gemm_fits(int64_t m, int64_t k, int g);
// Bytes of workspace the W4A8 GEMM uses for split K on this shape (0: it does
// not split); never above kSplitKMaxBytes.
size_t w4a8_gemm_workspace_bytes(int64_t m, int64_t k, int64_t n, int g);
// y = the sum, in order s = 0 .. S-1, of the float32 partials part + s *
// pstride ([M][N], MN elements each), rounded once to y_dtype.
hipError_t launch_splitk_reduce(const float* part, int S, int64_t mn, int64_t pstride, void* y,
                                int y_dtype, hipStream_t st);
hipError_t launch_w4a8_generic(const int8_t* xq, const float* xs, int64_t m, int64_t k,
                               const uint8_t* packed, const void* scales, const void* zeros,
                               int sz_dtype, int64_t n, int g, void* y, int y_dtype,
                               hipStream_t st);
// MXFP4: quantize, dequantize.
hipError_t launch_quantize_mxfp4(const void* w, int w_dtype, int64_t n, int64_t k, uint8_t* packed,
                                 uint8_t* scales, hipStream_t st);
hipError_t launch_dequant_mxfp4(const uint8_t* packed, const uint8_t* scales, int64_t n, int64_t k,
                                void* out, int out_dtype, hipStream_t st);
// MXFP4 products; by expert when offsets is not null (device memory, experts
// + 1 entries bounding each expert's rows), dense otherwise.
hipError_t launch_mx_rows(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                          const uint8_t* scales, int64_t n, void* y, int y_dtype, const int* offsets,
                          int experts, hipStream_t st);
bool mx_gemm_fits(int64_t k);
hipError_t launch_mx_gemm(const uint8_t* xq, const uint8_t* xs, int64_t m, int64_t k, const uint8_t* packed,
                          const uint8_t* scales, int64_t n, void* y, int y_dtype, const int* offsets,
                          int experts, hipStream_t st);
// W4A16 by expert: few rows an expert or float32 x, and many rows.
hipError_t launch_w4a16_grouped_rows(const void* x, int x_dtype, int64_t t, int64_t k, const int* offsets, int experts,
                                     const uint8_t* packed, const void* scales, const void* zeros, int sz_dtype,
                                     int64_t n, int g, void* y, int y_dtype, hipStream_t st);
bool w4a16_grouped_gemm_fits(int64_t k);
hipError_t launch_w4a16_grouped_gemm(const void* x, int64_t t, int64_t k, const int* offsets, int experts,
                                     const uint8_t* packed, const void* scales, const void* zeros, int sz_dtype,
                                     int64_t n, int g, void* y, int y_dtype, hipStream_t st);
// Activation checkpoints in 8 bits.
hipError_t launch_quantize_checkpoint(const void* x, int x_dtype, int64_t m, int64_t k, int8_t* xq, float* xs,
                                      hipStream_t st);
hipError_t launch_dequant_checkpoint(const int8_t* xq, const float* xs, int64_t m, int64_t k, void* out, int out_dtype,
                                     hipStream_t st);
// Low-rank adapters.  Rows in segments (offsets and which in device memory),
// matrices of `count` adapters of rank `rank` (a multiple of 8).
// low [M, R] = scaling x W^T, down: W [L, R, D] (D % 32 == 0), otherwise W [L, D, R].
struct LoraInto {
  bool down;
  const void* x;
  int x_dtype;
  int64_t m, d;
  const void* weights;
  int w_dtype;
  int64_t count;
  int rank;
  const float* scaling;
  const int* offsets;
  const int* which;
  int64_t segments;
  float* low;
  int parts;  // > 1, not down: low takes as many partial sums, [parts, M, R]
};
hipError_t launch_lora_into(const LoraInto& a, hipStream_t st);
// The parts of a sum over d that a call without `down` should have where the reader of low can add them.
size_t lora_into_parts(int64_t m, int64_t d, int64_t segments, int rank);
// The low-rank part that a product adds: low [M, R] times `out`, [L, N, R] beside
// x W^T (whose columns are N) and [L, R, K] beside dy W.  count 0: none.
struct LoraOut {
  const float* low;
  const void* out;
  int dtype;
  int64_t count;
  int rank;
  const int* offsets;
  const int* which;
  int64_t segments;
  int parts;     // > 1: low is as many partial sums, which the product's last kernel adds
  float* whole;  // and where it leaves the sums of the rows that have an adapter
};
// A W4A16 product of m rows: forward x [m, k] W^T, back x [m, n] W.  In tiles, for bf16 x: of 32 mi
// rows forward; back of 64 mi, with pw bf16 parts of a weight (2, or 3 with float32
// scales and a float32 result).  With parts > 1 float32 partial sums of `steps` steps each (256 columns
// forward, 64 weight rows back), forward the first of them with the low-rank part.
struct TilesArgs {
  bool back;
  const void* x;
  int64_t m, k, n;
  const uint8_t* packed;
  const void* scales;
  const void* zeros;
  int sz_dtype, g;
  void* y;
  int y_dtype;
  int mi, pw, parts, steps;
  int64_t row;  // back: values from a row of x to the next, a multiple of 8; zeros behind the n'th
};
hipError_t launch_w4a16_lora_gemm(const TilesArgs& a, const LoraOut& lo, hipStream_t st);  // forward
hipError_t launch_w4a16_tiles(const TilesArgs& a, const LoraOut& lo, hipStream_t st);      // back
// Forward for few rows, and for float32 x.
hipError_t launch_w4a16_lora_rows(const void* x, int x_dtype, int64_t m, int64_t k, const uint8_t* packed,
                                  const void* scales, const void* zeros, int sz_dtype, int64_t n, int g, void* y,
                                  int y_dtype, const LoraOut& lo, hipStream_t st);
// Either direction, whatever the sizes (args without x and what follows y_dtype), and the workspace's bytes (0: none).
size_t w4a16_lora_workspace_bytes(bool back, int64_t m, int64_t k, int64_t n, int g, int x_dtype, int sz_dtype,
                                  int y_dtype);
// Whether the call ends in the kernel that adds partial sums, which takes the low-rank values in parts too (back).
bool w4a16_lora_sums(bool back, int64_t m, int64_t k, int64_t n, int g, int x_dtype, int sz_dtype, int y_dtype);
hipError_t launch_w4a16_lora(const void* x, int x_dtype, const TilesArgs& args, const LoraOut& lo, void* ws,
                             hipStream_t st);
// Gradients of the adapters from the 8-bit checkpoint of x, dy and the low-rank values.
struct LoraGrads {
  const int8_t* xq;
  const float* xs;
  int64_t m, k;
  const void* dy;
  int dy_dtype;
  int64_t n;
  const float* u;
  const float* v;
  const int* offsets;
  const int* which;
  int64_t segments, count;
  int rank;
  float* da;
  float* db;
  void* ws;
};
size_t lora_grads_workspace_bytes(int64_t m, int64_t k, int64_t n, int dy_dtype, int64_t count, int rank);
hipError_t launch_lora_grads(const LoraGrads& a, hipStream_t st);
// Limits of the adapters.
constexpr int64_t kLoraMaxRows = (int64_t)1 << 24;
constexpr int64_t kLoraMaxSegments = (int64_t)1 << 20;
constexpr int64_t kLoraMaxAdapters = 65536;
constexpr int kLoraMaxRank = 256;
// Limits of the products by expert: tile numbers stay below 2^31.
constexpr int64_t kGroupedMaxRows = (int64_t)1 << 24;
constexpr int64_t kGroupedMaxExperts = 65536;

}  // namespace w4
