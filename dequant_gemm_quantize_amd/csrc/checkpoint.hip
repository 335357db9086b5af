// Activation checkpoints in 8 bits: blocks of 128 consecutive columns of a row
// (the last one shorter where K is no multiple of 128), each with a float32 scale.
//   scale = fl32(max |block| / 127)
//   code  = the whole number nearest to x / scale (ties to even), at most 127 in magnitude
//   value = fl32(code scale)
// The quotient that decides a code is the exact one: a first guess by the
// reciprocal is at most one off, and the remainder x - code scale, which one fma
// gives exactly next to the borders +- scale / 2, says which way.
//
// 16 lanes have a block, 8 columns each.  Bound by memory, with the vector unit close
// behind: 4096 x 11008 bf16 into codes 23 us (34 with the borders looked at for every value), back 22.
#include <type_traits>

#include "lora.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int CB = 128;  // columns of a block

// The codes of 8 values where a first guess may be off by one or a border is met.
__device__ __forceinline__ void codes_at_borders(const float (&v)[8], float s, uint32_t (&out)[2]) {
  const float inv = 1.0f / s, half = 0.5f * s;
  out[0] = out[1] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = rintf(v[i] * inv);
    const float rest = fmaf(-q, s, v[i]);
    const int c = (int)q;
    const bool odd = c & 1;
    int d = c;
    if (rest > half || (rest == half && odd)) d = c + 1;
    else if (rest < -half || (rest == -half && odd)) d = c - 1;
    d = d > 127 ? 127 : d < -127 ? -127 : d;
    out[i >> 2] |= (uint32_t)(uint8_t)d << (8 * (i & 3));
  }
}

template <typename TX>
__device__ __forceinline__ void quantize_block(const TX* __restrict__ x, uint32_t blk, int64_t K, uint32_t nb,
                                               int8_t* __restrict__ xq, float* __restrict__ xs) {
  const uint32_t row = blk / nb, j = blk - row * nb;
  const int l = threadIdx.x & 15;
  const int64_t col = (int64_t)CB * j + 8 * l;
  const bool in = col < K;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (in) values8(x + row * K + col, v);
  // magnitudes compare as their bits do, infinities and NaN above all others
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
    top = a > top ? a : top;
  }
  // the largest of the 16 lanes: within pairs, fours, eights and all of a row (register moves)
  auto other = [&](auto ctrl) {
    const uint32_t a = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, decltype(ctrl)::value, 0xf, 0xf, false);
    top = a > top ? a : top;
  };
  other(std::integral_constant<int, 0xb1>{});   // lanes 1 0 3 2 of four
  other(std::integral_constant<int, 0x4e>{});   // 2 3 0 1
  other(std::integral_constant<int, 0x141>{});  // the other way round in eight
  other(std::integral_constant<int, 0x140>{});  // and in sixteen
  const bool bad = top >= 0x7f800000u;
  const float s = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 127.0f;
  if (l == 0) xs[blk] = s;
  if (!in) return;
  uint32_t out[2] = {0, 0};
  if (!bad && s >= 0x1p-64f) {
    // The first guess, by a reciprocal good to one step, is right unless its remainder reaches half the scale.
    const float inv = __builtin_amdgcn_rcpf(s);
    float most = 0.0f;
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = rintf(v[i] * inv);
      most = fmaxf(most, fabsf(fmaf(-q, s, v[i])));
      c[i] = (uint32_t)(int)q;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __builtin_amdgcn_perm(c[4 * i + 1], c[4 * i], 0x0c0c0400u),
                     hi = __builtin_amdgcn_perm(c[4 * i + 3], c[4 * i + 2], 0x04000c0cu);
      out[i] = lo | hi;
    }
    if (most >= 0.5f * s) codes_at_borders(v, s, out);
  } else if (!bad && s != 0.0f) {
    // tiny scales: x and scale times 2^64, exactly, so that the reciprocal and half the scale are normal numbers
    float up[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) up[i] = v[i] * 0x1p64f;
    codes_at_borders(up, s * 0x1p64f, out);
  }
  *(u32x2*)(xq + row * K + col) = u32x2{out[0], out[1]};
}

template <typename TY>
__device__ __forceinline__ void dequant_block(const int8_t* __restrict__ xq, const float* __restrict__ xs, uint32_t blk,
                                              int64_t K, uint32_t nb, TY* __restrict__ y) {
  const uint32_t row = blk / nb, j = blk - row * nb;
  const int64_t col = (int64_t)CB * j + 8 * (threadIdx.x & 15);
  if (col >= K) return;
  const float s = xs[blk];
  const u32x2 q = *(const u32x2*)(xq + row * K + col);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = (float)(int8_t)(q[i >> 2] >> (8 * (i & 3))) * s;
    // no instruction: keeps the compiler from making the product and its rounding to
    // fp16 one instruction, which would round once where the definition rounds twice
    asm("" : "+v"(v[i]));
  }
  TY* out = y + row * K + col;
  if constexpr (sizeof(TY) == 4) {
    ((f32x4*)out)[0] = f32x4{v[0], v[1], v[2], v[3]};
    ((f32x4*)out)[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (__is_same(TY, _Float16)) b[i] = f32_to_f16_bits(v[2 * i]) | f32_to_f16_bits(v[2 * i + 1]) << 16;
      else b[i] = f32_to_bf16_bits(v[2 * i]) | f32_to_bf16_bits(v[2 * i + 1]) << 16;
    }
    *(u32x4*)out = b;
  }
}

// A workgroup has 16 blocks at a time; launches of more than 2^20 workgroups loop.
uint32_t checkpoint_grid(uint32_t blocks) {
  const uint32_t g = (blocks + 15u) / 16u;
  return g < (1u << 20) ? g : 1u << 20;
}

}  // namespace

template <typename TX>
__global__ __launch_bounds__(256) void k_quantize_checkpoint(const TX* __restrict__ x, uint32_t blocks, int64_t K,
                                                             uint32_t nb, int8_t* __restrict__ xq,
                                                             float* __restrict__ xs) {
  for (uint32_t blk = blockIdx.x * 16u + (threadIdx.x >> 4); blk < blocks; blk += gridDim.x * 16u)
    quantize_block(x, blk, K, nb, xq, xs);  // whole groups of 16 lanes
}

template <typename TY>
__global__ __launch_bounds__(256) void k_dequant_checkpoint(const int8_t* __restrict__ xq,
                                                            const float* __restrict__ xs, uint32_t blocks, int64_t K,
                                                            uint32_t nb, TY* __restrict__ y) {
  for (uint32_t blk = blockIdx.x * 16u + (threadIdx.x >> 4); blk < blocks; blk += gridDim.x * 16u)
    dequant_block(xq, xs, blk, K, nb, y);
}

hipError_t launch_quantize_checkpoint(const void* x, int x_dtype, int64_t m, int64_t k, int8_t* xq, float* xs,
                                      hipStream_t st) {
  const uint32_t nb = (uint32_t)((k + CB - 1) / CB), blocks = (uint32_t)(m * nb);
  const dim3 grid(checkpoint_grid(blocks));
  if (x_dtype == W4_F32)
    k_quantize_checkpoint<<<grid, 256, 0, st>>>((const float*)x, blocks, k, nb, xq, xs);
  else
    k_quantize_checkpoint<<<grid, 256, 0, st>>>((const uint16_t*)x, blocks, k, nb, xq, xs);
  return hipGetLastError();
}

hipError_t launch_dequant_checkpoint(const int8_t* xq, const float* xs, int64_t m, int64_t k, void* out, int out_dtype,
                                     hipStream_t st) {
  const uint32_t nb = (uint32_t)((k + CB - 1) / CB), blocks = (uint32_t)(m * nb);
  const dim3 grid(checkpoint_grid(blocks));
  if (out_dtype == W4_F32) k_dequant_checkpoint<<<grid, 256, 0, st>>>(xq, xs, blocks, k, nb, (float*)out);
  else if (out_dtype == W4_F16) k_dequant_checkpoint<<<grid, 256, 0, st>>>(xq, xs, blocks, k, nb, (_Float16*)out);
  else k_dequant_checkpoint<<<grid, 256, 0, st>>>(xq, xs, blocks, k, nb, (uint16_t*)out);
  return hipGetLastError();
}

}  // namespace w4
