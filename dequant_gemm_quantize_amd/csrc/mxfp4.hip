// Microscaled 4-bit floating point (MXFP4): quantize and dequantize.
//
// A block is 32 consecutive elements of a row.  With amax the largest
// magnitude of the block (OCP Microscaling Formats v1.0, section 6.3):
//   E = max(floor(log2(amax)) - 2, -127), scale = 2^E, stored as E + 127
//   code = RNE(x / scale) in E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6), at most 6 in
//          magnitude, sign kept
// E2M1's largest power of two is 2^2, hence the 2.  The float32 exponent field
// less 2 is the stored byte (a subnormal amax has field 0 and clamps to 0,
// which is -127).  v_cvt_scalef32_pk_fp4_f32 divides by a power of two and
// rounds two elements to E2M1 exactly as above.
//
// Both kernels stream: nothing is read twice, and each lane's 8 elements are
// one or two 16-byte accesses.  Bound by the bytes: bf16 [28672, 8192] there and
// back takes 201 us, 5.9 TB/s with the codes and scales written and read again,
// some of them from cache (a copy of 1 GiB reaches 5.1 - 5.2).
#include "w4_common.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int64_t kMxMaxBlocks = 65536;  // workgroups of 256; longer inputs loop

// Chunk c: elements 8c .. 8c + 7, a quarter of a block; lanes 4i .. 4i + 3
// hold one block and share its amax by two butterflies.
template <typename TIn>
__global__ __launch_bounds__(256) void k_quantize_mxfp4(const void* __restrict__ w, int64_t nchunks,
                                                        uint32_t* __restrict__ packed,
                                                        uint8_t* __restrict__ scales) {
  // nchunks is a multiple of 4, so the four lanes of a block leave the loop together
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < nchunks; c += (int64_t)gridDim.x * 256) {
    float v[8];
    if constexpr (sizeof(TIn) == 4) {
      const f32x4* p = (const f32x4*)w + 2 * c;
      const f32x4 a = ldg_nt(p), b = ldg_nt(p + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    } else {
      const u32x4 a = ldg_nt((const u32x4*)w + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(a[i]);
        v[2 * i + 1] = bf16_hi(a[i]);
      }
    }
    // the bit patterns of magnitudes order as the magnitudes do, with
    // infinity and NaN above every number
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
      top = top > b ? top : b;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const uint32_t b = (uint32_t)__shfl_xor((int)top, o, kWave);
      top = top > b ? top : b;
    }
    const uint32_t field = top >> 23;
    uint32_t byte = field > 2 ? field - 2 : 0;
    // the conversion takes the scale's exponent field alone: byte 0 is 2^-127
    const float scale = __uint_as_float(byte << 23);
    uint32_t word = 0;
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[0], v[1], scale, 0);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[2], v[3], scale, 1);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[4], v[5], scale, 2);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, v[6], v[7], scale, 3);
    if (field == 255) {  // the block holds an infinity or a NaN: the NaN scale
      byte = 255;
      word = 0;
    }
    packed[c] = word;
    if ((c & 3) == 0) scales[c >> 2] = (uint8_t)byte;
  }
}

// 2^(byte - 127) in float32 (2^-127 is subnormal; 255 is NaN).
__device__ __forceinline__ float e8m0(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

template <int OUT>
__global__ __launch_bounds__(256) void k_dequant_mxfp4(const uint32_t* __restrict__ packed,
                                                       const uint8_t* __restrict__ scales, int64_t nchunks,
                                                       void* __restrict__ out) {
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < nchunks; c += (int64_t)gridDim.x * 256) {
    const uint32_t word = packed[c];
    const float s = e8m0(scales[c >> 2]);
    // code values by the conversion at scale 1, then one float32 product:
    // exact unless it leaves the float32 range
    float v[8];
    f32x2 t;
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 0);
    v[0] = t.x * s, v[1] = t.y * s;
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 1);
    v[2] = t.x * s, v[3] = t.y * s;
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 2);
    v[4] = t.x * s, v[5] = t.y * s;
    t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, 3);
    v[6] = t.x * s, v[7] = t.y * s;
    if constexpr (OUT == W4_F32) {
      f32x4* o = (f32x4*)out + 2 * c;
      o[0] = f32x4{v[0], v[1], v[2], v[3]};
      o[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      u32x4 r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (OUT == W4_BF16)
          r[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
        else
          r[i] = f32_to_f16_bits(v[2 * i]) | (f32_to_f16_bits(v[2 * i + 1]) << 16);
      }
      ((u32x4*)out)[c] = r;
    }
  }
}

dim3 mx_grid(int64_t nchunks) {
  const int64_t blocks = (nchunks + 255) / 256;
  return dim3((unsigned)(blocks < kMxMaxBlocks ? blocks : kMxMaxBlocks));
}

}  // namespace

hipError_t launch_quantize_mxfp4(const void* w, int w_dtype, int64_t n, int64_t k, uint8_t* packed,
                                 uint8_t* scales, hipStream_t st) {
  const int64_t nchunks = n * k / 8;
  if (w_dtype == W4_F32)
    k_quantize_mxfp4<float><<<mx_grid(nchunks), 256, 0, st>>>(w, nchunks, (uint32_t*)packed, scales);
  else
    k_quantize_mxfp4<__bf16><<<mx_grid(nchunks), 256, 0, st>>>(w, nchunks, (uint32_t*)packed, scales);
  return hipGetLastError();
}

hipError_t launch_dequant_mxfp4(const uint8_t* packed, const uint8_t* scales, int64_t n, int64_t k,
                                void* out, int out_dtype, hipStream_t st) {
  const int64_t nchunks = n * k / 8;
  const dim3 grid = mx_grid(nchunks);
  const uint32_t* pk = (const uint32_t*)packed;
  if (out_dtype == W4_F32)
    k_dequant_mxfp4<W4_F32><<<grid, 256, 0, st>>>(pk, scales, nchunks, out);
  else if (out_dtype == W4_F16)
    k_dequant_mxfp4<W4_F16><<<grid, 256, 0, st>>>(pk, scales, nchunks, out);
  else
    k_dequant_mxfp4<W4_BF16><<<grid, 256, 0, st>>>(pk, scales, nchunks, out);
  return hipGetLastError();
}

}  // namespace w4
