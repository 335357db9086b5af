// Pieces shared by the products that feed the matrix cores from LDS tiles
// filled straight from memory.
#pragma once

#include "w4_common.h"

namespace w4 {

// Raw buffer resource that answers reads past `bytes` with zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_rsrc_n(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// 16 bytes a lane from the resource at the lane's offset to LDS at dst + 16
// lane (dst the same in every lane), without passing through registers.
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t rs, uint8_t* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, (int)off, 0, 0, 0);
}

// The same with a part of the offset that is the same in every lane; the range is that of the lane's part alone.
__device__ __forceinline__ void load_lds_at(__amdgpu_buffer_rsrc_t rs, uint8_t* dst, uint32_t off, uint32_t all) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, (int)off, (int)all, 0,
                                           0);
}

// The same with 4 bytes a lane, to dst + 4 lane.
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t rs, uint8_t* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 4, (int)off, 0, 0, 0);
}

// Orders R LDS reads among the M MFMAs that precede this call: at most 15 reads
// of a wave can be outstanding, and one more would hold up the MFMAs behind it.
template <int M, int R>
__device__ __forceinline__ void interleave() {
  if constexpr (M > 0 && R > 0) {
    constexpr int per = (R + M - 1) / M;
    __builtin_amdgcn_sched_group_barrier(0x100, per, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    interleave<M - 1, R - per>();
  }
}

// Tile t of tiles_m x tiles_n in bands of 8 M tiles (the last may have fewer).
__device__ __forceinline__ void band(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
  const uint32_t b = t / (8 * tiles_n), in = t - b * 8 * tiles_n;
  const uint32_t width = tiles_m - 8 * b < 8 ? tiles_m - 8 * b : 8;
  tn = in / width;
  tm = 8 * b + in % width;
}

constexpr uint32_t kPastEnd = 0x80000000u;  // beyond every resource: their sizes stay below 2^31

// Which tile of `total` a workgroup has.  Each XCD (workgroup number mod 8)
// takes a contiguous eighth of the list, SLOTS tiles at a time (32 CUs times
// the workgroups that one holds).  With SPLIT, tiles beyond the last whole round
// of SLOTS are split into halves of half the rows when all the halves fit one
// round, which then takes 0.6 of the time (2048 x 4096 x 11008 in MXFP4 63 us
// without, 58 with).  `half` is -1 (a whole tile), 0 or 1.
// False: nothing to do.  A launch has xcd_grid(tiles) workgroups.
template <uint32_t SLOTS, bool SPLIT>
__device__ __forceinline__ bool xcd_tile(uint32_t total, uint32_t& tile, int& half) {
  const uint32_t per = (total + 7) / 8, first = (blockIdx.x & 7) * per, j = blockIdx.x >> 3;
  half = -1;
  if (first >= total) return false;
  const uint32_t mine = total - first < per ? total - first : per;
  const uint32_t rest = mine % SLOTS, whole = mine - rest;
  uint32_t at = j;
  if (SPLIT && j >= whole && rest <= SLOTS / 2) {
    at = whole + (j - whole) / 2;
    half = (int)((j - whole) & 1);
  }
  tile = first + at;
  return at < mine;
}
template <uint32_t SLOTS, bool SPLIT>
inline int64_t xcd_grid(int64_t tiles) {
  return (tiles + 7) / 8 * 8 + (SPLIT ? 8 * (SLOTS / 2) : 0);
}

// Rounds of tiles, a round of halves taking `part` of one.
template <uint32_t SLOTS>
inline double xcd_rounds(int64_t tiles, double part) {
  const int64_t mine = (tiles + 7) / 8, rest = mine % SLOTS;
  return (double)(mine / SLOTS) + (rest == 0 ? 0.0 : rest <= SLOTS / 2 ? part : 1.0);
}

// Turns a wave's 32 x 32 blocks around in LDS and stores them to y.
//
// WFIRST: register e of acc[i][j] holds y row r = lane % 32 of block row i,
// column 8 (e / 4) + 4 (lane / 32) + e % 4 of block column j (the weights are
// the MFMA's first operand), so four registers are four consecutive columns.
// Otherwise the other way round (x is the first operand).  32
// rows at a time go to `turn` (turn_bytes of the wave's own) and leave it in
// whole rows, 16 bytes a lane: stores of single elements made the MXFP4
// product of 2048 x 11008 x 4096 take 84 us against 73.  Slot c ^ (row % SW)
// of a row holds its 16-byte chunk c, which keeps the reads, and the stores
// but for one conflict in four, apart in the banks.  The LDS operations of a
// wave complete in order; the wave barriers (no instruction) keep the compiler,
// which looks at one lane alone, from changing that order.
template <typename TY, int NJ>
constexpr int turn_bytes() {
  return 32 * 32 * NJ * (int)sizeof(TY);
}

template <typename TY, int MI, int NJ, bool WFIRST = true>
__device__ __forceinline__ void turn_store(uint8_t* turn, int lane, const f32x16 (&acc)[MI][NJ], TY* y, int64_t N,
                                           int64_t mb, int64_t mend, int64_t nb) {
  constexpr int CB = 32 * NJ * (int)sizeof(TY);  // bytes of a row of the block
  constexpr int CH = CB / 16;                    // its chunks
  constexpr int SW = (CH & -CH) < 16 ? (CH & -CH) : 16;
  constexpr int PER = 16 / (int)sizeof(TY);      // elements of a chunk
  const int r = lane & 31, h = lane >> 5;
  const bool wide = N % PER == 0;  // rows of y start at 16-byte addresses
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    if (mb + 32 * i >= mend) break;  // the same in every lane
    if constexpr (WFIRST) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v0 = acc[i][j][4 * q], v1 = acc[i][j][4 * q + 1], v2 = acc[i][j][4 * q + 2],
                      v3 = acc[i][j][4 * q + 3];
          const int col = 32 * j + 8 * q + 4 * h;
          uint8_t* dst = turn + r * CB + 16 * ((col / PER) ^ (r & (SW - 1)));
          if constexpr (sizeof(TY) == 4) {
            *(f32x4*)dst = f32x4{v0, v1, v2, v3};
          } else {
            u32x2 b;
            b.x = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v0, (__bf16)v1});
            b.y = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v2, (__bf16)v3});
            *(u32x2*)(dst + 8 * h) = b;
          }
        }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int row = 8 * (e >> 2) + 4 * h + (e & 3);
        uint8_t* dst = turn + row * CB + sizeof(TY) * (r % PER);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          uint8_t* at = dst + 16 * (((32 * j + r) / PER) ^ (row & (SW - 1)));
          if constexpr (sizeof(TY) == 4) *(float*)at = acc[i][j][e];
          else *(uint16_t*)at = (uint16_t)f32_to_bf16_bits(acc[i][j][e]);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (wide) {
#pragma unroll
      for (int t = 0; t < 32 * CH / 64; ++t) {
        const int at = 64 * t + lane, row = at / CH, c = at % CH;
        const u32x4 v = *(const u32x4*)(turn + row * CB + 16 * (c ^ (row & (SW - 1))));
        const int64_t m = mb + 32 * i + row, n = nb + PER * c;
        if (m < mend && n < N) *(u32x4*)(y + m * N + n) = v;
      }
    } else {
      for (int at = lane; at < 32 * 32 * NJ; at += 64) {
        const int row = at / (32 * NJ), col = at % (32 * NJ);
        const TY v = *(const TY*)(turn + row * CB + 16 * ((col / PER) ^ (row & (SW - 1))) + sizeof(TY) * (col % PER));
        const int64_t m = mb + 32 * i + row, n = nb + col;
        if (m < mend && n < N) y[m * N + n] = v;
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace w4
