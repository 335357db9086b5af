// Low-rank adapters beside a product: which adapter a row has, and operands of
// bf16 or float32 adapters for the bf16 matrix cores.
//
// Rows come in segments (requests): offsets[0 .. S] (device memory, int32,
// rising) bound them, segment s has adapter which[s]; a negative number, or one
// past the last adapter, stands for none.  The host does not know them.  Every
// value read is clamped, so no offsets and no adapter numbers lead out of bounds.
#pragma once

#include "grouped.h"
#include "w4_common.h"
#include "w4_internal.h"

namespace w4 {

// The adapters of a product: the adapters' outer matrices `out` [L, D, R], rows of R
// values in a product's columns D, and the rows' low-rank values [M, R].
struct Adapters {
  static constexpr bool any = true;
  const float* low;
  const void* out;
  const int* offsets;
  const int* which;
  int segments, count, rank, wide;  // wide: `out` is float32, otherwise bf16
  int parts;     // > 1: low is [parts, M, R], to be added (k_w4a16_sum alone does)
  float* whole;  // the sums, of the rows that have an adapter
};
inline Adapters adapters_of(const LoraOut& lo) {
  return Adapters{lo.low, lo.out, lo.offsets, lo.which, (int)lo.segments, (int)lo.count, lo.rank, lo.dtype == W4_F32, lo.parts,
                  lo.whole};
}
struct NoAdapters {
  static constexpr bool any = false;
};

// How many of the segments end at or before row m: the segment of m, or S.  The
// same in every lane; all 64 lanes call it.
__device__ __forceinline__ int segments_before(const int* offsets, int segments, int64_t m, int lane) {
  int n = 0;
  for (int base = 0; base < segments; base += kWave) {
    const bool ends = base + lane < segments && offsets[base + lane + 1] <= m;
    n += __builtin_popcountll(__ballot(ends));
  }
  return n;
}

// The adapter of row m, or -1.  The same in every lane; all 64 lanes call it.  The
// adapters' numbers are loaded beside the offsets, not behind them.
__device__ __forceinline__ int row_adapter(const Adapters& a, int64_t m, int lane) {
  for (int base = 0; base < a.segments; base += kWave) {
    const bool in = base + lane < a.segments;
    const int begin = in ? a.offsets[base + lane] : 0, end = in ? a.offsets[base + lane + 1] : 0;
    const int w = in ? a.which[base + lane] : -1;
    const uint64_t past = __ballot(in && end > m);
    if (past != 0) {  // the first segment that ends behind m
      const int f = __builtin_ctzll(past), ad = __builtin_amdgcn_readlane(w, f);
      return __builtin_amdgcn_readlane(begin, f) <= m && ad >= 0 && ad < a.count ? ad : -1;
    }
  }
  return -1;
}

// A tile of bm rows of one segment, `width` tiles side by side.
struct SegmentTile {
  int adapter;   // -1: none
  int64_t m0;    // first row
  int rows;
  uint32_t side;  // which of the `width`
};
// Tile `want` of the list in which every segment has its tiles of bm rows times
// `width`, as find_group_tile; the adapters' numbers are loaded beside the offsets, not behind them.
__device__ __forceinline__ bool find_segment_tile(const int* offsets, const int* which, int segments, int count, int M,
                                                  int bm, uint32_t width, int64_t want, int lane, SegmentTile& t) {
  int64_t before = 0;
  for (int base = 0; base < segments; base += kWave) {
    int row0;
    const int w = base + lane < segments ? which[base + lane] : -1;
    const int rows = group_rows(offsets, segments, M, base, lane, row0);
    const int mine = (rows + bm - 1) / bm;
    const int upto = wave_scan(mine);
    const uint64_t past = __ballot((before + upto) * width > want);
    if (past != 0) {
      const int f = __builtin_ctzll(past);
      const int ad = __builtin_amdgcn_readlane(w, f), have = __builtin_amdgcn_readlane(rows, f);
      const uint32_t tile = (uint32_t)(want - (before + __builtin_amdgcn_readlane(upto - mine, f)) * width);
      const int skip = bm * (int)(tile / width);
      t.adapter = ad >= 0 && ad < count ? ad : -1;
      t.m0 = __builtin_amdgcn_readlane(row0, f) + skip;
      t.rows = have - skip < bm ? have - skip : bm;
      t.side = tile % width;
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  return false;
}

// 8 float32 as hi + mid + lo, each 8 bf16: the upper halves of the words, of
// what they lack, and of what that lacks, which is exact for normal values.
__device__ __forceinline__ void split8(u32x4 v0, u32x4 v1, bf16x8 (&out)[3]) {
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    u32x4 r;
    r.x = __builtin_amdgcn_perm(v0.y, v0.x, 0x07060302u);
    r.y = __builtin_amdgcn_perm(v0.w, v0.z, 0x07060302u);
    r.z = __builtin_amdgcn_perm(v1.y, v1.x, 0x07060302u);
    r.w = __builtin_amdgcn_perm(v1.w, v1.z, 0x07060302u);
    out[p] = __builtin_bit_cast(bf16x8, r);
    if (p < 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v0[i] = __float_as_uint(__uint_as_float(v0[i]) - __uint_as_float(v0[i] & 0xffff0000u));
        v1[i] = __float_as_uint(__uint_as_float(v1[i]) - __uint_as_float(v1[i] & 0xffff0000u));
      }
    }
  }
}

// 8 float32 as hi + lo, each 8 bf16: the upper halves, and what they lack rounded to nearest; off by 2^-16 of a value at
// most, and exact where it has no more than 16 bits.
__device__ __forceinline__ void split8(u32x4 v0, u32x4 v1, bf16x8 (&out)[2]) {
  u32x4 r;
  r.x = __builtin_amdgcn_perm(v0.y, v0.x, 0x07060302u);
  r.y = __builtin_amdgcn_perm(v0.w, v0.z, 0x07060302u);
  r.z = __builtin_amdgcn_perm(v1.y, v1.x, 0x07060302u);
  r.w = __builtin_amdgcn_perm(v1.w, v1.z, 0x07060302u);
  out[0] = __builtin_bit_cast(bf16x8, r);
  float left[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    left[i] = __uint_as_float(v0[i]) - __uint_as_float(v0[i] & 0xffff0000u);
    left[4 + i] = __uint_as_float(v1[i]) - __uint_as_float(v1[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)left[2 * i], (__bf16)left[2 * i + 1]});
  out[1] = __builtin_bit_cast(bf16x8, r);
}

// 8 consecutive bf16 or float32 at p (16-byte aligned) as float32.
template <typename T>
__device__ __forceinline__ void values8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    const u32x4 b = *(const u32x4*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(b[i]), v[2 * i + 1] = bf16_hi(b[i]);
  } else {
    const f32x4 a = ((const f32x4*)p)[0], b = ((const f32x4*)p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  }
}

__device__ __forceinline__ bf16x8 zero8() { return __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0}); }

// bf16 parts of a type's values: what a value is the exact sum of.
template <typename T> struct Parts;
template <> struct Parts<uint16_t> { static constexpr int n = 1; };
template <> struct Parts<float> { static constexpr int n = 3; };

// 8 consecutive values at p (16-byte aligned) as operands.
__device__ __forceinline__ void load8(const uint16_t* p, bf16x8 (&out)[1]) { out[0] = *(const bf16x8*)p; }
__device__ __forceinline__ void load8(const float* p, bf16x8 (&out)[3]) {
  split8(((const u32x4*)p)[0], ((const u32x4*)p)[1], out);
}
// 8 values already in registers.
__device__ __forceinline__ void pack8(const uint16_t (&v)[8], bf16x8 (&out)[1]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)v[2 * i] | (uint32_t)v[2 * i + 1] << 16;
  out[0] = __builtin_bit_cast(bf16x8, r);
}
__device__ __forceinline__ void pack8(const float (&v)[8], bf16x8 (&out)[3]) {
  u32x4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = __float_as_uint(v[i]), b[i] = __float_as_uint(v[4 + i]);
  split8(a, b, out);
}

// 16 bytes at an address that is a multiple of the element's size only (global loads take any).
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
__device__ __forceinline__ void load8_any(const uint16_t* p, bf16x8 (&out)[1]) {
  out[0] = __builtin_bit_cast(bf16x8, (u32x4) * (const u32x4_at2*)p);
}
__device__ __forceinline__ void load8_any(const float* p, bf16x8 (&out)[3]) {
  split8(*(const u32x4_at4*)p, *(const u32x4_at4*)(p + 4), out);
}

// 8 consecutive values of a row at d, zeros from D on or where the row is not real.
template <typename TX>
__device__ __forceinline__ void row8(const TX* row, int64_t d, int64_t D, bool real, bf16x8 (&out)[Parts<TX>::n]) {
  if (real && d + 8 <= D) {
    load8_any(row + d, out);
  } else {
    TX v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = real && d + i < D ? row[d + i] : (TX)0;
    pack8(v, out);
  }
}

// acc += a b, 16 x 16 with 32 products each, of operands in parts.  The upper
// parts' product goes to acc[0], the others, small and rounded finely, to
// acc[1].  Of two operands in three parts the products mid lo, lo mid and lo lo are left out: the parts
// are cut off, so mid is below 2^-7 of its value and lo below 2^-15, and what is left out is below 2^-21 of the whole
// product (2^-24 on average) and has its sign.
template <int PA, int PB>
__device__ __forceinline__ void mfma_parts(const bf16x8 (&a)[PA], const bf16x8 (&b)[PB], f32x4 (&acc)[2]) {
#pragma unroll
  for (int i = 0; i < PA; ++i)
#pragma unroll
    for (int j = 0; j < PB; ++j)
      if (i + j < 3) {
        f32x4& d = acc[i + j == 0 ? 0 : 1];
        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], d, 0, 0, 0);
      }
}

// The sum over the ranks of low[r] out[r] for one row and one column, both of
// `rank` values (a multiple of 8) at 16-byte aligned addresses.
__device__ __forceinline__ float rank_dot(const float* low, const void* out, int64_t at, int rank, int wide) {
  float v = 0.0f;
  if (wide) {
    const float* b = (const float*)out + at;
    for (int r = 0; r < rank; r += 4) {
      const f32x4 l = *(const f32x4*)(low + r), c = *(const f32x4*)(b + r);
#pragma unroll
      for (int i = 0; i < 4; ++i) v = fmaf(l[i], c[i], v);
    }
  } else {
    const uint16_t* b = (const uint16_t*)out + at;
    for (int r = 0; r < rank; r += 8) {
      const f32x4 l0 = *(const f32x4*)(low + r), l1 = *(const f32x4*)(low + r + 4);
      const u32x4 c = *(const u32x4*)(b + r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v = fmaf(i < 2 ? l0[2 * i] : l1[2 * i - 4], bf16_lo(c[i]), v);
        v = fmaf(i < 2 ? l0[2 * i + 1] : l1[2 * i - 3], bf16_hi(c[i]), v);
      }
    }
  }
  return v;
}

}  // namespace w4
