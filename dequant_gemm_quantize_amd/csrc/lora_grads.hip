// Gradients of low-rank adapters from the 8-bit checkpoint of x, for every adapter l:
//   da[l, r, k] = sum over the rows m of l of v[m, r] xq[m, k] xs[m, k / 128]
//   db[l, n, r] = sum over the rows m of l of u[m, r] dy[m, n]
// float32, on v_mfma_f32_16x16x32_bf16.  An adapter without rows gets zeros.
//
// The sums run over rows, along which no operand lies together in memory.  A
// lane loads 8 consecutive columns of each of 8 rows and picks pairs out of them
// (32 v_perm for 64 values): the 8 values of one column are the operand of one
// of 8 MFMAs, which has columns 8 l16 + j.  A wave so has 128 columns, one block
// of the checkpoint, whose scale goes to v.  int8 codes are exact bf16 values; the
// low-rank values, and float32 dy, are sums of three bf16 values each.
//
// Bound by reading xq and dy once: 4096 rows of [11008, 4096], rank 16, 25 us for 109 MB, and 4 for the
// parts' sums; 601 rows, float32 dy, rank 64, 15 us, a step or two a wave.  The rows are shared by the waves of a workgroup
// and by `parts` workgroups, whose partial sums a second kernel adds in order.
#include "lora.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int kGWaves = 4;
constexpr int kGCols = 128;  // columns of a workgroup

struct GPlan {
  int rb;  // blocks of 16 ranks a workgroup has
  int64_t strips_k, strips_n, rgroups, parts;
};

GPlan g_plan(int64_t m, int64_t k, int64_t n, int dy_dtype, int64_t count, int rank) {
  GPlan p;
  p.rb = rank <= 16 ? 1 : rank <= 32 || dy_dtype == W4_F32 ? 2 : 4;
  p.strips_k = (k + kGCols - 1) / kGCols;
  p.strips_n = (n + kGCols - 1) / kGCols;
  p.rgroups = (rank + 16 * p.rb - 1) / (16 * p.rb);
  const int64_t groups = (p.strips_k + p.strips_n) * p.rgroups * count;
  int64_t parts = 512 / (groups > 0 ? groups : 1);
  const int64_t most = m / (64 * kGWaves);  // two steps a wave at least
  if (parts > most) parts = most;
  p.parts = parts < 1 ? 1 : parts;
  return p;
}

// 8 consecutive columns of a row, as they are in memory; columns past the end read as zero.
struct RowI8 {
  u32x2 v;
  __device__ __forceinline__ void load(const int8_t* row, int64_t c, int64_t C) {
    v = c < C ? *(const u32x2*)(row + c) : u32x2{0, 0};  // C is a multiple of 32
  }
};
struct RowB16 {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* row, int64_t c, int64_t C) {
    if (c + 8 <= C) {
      v = *(const u32x4_at2*)(row + c);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = c + 2 * i < C ? row[c + 2 * i] : 0, hi = c + 2 * i + 1 < C ? row[c + 2 * i + 1] : 0;
        v[i] = lo | hi << 16;
      }
    }
  }
};
struct RowF32 {
  u32x4 v[2];
  __device__ __forceinline__ void load(const float* row, int64_t c, int64_t C) {
    if (c + 8 <= C) {
      v[0] = *(const u32x4_at4*)(row + c), v[1] = *(const u32x4_at4*)(row + c + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = c + i < C ? __float_as_uint(row[c + i]) : 0;
    }
  }
};
template <typename T> struct RowOf;
template <> struct RowOf<int8_t> { typedef RowI8 type; static constexpr int n = 1; };
template <> struct RowOf<uint16_t> { typedef RowB16 type; static constexpr int n = 1; };
template <> struct RowOf<float> { typedef RowF32 type; static constexpr int n = 3; };

// Column j of 8 rows as an operand.
__device__ __forceinline__ void column(const RowI8 (&t)[8], int j, bf16x8 (&out)[1]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = (float)(int8_t)(t[2 * i].v[j >> 2] >> (8 * (j & 3)));
    const float b = (float)(int8_t)(t[2 * i + 1].v[j >> 2] >> (8 * (j & 3)));
    r[i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
  }
  out[0] = __builtin_bit_cast(bf16x8, r);
}
__device__ __forceinline__ void column(const RowB16 (&t)[8], int j, bf16x8 (&out)[1]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __builtin_amdgcn_perm(t[2 * i + 1].v[j >> 1], t[2 * i].v[j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
  out[0] = __builtin_bit_cast(bf16x8, r);
}
__device__ __forceinline__ void column(const RowF32 (&t)[8], int j, bf16x8 (&out)[3]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(t[i].v[j >> 2][j & 3]);
  pack8(v, out);
}

// One strip of 128 columns of src [M, C] against low [M, R] for the ranks from r0
// and the rows of adapter l that are this part's.  RANK_ROWS: the result is
// [R, C] (ranks are the MFMA's rows), otherwise [C, R].  xs: the scales of an int8 src.
template <typename T, bool RANK_ROWS, int RB>
__device__ __forceinline__ void strip(float* sums, const T* __restrict__ src, const float* __restrict__ xs, int64_t M,
                                      int64_t C, int64_t c0, const float* __restrict__ low, int R, int r0, int l,
                                      const int* __restrict__ offsets, const int* __restrict__ which, int segments,
                                      int part, int parts, float* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, h = lane >> 4;
  const int64_t c = c0 + 8 * l16;
  const int64_t nb = (C + 127) / 128, blk = c0 / 128;
  constexpr int P = RowOf<T>::n;
  f32x4 acc[8][RB];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[j][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // the wave's steps of 32 rows: numbers first, first + stride, .. of the list of all the adapter's steps
  int64_t want = (int64_t)part * kGWaves + w, before = 0;
  const int64_t stride = (int64_t)parts * kGWaves;
  for (int base = 0; base < segments; base += kWave) {
    int row0;
    int rows = group_rows(offsets, segments, (int)M, base, lane, row0);
    if (base + lane >= segments || which[base + lane] != l) rows = 0;
    const int upto = wave_scan((rows + 31) / 32);
    const int64_t after = before + __builtin_amdgcn_readlane(upto, kWave - 1);
    // (Two steps a wave in registers left half as many waves and took 37 us for 4096 rows where one takes 24.)
    struct Step {
      typename RowOf<T>::type t[8];
      float lv[RB][8], s[8];
    };
    auto load = [&](Step& p) {
      const int f = __builtin_ctzll(__ballot(before + upto > want));
      const int begin = __builtin_amdgcn_readlane(row0, f), have = __builtin_amdgcn_readlane(rows, f);
      const int64_t skipped = before + __builtin_amdgcn_readlane(upto - (rows + 31) / 32, f);
      const int64_t m0 = begin + 32 * (want - skipped), end = (int64_t)begin + have;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t m = m0 + 8 * h + i;
        const bool real = m < end;
        const int64_t mm = real ? m : end - 1;  // a row of the segment, times zero
        p.t[i].load(src + mm * C, c, C);
        p.s[i] = sizeof(T) == 1 && real ? xs[mm * nb + blk] : 1.0f;
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const int r = r0 + 16 * b + l16;
          p.lv[b][i] = real && r < R ? low[mm * R + r] : 0.0f;
        }
      }
      want += stride;
    };
    auto compute = [&](const Step& p) {
      bf16x8 lo[RB][3];
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = sizeof(T) == 1 ? p.lv[b][i] * p.s[i] : p.lv[b][i];
        pack8(v, lo[b]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        bf16x8 v[P];
        column(p.t, j, v);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          // the lower parts first; with float32 dy the products mid lo, lo mid and lo lo are left out, below 2^-21 of
          // the whole product (2^-24 on average)
#pragma unroll
          for (int q = 2; q >= 0; --q)
#pragma unroll
            for (int e = P - 1; e >= 0; --e)
              if (q + e < 3)
                acc[j][b] = RANK_ROWS ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo[b][q], v[e], acc[j][b], 0, 0, 0)
                                      : __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[e], lo[b][q], acc[j][b], 0, 0, 0);
        }
      }
    };
    while (want < after) {
      Step p;
      load(p);
      compute(p);
    }
    before = after;
  }

  // register e: MFMA row 4 h + e, column l16
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = acc[j][b][e];
        const int mr = 4 * h + e;
        // [16 ranks][128 columns], or [128 columns][16 ranks]
        sums[w * 16 * kGCols + (RANK_ROWS ? mr * kGCols + 8 * l16 + j : (8 * mr + j) * 16 + l16)] = v;
      }
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * kGCols; o += 64 * kGWaves) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kGWaves; ++i) v += sums[i * 16 * kGCols + o];
      const int64_t col = c0 + (RANK_ROWS ? o % kGCols : o / 16);
      const int r = r0 + 16 * b + (RANK_ROWS ? o / kGCols : o % 16);
      if (col < C && r < R) out[RANK_ROWS ? (int64_t)r * C + col : col * R + r] = v;
    }
  }
}

}  // namespace

// part p of da goes to da + p * pstride, of db to db + p * pstride.
template <typename TD, int RB>
__global__ __launch_bounds__(64 * kGWaves) void k_lora_grads(LoraGrads a, uint32_t strips_k, uint32_t strips, uint32_t rgroups,
                                                             int parts, float* __restrict__ da,
                                                             float* __restrict__ db, int64_t pstride) {
  __shared__ __attribute__((aligned(16))) float sums[kGWaves * 16 * kGCols];
  const uint64_t tiles = (uint64_t)strips * rgroups * (uint64_t)a.count;
  const int part = blockIdx.y;
  for (uint64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const uint32_t st = (uint32_t)(tile % strips);
    const uint64_t rest = tile / strips;
    const int r0 = (int)(rest % rgroups) * 16 * RB, l = (int)(rest / rgroups);
    if (st < strips_k)
      strip<int8_t, true, RB>(sums, a.xq, a.xs, a.m, a.k, (int64_t)kGCols * st, a.v, a.rank, r0, l, a.offsets, a.which,
                              (int)a.segments, part, parts, da + part * pstride + (int64_t)l * a.rank * a.k);
    else
      strip<TD, false, RB>(sums, (const TD*)a.dy, nullptr, a.m, a.n, (int64_t)kGCols * (st - strips_k), a.u, a.rank, r0,
                           l, a.offsets, a.which, (int)a.segments, part, parts,
                           db + part * pstride + (int64_t)l * a.rank * a.n);
    __syncthreads();
  }
}

// out[i] = the sum of the parts, in order; da is the first `na` elements, db the rest.
__global__ __launch_bounds__(256) void k_lora_grads_sum(const float* __restrict__ ws, int parts, int64_t na, int64_t all,
                                                        float* __restrict__ da, float* __restrict__ db) {
  for (int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x); i < all; i += 4 * 256 * (int64_t)gridDim.x) {
    f32x4 v = *(const f32x4*)(ws + i);
    for (int p = 1; p < parts; ++p) v += *(const f32x4*)(ws + (int64_t)p * all + i);
    *(f32x4*)(i < na ? da + i : db + (i - na)) = v;
  }
}

size_t lora_grads_workspace_bytes(int64_t m, int64_t k, int64_t n, int dy_dtype, int64_t count, int rank) {
  const GPlan p = g_plan(m, k, n, dy_dtype, count, rank);
  return p.parts > 1 ? (size_t)p.parts * (size_t)(count * rank * (k + n)) * 4 : 0;
}

template <typename TD, int RB>
static hipError_t grads_go(const LoraGrads& a, const GPlan& p, hipStream_t st) {
  const int64_t strips = p.strips_k + p.strips_n, tiles = strips * p.rgroups * a.count;
  const int64_t na = a.count * a.rank * a.k, all = a.count * a.rank * (a.k + a.n);
  float* da = p.parts > 1 ? (float*)a.ws : a.da;
  float* db = p.parts > 1 ? (float*)a.ws + na : a.db;
  const dim3 grid((unsigned)(tiles < (1 << 20) ? tiles : 1 << 20), (unsigned)p.parts);
  k_lora_grads<TD, RB><<<grid, 64 * kGWaves, 0, st>>>(a, (uint32_t)p.strips_k, (uint32_t)strips, (uint32_t)p.rgroups,
                                                     (int)p.parts, da, db, all);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.parts == 1) return e;
  const int64_t groups = (all / 4 + 255) / 256;
  k_lora_grads_sum<<<dim3((unsigned)(groups < 4096 ? groups : 4096)), 256, 0, st>>>((const float*)a.ws, (int)p.parts,
                                                                                   na, all, a.da, a.db);
  return hipGetLastError();
}

hipError_t launch_lora_grads(const LoraGrads& a, hipStream_t st) {
  const GPlan p = g_plan(a.m, a.k, a.n, a.dy_dtype, a.count, a.rank);
  if (a.dy_dtype == W4_F32) return p.rb == 1 ? grads_go<float, 1>(a, p, st) : grads_go<float, 2>(a, p, st);
  if (p.rb == 4) return grads_go<uint16_t, 4>(a, p, st);
  return p.rb == 1 ? grads_go<uint16_t, 1>(a, p, st) : grads_go<uint16_t, 2>(a, p, st);
}

}  // namespace w4
