// Into the low rank: for the rows of a segment with adapter l,
//   low[m, r] = scaling[l] sum_d x[m, d] W[l, r, d]     (x into A [L, R, K]), or
//   low[m, r] = scaling[l] sum_d x[m, d] W[l, d, r]     (dy into B [L, N, R]),
// float32, on v_mfma_f32_16x16x32_bf16: bf16 values as they are, float32 ones as the
// exact sum of three bf16 values.  Rows of no adapter are left as they were.
//
// A workgroup has 16 rows of one segment and some ranks; its waves go through D in
// turn and add their sums through LDS.  Segments of a row or two (decode) leave
// most of an MFMA's rows empty, and its loads, 16 rows each, with them: they take the
// vector unit, four rows and four ranks a workgroup.
//
// Bound by latency where rows are few, by what a CU takes in from the L2 cache
// where they are many: a wave has all loads of its values under way before it waits.  [11008, 4096]: one row, 16 ranks,
// 4 us; 2048 rows, 64 ranks, 21; dy of 12 rows into 16 ranks 5.
#include "lora.h"
#include "lds_gemm.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int64_t kIntoGrid = 1 << 20;  // workgroups; more tiles than that loop

// The waves' sums, added: part [waves][rows][ranks] -> low.
template <int BM, int RANKS>
__device__ __forceinline__ void into_store(const float* part, int waves, const SegmentTile& t, int rank0, int R,
                                           float c, float* low) {
  for (int o = threadIdx.x; o < t.rows * RANKS; o += blockDim.x) {
    const int row = o / RANKS, q = o % RANKS;
    if (rank0 + q >= R) continue;
    float v = 0.0f;
#pragma unroll 8
    for (int i = 0; i < waves; ++i) v += part[(i * BM + row) * RANKS + q];
    low[(t.m0 + row) * R + rank0 + q] = c * v;
  }
}

}  // namespace

// x into A, 16 RB ranks a workgroup.
constexpr int kDownWaves = 16;
// The same for tiles of up to four rows, four ranks a workgroup: a lane has 8 values of D of
// each, on the vector unit, so every load is 1 KB (2 KB) of one row.
constexpr int kFewWaves = 8;
template <int ROWS, typename TX, typename TW>
__device__ __forceinline__ void few_rows(const TX* x, int64_t D, const TW* weights, int w, int lane, float* part) {
  float acc[ROWS][4];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
  for (int64_t d = 512 * w + 8 * lane; d < D; d += 512 * kFewWaves) {
    float wv[4][8], xv[ROWS][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) values8(weights + j * D + d, wv[j]);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) values8(x + i * D + d, xv[i]);
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][j] = fmaf(xv[i][e], wv[j][e], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = wave_sum<64>(acc[i][j]);
      if (lane == 0) part[(w * 4 + i) * 4 + j] = v;
    }
}

template <typename TX, typename TW>
__global__ __launch_bounds__(64 * kFewWaves) void k_lora_down_few(
    const TX* __restrict__ x, int64_t M, int64_t D, const TW* __restrict__ weights, int count, int R,
    const float* __restrict__ scaling, const int* __restrict__ offsets, const int* __restrict__ which, int segments,
    float* __restrict__ low, uint32_t rblocks, int64_t tiles) {
  __shared__ float part[kFewWaves * 16];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    SegmentTile t;
    if (!find_segment_tile(offsets, which, segments, count, (int)M, 4, rblocks, tile, lane, t)) return;
    if (t.adapter < 0) continue;
    const int rank0 = 4 * (int)t.side;  // R is a multiple of 8
    const float c = scaling[t.adapter];
    const TX* xt = x + t.m0 * D;
    const TW* wt = weights + ((int64_t)t.adapter * R + rank0) * D;
    if (t.rows == 1) few_rows<1>(xt, D, wt, w, lane, part);
    else if (t.rows == 2) few_rows<2>(xt, D, wt, w, lane, part);
    else if (t.rows == 3) few_rows<3>(xt, D, wt, w, lane, part);
    else few_rows<4>(xt, D, wt, w, lane, part);
    __syncthreads();
    into_store<4, 4>(part, kFewWaves, t, rank0, R, c, low);
    __syncthreads();  // the next tile writes part again
  }
}

template <int RB, typename TX, typename TW>
__global__ __launch_bounds__(64 * kDownWaves) void k_lora_down(
    const TX* __restrict__ x, int64_t M, int64_t D, const TW* __restrict__ weights, int count, int R,
    const float* __restrict__ scaling, const int* __restrict__ offsets, const int* __restrict__ which, int segments,
    float* __restrict__ low, uint32_t rblocks, int64_t tiles) {
  constexpr int RANKS = 16 * RB;
  // values of D that a wave loads at a time: what its registers hold
  constexpr int LB = (int)sizeof(TX) + RB * (int)sizeof(TW), CK = LB <= 4 ? 256 : LB <= 8 ? 128 : LB < 12 ? 64 : 32;
  extern __shared__ __attribute__((aligned(16))) float part[];  // [waves][16][RANKS]
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, h = lane >> 4;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    SegmentTile t;
    if (!find_segment_tile(offsets, which, segments, count, (int)M, 16, rblocks, tile, lane, t)) return;
    if (t.adapter < 0) continue;
    const int rank0 = RANKS * (int)t.side;
    const float c = scaling[t.adapter];
    // rows and ranks past the end repeat the last: nobody stores what they give
    const TX* xp = x + (t.m0 + (l16 < t.rows ? l16 : t.rows - 1)) * D + 8 * h;
    const TW* wp[RB];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int r = rank0 + 16 * i + l16;
      wp[i] = weights + ((int64_t)t.adapter * R + (r < R ? r : R - 1)) * D + 8 * h;
    }
    f32x4 acc[RB][2];
#pragma unroll
    for (int j = 0; j < RB; ++j) acc[j][0] = acc[j][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto slices = [&](int64_t d0, auto count_c) {
      constexpr int n = decltype(count_c)::value;
      bf16x8 a[n][Parts<TX>::n], b[n][RB][Parts<TW>::n];
#pragma unroll
      for (int q = 0; q < n; ++q) {
#pragma unroll
        for (int j = 0; j < RB; ++j) load8(wp[j] + d0 + 32 * q, b[q][j]);
        load8(xp + d0 + 32 * q, a[q]);
      }
      __builtin_amdgcn_sched_barrier(0);  // every load is on its way before the first is waited for
#pragma unroll
      for (int q = 0; q < n; ++q)
#pragma unroll
        for (int j = 0; j < RB; ++j) mfma_parts(a[q], b[q][j], acc[j]);
    };
    for (int64_t d0 = CK * w; d0 < D; d0 += CK * kDownWaves) {
      if (d0 + CK <= D) {
        slices(d0, std::integral_constant<int, CK / 32>{});
      } else {
        for (int64_t d = d0; d < D; d += 32) slices(d, std::integral_constant<int, 1>{});
      }
    }
    // lane holds rows 4 h + e of rank l16
#pragma unroll
    for (int j = 0; j < RB; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[(w * 16 + 4 * h + e) * RANKS + 16 * j + l16] = acc[j][0][e] + acc[j][1][e];
    __syncthreads();
    into_store<16, RANKS>(part, kDownWaves, t, rank0, R, c, low);
    __syncthreads();  // the next tile writes part again
  }
}

// dy into B, 16 rows and 16 ranks a workgroup.  The sum runs over rows of B, so an
// operand's 8 values are a column of it: B goes from memory to the wave's own place in LDS,
// 2 or 4 KB at a time, and is read from there value by value; row n of 32 is at place
// 4 (n % 8) + n / 8, which puts the four rows that a read meets beside each other, on
// all banks once.  dy takes the same way where its rows start at 16-byte addresses
// (piece c of row m at slot c ^ m, modulo the row's pieces).  (Loads of single values of B from memory, 16
// lanes an address pass, took 77 us for 12 rows against [11008, 16].)
constexpr int kUpWaves = 8;
template <typename TX, typename TW> struct UpPlace {
  static constexpr int CH = sizeof(TX) + sizeof(TW) > 4 ? 64 : 128;  // rows of B a step
  static constexpr int WB = 16 * CH * (int)sizeof(TW), XB = 16 * CH * (int)sizeof(TX);  // bytes of B and of 16 rows of dy
  static constexpr int STAGE = WB + XB;
  static constexpr size_t lds = 2 * (size_t)kUpWaves * STAGE;
};
template <typename TX, typename TW, bool WIDE>
__global__ __launch_bounds__(64 * kUpWaves) void k_lora_up(
    const TX* __restrict__ x, int64_t M, int64_t D, const TW* __restrict__ weights, int count, int R,
    const float* __restrict__ scaling, const int* __restrict__ offsets, const int* __restrict__ which, int segments,
    float* __restrict__ low, uint32_t rblocks, int64_t tiles, int64_t part_d) {
  typedef UpPlace<TX, TW> P;
  constexpr int CH = P::CH, Q = CH / 32;
  constexpr int XC = CH * (int)sizeof(TX) / 16;          // 16-byte pieces of a row of dy
  constexpr int XL = P::XB / 1024, WL = P::WB / 1024;    // loads of dy and B a step
  constexpr int PX = Parts<TX>::n, PW = Parts<TW>::n, LOADS = WL + (WIDE ? XL : 0);
  extern __shared__ __attribute__((aligned(1024))) uint8_t su[];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, h = lane >> 4;
  uint8_t* mine = su + w * 2 * P::STAGE;
  float* part = (float*)su;  // [waves][16][16], when the places are done with
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    SegmentTile t;
    if (!find_segment_tile(offsets, which, segments, count, (int)M, 16, rblocks, tile, lane, t)) return;
    if (t.adapter < 0) continue;
    const int rank0 = 16 * (int)t.side;
    const float c = scaling[t.adapter];
    const TW* wl = weights + (int64_t)t.adapter * D * R;
    const TX* xt = x + t.m0 * D;
    const uint32_t xrow = (uint32_t)(D * (int64_t)sizeof(TX)), wrow = (uint32_t)R * (uint32_t)sizeof(TW);
    const __amdgpu_buffer_rsrc_t xr = buf_rsrc_n(uniform_ptr(xt), (uint32_t)t.rows * xrow);
    constexpr int SL = (int)sizeof(TW);  // 16-byte pieces of a row's 16 ranks
    auto issue = [&](int64_t d0, int stage) {
      uint8_t* place = mine + stage * P::STAGE;
      const int64_t have = d0 < D ? (D - d0 < CH ? D - d0 : CH) : 0;
      const __amdgpu_buffer_rsrc_t wr = buf_rsrc_n(uniform_ptr(wl + (d0 < D ? d0 : 0) * R), (uint32_t)have * wrow);
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        const int s = 64 * i + lane, p = s / SL, piece = s % SL;
        const int n = (p & 31) / 4 + 8 * (p & 3) + (p & ~31);
        const bool in = rank0 + piece * (16 / (int)sizeof(TW)) < R;
        load_lds(wr, place + 1024 * i,
                 in ? (uint32_t)n * wrow + (uint32_t)rank0 * (uint32_t)sizeof(TW) + 16u * piece : kPastEnd);
      }
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < XL; ++i) {
          const int s = 64 * i + lane, row = s / XC, piece = (s % XC) ^ (row & (XC - 1));
          const bool in = d0 + (int64_t)piece * (16 / (int)sizeof(TX)) < D;
          load_lds(xr, place + P::WB + 1024 * i,
                   in ? (uint32_t)row * xrow + (uint32_t)(d0 * (int64_t)sizeof(TX)) + 16u * piece : kPastEnd);
        }
      }
    };
    f32x4 acc[2];
    acc[0] = acc[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // this part's values of D, and of those this wave's
    constexpr int64_t stride = CH * kUpWaves;
    const int64_t begin = part_d * blockIdx.y + (int64_t)CH * w, end = D - part_d * blockIdx.y < part_d ? D : part_d * (blockIdx.y + 1);
    int stage = 0;
    if (begin < end) issue(begin, 0);
    for (int64_t d0 = begin; d0 < end; d0 += stride, stage ^= 1) {
      issue(d0 + stride < end ? d0 + stride : D, stage ^ 1);  // past D nothing, as many loads
      bf16x8 a[Q][PX];
      if constexpr (!WIDE) {
#pragma unroll
        for (int q = 0; q < Q; ++q) row8(xt + (l16 < t.rows ? l16 : 0) * D, d0 + 32 * q + 8 * h, D, true, a[q]);
      }
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
      const uint8_t* place = mine + stage * P::STAGE;
      if constexpr (WIDE) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          constexpr int per = (int)sizeof(TX) / 2;  // pieces of 8 values
          u32x4 v[per];
#pragma unroll
          for (int i = 0; i < per; ++i)
            v[i] = *(const u32x4*)(place + P::WB + 16 * (XC * l16 + ((per * (4 * q + h) + i) ^ (l16 & (XC - 1)))));
          if constexpr (per == 1) a[q][0] = __builtin_bit_cast(bf16x8, v[0]);
          else split8(v[0], v[1], a[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        TW v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = ((const TW*)place)[16 * (32 * q + 4 * i + h) + l16];
        bf16x8 b[PW];
        pack8(v, b);
        mfma_parts(a[q], b, acc);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the place is written again
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) part[(w * 16 + 4 * h + e) * 16 + l16] = acc[0][e] + acc[1][e];
    __syncthreads();
    into_store<16, 16>(part, kUpWaves, t, rank0, R, c, low + (int64_t)blockIdx.y * M * R);
    __syncthreads();  // the next tile writes there again
  }
}

template <int RB, typename TX, typename TW>
static hipError_t down_go(const LoraInto& a, hipStream_t st) {
  constexpr size_t lds = (size_t)kDownWaves * 16 * 16 * RB * 4;  // at most 64 KB
  const int64_t rblocks = (a.rank + 16 * RB - 1) / (16 * RB);
  const int64_t tiles = grouped_max_tiles(a.m, a.segments, 16) * rblocks;
  k_lora_down<RB, TX, TW><<<dim3((unsigned)(tiles < kIntoGrid ? tiles : kIntoGrid)), 64 * kDownWaves, lds, st>>>(
      (const TX*)a.x, a.m, a.d, (const TW*)a.weights, (int)a.count, a.rank, a.scaling, a.offsets, a.which,
      (int)a.segments, a.low, (uint32_t)rblocks, tiles);
  return hipGetLastError();
}

template <typename TX, typename TW>
static hipError_t few_go(const LoraInto& a, hipStream_t st) {
  const int64_t rblocks = a.rank / 4, tiles = grouped_max_tiles(a.m, a.segments, 4) * rblocks;
  k_lora_down_few<TX, TW><<<dim3((unsigned)(tiles < kIntoGrid ? tiles : kIntoGrid)), 64 * kFewWaves, 0, st>>>(
      (const TX*)a.x, a.m, a.d, (const TW*)a.weights, (int)a.count, a.rank, a.scaling, a.offsets, a.which,
      (int)a.segments, a.low, (uint32_t)rblocks, tiles);
  return hipGetLastError();
}

template <typename TX, typename TW, bool WIDE>
static hipError_t up_go(const LoraInto& a, hipStream_t st) {
  static std::atomic<uint64_t> attr_done{0};  // LDS above the 64 KB default
  constexpr size_t lds = UpPlace<TX, TW>::lds;
  const hipError_t e = once_per_device(attr_done, [] {
    return hipFuncSetAttribute((const void*)k_lora_up<TX, TW, WIDE>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  });
  if (e != hipSuccess) return e;
  const int64_t rblocks = (a.rank + 15) / 16;
  const int64_t tiles = grouped_max_tiles(a.m, a.segments, 16) * rblocks;
  const int64_t parts = a.parts > 1 ? a.parts : 1, chunks = (a.d + 127) / 128;
  const dim3 grid((unsigned)(tiles < kIntoGrid ? tiles : kIntoGrid), (unsigned)parts);
  k_lora_up<TX, TW, WIDE><<<grid, 64 * kUpWaves, lds, st>>>(
      (const TX*)a.x, a.m, a.d, (const TW*)a.weights, (int)a.count, a.rank, a.scaling, a.offsets, a.which,
      (int)a.segments, a.low, (uint32_t)rblocks, tiles, 128 * ((chunks + parts - 1) / parts));
  return hipGetLastError();
}

template <typename TX, typename TW>
static hipError_t into_types(const LoraInto& a, hipStream_t st) {
  if (a.down) {
    // A CU takes in about 40 KB a us from the L2 cache, whatever the kernel, so the
    // tile is the one whose rounds of 256 workgroups read the least: rows and ranks, D values each.  (us
    // for 2048 rows of nine segments, D 4096, 64 ranks in blocks of 16, 32 and 64: 28, 27 and 21.)
    auto rounds = [&](int rows, int ranks) {
      const int64_t tiles = grouped_max_tiles(a.m, a.segments, rows) * ((a.rank + ranks - 1) / ranks);
      return (tiles + 255) / 256 * (rows + ranks);
    };
    const int64_t few = rounds(4, 4), r1 = rounds(16, 16), r2 = rounds(16, 32), r4 = rounds(16, 64);
    if (5 * few <= 4 * r1 && 5 * few <= 4 * r2 && 5 * few <= 4 * r4) return few_go<TX, TW>(a, st);
    if (r1 <= r2 && r1 <= r4) return down_go<1, TX, TW>(a, st);
    return r2 <= r4 ? down_go<2, TX, TW>(a, st) : down_go<4, TX, TW>(a, st);
  }
  // 16 rows of dy by byte offsets below 2^31
  if (a.d * (int64_t)sizeof(TX) % 16 == 0 && a.d * (int64_t)sizeof(TX) < ((int64_t)1 << 27)) return up_go<TX, TW, true>(a, st);
  return up_go<TX, TW, false>(a, st);
}

// Few tiles leave most CUs idle, and a CU's intake is what bounds them (12 rows of three segments against [11008, 16]:
// 12 us in one part, 5 in ten): parts of 1024 values, one step a wave, on at most 128 CUs.
size_t lora_into_parts(int64_t m, int64_t d, int64_t segments, int rank) {
  const int64_t tiles = grouped_max_tiles(m, segments, 16) * ((rank + 15) / 16);
  int64_t parts = tiles > 0 ? 128 / tiles : 1;
  if (parts > d / 1024) parts = d / 1024;
  if (parts > 16) parts = 16;
  return (size_t)(parts < 1 ? 1 : parts);
}

hipError_t launch_lora_into(const LoraInto& a, hipStream_t st) {
  if (a.x_dtype == W4_F32)
    return a.w_dtype == W4_F32 ? into_types<float, float>(a, st) : into_types<float, uint16_t>(a, st);
  return a.w_dtype == W4_F32 ? into_types<uint16_t, float>(a, st) : into_types<uint16_t, uint16_t>(a, st);
}

}  // namespace w4
