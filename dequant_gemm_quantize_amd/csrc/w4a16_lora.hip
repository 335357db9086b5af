// W4A16 products with low-rank adapters, x W^T forward and dy W back: the choice of
// a kernel, the kernel for few rows back, and the sum of split products.
//
// Forward, few rows and float32 x take the few-row kernel (w4a16_lora_rows.hip), many
// rows of bf16 x the product's by expert (w4a16_lora_gemm.hip).
// Back, few rows and float32 dy take k_w4a16_back_rows, on v_mfma_f32_16x16x32_bf16.  A wave has
// 256 columns of 16 MB rows of dx and goes through N 32 weight rows at a time.
// The sum runs over weight rows, the codes of a word over columns: lane (l16,
// h) loads 16 codes (8 bytes) of each of rows 8 h .. 8 h + 7, and the eight
// values of one column, one out of each word, are the operand of one of 16 MFMAs, whose 16
// columns are 16 l16 + j.  So nothing is transposed in memory or LDS.  The waves of
// a workgroup and the workgroups of a strip share N; the partial sums, float32, meet
// in LDS and in the workspace, where k_w4a16_sum adds them in order, and the low-rank part.  12 rows of
// [11008, 4096]: 18 us and 5, the first loads 6 of them, the rest about five vector instructions a code, of which
// half make the two bf16 parts of a weight (one, rounded to bf16: 16 us).
//
// Back, many rows of bf16 dy take tiles (w4a16_tiles.h).  Both products of many rows split the
// sum where the tiles are few.
//
// Rounding: forward none of a weight.  Back, a weight is the sum of bf16 parts: two with fp16 scales
// (15 bits, so exact) and for a bf16 result of bf16 dy (16 bits, off by 2^-16 at most beside
// the result's 2^-8), otherwise three (24 bits).
#include "lds_gemm.h"
#include "lora.h"
#include "w4_internal.h"

namespace w4 {

namespace {

constexpr int kTWaves = 8;
constexpr int kTStrip = 256;  // columns of a workgroup
constexpr int64_t kTGrid = 1 << 20;  // workgroups of a part; more tiles than that loop
constexpr int64_t kTSumGrid = 1 << 22;

// How a call is computed: in tiles (w4a16_lora_gemm.hip, w4a16_tiles.h) or by a kernel for few rows, and
// how it splits the sum: parts of `steps` steps of 256 columns forward, of 64 weight rows in tiles back, of 32 otherwise.
struct LoraPlan {
  bool tiles;
  int mi, pw;          // tiles of 32 mi rows forward, 64 mi back; bf16 parts of a weight (back)
  int mb;              // blocks of 16 rows a workgroup of k_w4a16_back_rows
  int64_t rows, strips, parts, steps;
  int64_t pad;         // > 0: dy is copied into rows of as many values first
  size_t sums, bytes;  // of the partial sums in the workspace, and of all of it
};

void split(LoraPlan& p, int64_t all, int64_t parts) {
  if (parts < 1) parts = 1;
  p.steps = (all + parts - 1) / parts;
  p.parts = (all + p.steps - 1) / p.steps;
}

LoraPlan lora_plan(bool back, int64_t m, int64_t k, int64_t n, int g, int x_dtype, int sz_dtype, int y_dtype) {
  const bool whole = x_dtype != W4_BF16 || y_dtype != W4_BF16;  // weights of float32 scales keep all their bits
  LoraPlan p{};
  p.pw = whole && sz_dtype == W4_F32 ? 3 : 2;
  p.parts = 1;
  if (!back) {
    // us of the few-row kernel / tiles, one request: [4096, 11008] 65 rows 52 / 35, 128 rows 63 / 39; [11008, 4096] 65 rows
    // 51 / 33; [4096, 4096] 128 rows 33 / 28, 200 rows 57 / 32; [2050, 2048] 300 rows 29 / 30, 500 rows 40 / 30.
    // (The few-row kernel adds the adapters of requests of one row faster.)  128 rows of x stay below 2^31 bytes.
    p.tiles = x_dtype == W4_BF16 && m > 64 && m * n * k > ((int64_t)1 << 31) && k <= ((int64_t)1 << 21);
    if (!p.tiles) return p;
    p.strips = (n + 127) / 128;
    // us with 64 / 128 rows a tile, each with its best parts: [4096, 4096] 200 rows 32 / 36, 600 rows 56 / 55; [2050, 2048] 500
    // rows 30 / 37; [4096, 11008] 333 rows 67 / 68; [11008, 4096] 1024 rows 143 / 137, 2048 rows 247 / 241.  (A launch has fewer than
    // 2^32 threads.)
    p.mi = m > 512 || (m + 63) / 64 * p.strips >= (1 << 24) - 8 ? 4 : 2;
    p.rows = (m + 32 * p.mi - 1) / (32 * p.mi);
    // Parts of 1024 columns at least, so many that a CU has its two or three workgroups; two parts gain less
    // than their sum costs.  us in one, two and four parts: 65 rows of [11008, 4096] 39, 35 and 32; [4096, 4096] 333
    // rows 42, 38 and 39, 1024 rows 61, 64 and 76; [2050, 2048] 500 rows 30, 35 and 33.
    const int64_t all = (k + 255) / 256, room = (p.mi == 4 ? 512 : 768) / (p.rows * p.strips);
    const int64_t parts = room < all / 4 ? room : all / 4;
    split(p, all, parts < 3 ? 1 : parts);
    p.bytes = p.sums = p.parts == 1 ? 0 : (size_t)p.parts * (size_t)m * (size_t)n * 4;
    return p;
  }
  // 256 rows of dy, and 64 of codes and scales, stay below 2^31 bytes; an even number of fp16 scales.  us of the few-row
  // kernel / tiles: [11008, 4096] 32 rows 27 / 29, 48 rows 34 / 30; [4096, 11008] 32 rows 27 / 36, 48 rows 41 / 38;
  // [4096, 4096] 24 rows 16 / 17, 48 rows 20 / 19.  Where rows of dy do not start at 16-byte addresses they are copied
  // into ones that do, 4 to 8 us more: [11001, 4096] 64 rows 34 / 38, 65 rows 47 / 38, 2048 rows 620 / 317; [4095, 4096] 64 rows
  // 22 / 25, 128 rows 29 / 30, 333 rows 72 / 44; [2050, 2048] 128 rows 18 / 21, 333 rows 28 / 27; [9010, 256] 200 rows 19 / 30;
  // [1500, 1024] 1000 rows 27 / 29.
  const bool aligned = n % 8 == 0;
  const bool many = aligned ? m > 32 : m > 64 && m * n * k > ((int64_t)3 << 29);
  p.tiles = x_dtype == W4_BF16 && many && n <= ((int64_t)1 << 21) &&
            (sz_dtype == W4_F32 || n * (k / g) % 2 == 0);
  // us in tiles of 128 / 256 rows: [11008, 4096] 100 rows 34 / 41, 200 rows 52 / 46, 2048 rows 358 / 266; [4096, 4096] 128
  // rows 25 / 29, 256 rows 29 / 30, 333 rows 40 / 37; [4096, 11008] 333 rows 120 / 77 (600 rows, where the larger ones need a
  // second round for two tiles, 124 / 167).  Three parts of a weight leave room for the smaller ones only.
  p.mi = p.pw == 3 || m <= 128 ? 2 : 4;
  p.rows = (m + 64 * p.mi - 1) / (64 * p.mi);
  p.strips = (k + 127) / 128;
  if (p.rows * p.strips > (1 << 22)) p.tiles = false;  // a launch has fewer than 2^32 threads
  if (p.tiles) {
    const int64_t all = (n + 63) / 64, parts = 256 / (p.rows * p.strips);
    split(p, all, parts < all / 8 ? parts : all / 8);
    p.sums = p.parts == 1 ? 0 : (size_t)p.parts * (size_t)m * (size_t)k * 4;
    p.pad = aligned ? 0 : (n + 7) / 8 * 8;
    p.bytes = p.sums + ((size_t)m * (size_t)p.pad * 2 + 127) / 128 * 128;
  } else {
    p.strips = (k + kTStrip - 1) / kTStrip;
    // a workgroup a CU; two steps a wave at least, for the partial sums cost as much as
    // the codes with 16 rows and 44 parts of [11008, 4096]
    const int64_t all = (n + 31) / 32, most = (all + 2 * kTWaves - 1) / (2 * kTWaves);
    // Two blocks of 16 rows a workgroup where those fill the CUs: us with one / two, 32 rows of [11008, 4096] 28 / 27, [4096,
    // 11008] 35 / 27, [4096, 4096] 16 / 19; 128 rows of [2050, 2048] 18 / 19, 333 rows 35 / 28, of [11001, 4096] 255 / 162.
    const bool two = x_dtype == W4_BF16 && p.pw == 2 && m > 16 && (m + 31) / 32 * p.strips * most >= 256;
    p.mb = two ? 2 : 1;
    p.rows = (m + 16 * p.mb - 1) / (16 * p.mb);
    const int64_t parts = 256 / (p.rows * p.strips);
    split(p, all, parts < most ? parts : most);
    p.bytes = p.sums = (size_t)p.parts * (size_t)m * (size_t)k * 4;
  }
  return p;
}

}  // namespace

// PW: bf16 parts of a weight.
template <typename TX, typename TS, int PW, int MB>
__global__ __launch_bounds__(64 * kTWaves, 2) void k_w4a16_back_rows(
    const TX* __restrict__ dy, int64_t M, int64_t N, const uint8_t* __restrict__ packed,
    const void* __restrict__ scales, const void* __restrict__ zeros, int64_t K, int g, int steps,
    float* __restrict__ part) {
  constexpr int PX = Parts<TX>::n;
  constexpr int NA = MB == 1 ? 2 : 1;  // sums: the upper parts' and the others', or of both (registers)
  extern __shared__ __attribute__((aligned(16))) float sums[];  // [waves / 2][16][256], then the waves' scales
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, h = lane >> 4;
  float* mine = sums + kTWaves / 2 * 16 * kTStrip + w * 512;  // [scales, zero-points][groups of the strip][32 rows]
  const int64_t strips = (K + kTStrip - 1) / kTStrip, tiles = strips * ((M + 16 * MB - 1) / (16 * MB));
  const int64_t ng = K / g, half = K / 2;
  const int64_t all = (N + 31) / 32, first = (int64_t)steps * blockIdx.y;
  const int64_t last = first + steps < all ? first + steps : all;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t k0 = kTStrip * (tile % strips), m0 = 16 * MB * (tile / strips);
    const int64_t col = k0 + 16 * l16;
    const int64_t cc = col < K ? col : k0;  // lanes past K compute what nobody stores
    // The strip's groups, eight at most.  One value a lane, 64 at a time: loaded where they are
    // used, 16 loads of which 16 lanes get the same, they took longer than the codes.
    const int64_t g0 = k0 / g, g1 = ((k0 + kTStrip < K ? k0 + kTStrip : K) - 1) / g;
    const int values = 32 * (int)(g1 - g0 + 1), mygroup = (int)(cc / g - g0);

    f32x4 acc[MB][16][NA];
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int a = 0; a < NA; ++a) acc[b][j][a] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    struct Step {
      u32x2 p[8];
      uint32_t s[4], z[4];
      bf16x8 a[MB][PX];
    };
    // 32-bit offsets from a step's first weight row; rows past the last read as zero
    const uint32_t po = (uint32_t)(8 * h) * (uint32_t)half + (uint32_t)(cc / 2);
    uint32_t so[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int v = lane + 64 * i;
      so[i] = ((uint32_t)(v & 31) * (uint32_t)ng + (uint32_t)g0 + (v < values ? v >> 5 : 0)) * (uint32_t)sizeof(TS);
    }
    const TX* dyp = dy + (m0 + l16 < M ? m0 + l16 : M - 1) * N;
    auto load = [&](int64_t st, Step& r) {
      const int64_t n0 = st < last ? 32 * st : N;  // steps past the last: nothing
      const uint32_t have = (uint32_t)(N - n0 < 32 ? N - n0 : 32);
      const __amdgpu_buffer_rsrc_t pr = buf_rsrc_n(uniform_ptr(packed + n0 * half), have * (uint32_t)half);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        r.p[i] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(pr, po + i * (uint32_t)half, 0, 0));
      const uint32_t bytes = have * (uint32_t)ng * (uint32_t)sizeof(TS);
      const int64_t at = n0 * ng * (int64_t)sizeof(TS);
      const __amdgpu_buffer_rsrc_t sr = buf_rsrc_n(uniform_ptr((const char*)scales + at), bytes);
      const __amdgpu_buffer_rsrc_t zr = buf_rsrc_n(uniform_ptr((const char*)zeros + at), bytes);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (64 * i >= values) break;  // the same in every lane
        if constexpr (sizeof(TS) == 2) {
          r.s[i] = __builtin_amdgcn_raw_buffer_load_b16(sr, so[i], 0, 0);
          r.z[i] = __builtin_amdgcn_raw_buffer_load_b16(zr, so[i], 0, 0);
        } else {
          r.s[i] = __builtin_amdgcn_raw_buffer_load_b32(sr, so[i], 0, 0);
          r.z[i] = __builtin_amdgcn_raw_buffer_load_b32(zr, so[i], 0, 0);
        }
      }
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const int64_t m = m0 + 16 * b + l16;
        row8(MB == 1 ? dyp : dy + (m < M ? m : 0) * N, n0 + 8 * h, N, m < M, r.a[b]);
      }
    };
    auto value = [](uint32_t v) {
      if constexpr (sizeof(TS) == 2) return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
      else return __uint_as_float(v);
    };
    auto compute = [&](const Step& r) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (64 * i >= values) break;
        mine[lane + 64 * i] = value(r.s[i]), mine[256 + lane + 64 * i] = value(r.z[i]);
      }
      __builtin_amdgcn_wave_barrier();  // LDS operations of a wave complete in order
      const float* sp = mine + 32 * mygroup + 8 * h;
      const f32x4 s0 = *(const f32x4*)sp, s1 = *(const f32x4*)(sp + 4);
      f32x4 z0 = *(const f32x4*)(sp + 256), z1 = *(const f32x4*)(sp + 260);
      __builtin_amdgcn_wave_barrier();
      if constexpr (PW == 2) {  // -zp s: exact with fp16 scales, 11 bits times 11
#pragma unroll
        for (int i = 0; i < 4; ++i) z0[i] *= -s0[i], z1[i] *= -s1[i];
      }
      uint32_t lo[8], hi[8];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (j % 8 == 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            lo[i] = r.p[i][j >> 3] & 0x0f0f0f0fu;
            hi[i] = (r.p[i][j >> 3] >> 4) & 0x0f0f0f0fu;
            asm("" : "+v"(lo[i]), "+v"(hi[i]));  // no instruction: bytes are converted in place, not masked again
          }
        }
        u32x4 v0, v1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float q = (float)(uint8_t)((j & 1 ? hi : lo)[i] >> (8 * (j >> 1 & 3)));
          const float s = i < 4 ? s0[i] : s1[i - 4], z = i < 4 ? z0[i] : z1[i - 4];
          const float v = PW == 2 ? fmaf(q, s, z) : (q - z) * s;
          if (i < 4) v0[i] = __float_as_uint(v);
          else v1[i - 4] = __float_as_uint(v);
        }
        bf16x8 b[PW];
        split8(v0, v1, b);
        if constexpr (NA == 2) {
          mfma_parts(r.a[0], b, acc[0][j]);
        } else {
#pragma unroll
          for (int p = PW - 1; p >= 0; --p)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
              acc[mb][j][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(r.a[mb][0], b[p], acc[mb][j][0], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);  // one column's values at a time: registers
      }
    };
    for (int64_t st = first + w; st < last; st += kTWaves) {
      Step r;
      load(st, r);
      asm volatile("" ::: "memory");
      compute(r);
    }

    // register e: row 4 h + e, columns 16 l16 + j.  The upper four waves' sums go to
    // LDS, the lower four add their own, and all threads add the four.
    float* out = part + (int64_t)blockIdx.y * M * K;
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      float* place = sums + (w & (kTWaves / 2 - 1)) * 16 * kTStrip + 4 * h * kTStrip + 16 * l16;
      auto sum4 = [&](int e, int j) {
        f32x4 v;
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = NA == 1 ? acc[b][j + t][0][e] : acc[b][j + t][0][e] + acc[b][j + t][NA - 1][e];
        return v;
      };
      __syncthreads();
      if (w >= kTWaves / 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < 16; j += 4) *(f32x4*)(place + e * kTStrip + j) = sum4(e, j);
      }
      __syncthreads();
      if (w < kTWaves / 2) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            f32x4* at = (f32x4*)(place + e * kTStrip + j);
            *at = *at + sum4(e, j);
          }
      }
      __syncthreads();
      for (int o = 4 * threadIdx.x; o < 16 * kTStrip; o += 4 * 64 * kTWaves) {
        const int64_t m = m0 + 16 * b + o / kTStrip, k = k0 + o % kTStrip;
        if (m >= M || k >= K) continue;
        f32x4 v = *(const f32x4*)(sums + o);
#pragma unroll
        for (int i = 1; i < kTWaves / 2; ++i) v += *(const f32x4*)(sums + i * 16 * kTStrip + o);
        *(f32x4*)(out + m * K + k) = v;
      }
    }
  }
}

// Rows of dy into rows of `pad` values, a multiple of 8, zeros behind the last.  Bound by bytes: 2048 rows of 11001 15 us.
__global__ __launch_bounds__(256) void k_pad_rows(const uint16_t* __restrict__ dy, int64_t M, int64_t N, int64_t pad,
                                                  uint16_t* __restrict__ out) {
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x)
    for (int64_t n = 8 * (int64_t)threadIdx.x; n < pad; n += 8 * 256) {
      bf16x8 v[1];
      row8(dy + m * N, n, N, true, v);
      *(bf16x8*)(out + m * pad + n) = v[0];
    }
}

// Back every row reads its adapter's [R, C] for itself: bound by that from about 64 ranks on (256 rows of 4096 columns in
// eight parts, ranks 16, 64, 128 and 256: 12, 18, 26 and 42 us; the tiles before it 22).
//
// A wave has 64 V columns of one row of the result at a time (V 4: at 16-byte
// addresses): the partial sums, in order, and, back, the low-rank part of the row's
// adapter from `out` [L, R, C].  (Forward the first part's tiles have added it: a dot product an output here,
// with every row's own read of [L, C, R], took 16 us for 128 rows of [11008, 4096] and 16 ranks, and 52 for 256 with float32 adapters.)
template <bool BACK, int V, typename TY>
__global__ __launch_bounds__(64) void k_w4a16_sum(const float* __restrict__ part, int parts, int64_t M, int64_t C,
                                                  Adapters ad, TY* __restrict__ y) {
  typedef float fV __attribute__((ext_vector_type(V)));
  __shared__ __attribute__((aligned(16))) float lows[kLoraMaxRank];  // the row's low-rank values (back)
  const int lane = threadIdx.x;
  const int64_t strips = (C + 64 * V - 1) / (64 * V), tiles = M * strips;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t m = tile / strips, c = 64 * V * (tile % strips) + V * lane;
    const bool in = c < C;
    const float* p = part + m * C + (in ? c : 0);
    // eight loads of the sums are under way while the row's adapter is found
    fV first[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) first[s] = *(const fV*)(p + (int64_t)(s < parts ? s : 0) * M * C);
    float u[kLoraMaxRank / kWave] = {};
    if (BACK && ad.count > 0) {  // the same in every lane
#pragma unroll
      for (int i = 0; i < kLoraMaxRank / kWave; ++i) {
        const int r = lane + kWave * i;
        if (kWave * i >= ad.rank) break;
        const float* low = ad.low + m * ad.rank + (r < ad.rank ? r : 0);
        // at most 16 parts, all of them under way at once
        float w[16];
#pragma unroll
        for (int s = 0; s < 16; ++s) w[s] = low[(int64_t)(s < ad.parts ? s : 0) * M * ad.rank];
        u[i] = w[0];
#pragma unroll
        for (int s = 1; s < 16; ++s) u[i] += s < ad.parts ? w[s] : 0.0f;
      }
    }
    asm volatile("" ::: "memory");
    const int l = BACK && ad.count > 0 ? row_adapter(ad, m, lane) : -1;
    fV v = first[0];
#pragma unroll
    for (int s = 1; s < 8; ++s)
      if (s < parts) v += first[s];
    for (int s0 = 8; s0 < parts; s0 += 8) {  // eight at a time
#pragma unroll
      for (int s = 0; s < 8; ++s) first[s] = *(const fV*)(p + (int64_t)(s0 + s < parts ? s0 + s : 0) * M * C);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s0 + s < parts) v += first[s];
    }
    if (BACK && l >= 0) {
#pragma unroll
      for (int i = 0; i < kLoraMaxRank / kWave; ++i) {
        const int r = lane + kWave * i;
        if (r >= ad.rank) break;
        lows[r] = u[i];
        if (ad.parts > 1 && tile % strips == 0) ad.whole[m * ad.rank + r] = u[i];
      }
      __builtin_amdgcn_wave_barrier();  // LDS operations of a wave complete in order
    }
    if (in && l >= 0) {
      if constexpr (BACK) {
        static_assert(V == 4, "C is a multiple of 32");
        fV d = {0.0f, 0.0f, 0.0f, 0.0f};
        if (ad.wide) {
          const float* a = (const float*)ad.out + (int64_t)l * ad.rank * C + c;
#pragma unroll 8
          for (int r = 0; r < ad.rank; ++r) {
            const f32x4 e = *(const f32x4*)(a + r * C);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = fmaf(lows[r], e[i], d[i]);
          }
        } else {
          const uint16_t* a = (const uint16_t*)ad.out + (int64_t)l * ad.rank * C + c;
#pragma unroll 8
          for (int r = 0; r < ad.rank; ++r) {
            const u32x2 e = *(const u32x2*)(a + r * C);
            d[0] = fmaf(lows[r], bf16_lo(e.x), d[0]);
            d[1] = fmaf(lows[r], bf16_hi(e.x), d[1]);
            d[2] = fmaf(lows[r], bf16_lo(e.y), d[2]);
            d[3] = fmaf(lows[r], bf16_hi(e.y), d[3]);
          }
        }
        v += d;
      }
      __builtin_amdgcn_wave_barrier();  // the next row's values take the place
    }
    if (in) {
      TY* out = y + m * C + c;
      if constexpr (sizeof(TY) == 4) {
        *(fV*)out = v;
      } else if constexpr (V == 4) {
        u32x2 b;
        b.x = f32_to_bf16_bits(v[0]) | f32_to_bf16_bits(v[1]) << 16;
        b.y = f32_to_bf16_bits(v[2]) | f32_to_bf16_bits(v[3]) << 16;
        *(u32x2*)out = b;
      } else {
        *out = (TY)f32_to_bf16_bits(v[0]);
      }
    }
  }
}

template <bool BACK, int V>
static hipError_t sum_go(const float* part, int parts, int64_t m, int64_t c, const Adapters& ad, void* y, int y_dtype,
                         hipStream_t st) {
  const int64_t tiles = m * ((c + 64 * V - 1) / (64 * V));
  const dim3 grid((unsigned)(tiles < kTSumGrid ? tiles : kTSumGrid));
  if (y_dtype == W4_F32) k_w4a16_sum<BACK, V><<<grid, 64, 0, st>>>(part, parts, m, c, ad, (float*)y);
  else k_w4a16_sum<BACK, V><<<grid, 64, 0, st>>>(part, parts, m, c, ad, (uint16_t*)y);
  return hipGetLastError();
}

bool w4a16_lora_sums(bool back, int64_t m, int64_t k, int64_t n, int g, int x_dtype, int sz_dtype, int y_dtype) {
  return lora_plan(back, m, k, n, g, x_dtype, sz_dtype, y_dtype).sums > 0;
}

size_t w4a16_lora_workspace_bytes(bool back, int64_t m, int64_t k, int64_t n, int g, int x_dtype, int sz_dtype,
                                  int y_dtype) {
  return lora_plan(back, m, k, n, g, x_dtype, sz_dtype, y_dtype).bytes;
}

template <typename TX, typename TS, int PW, int MB>
static hipError_t back_rows_go(const TilesArgs& a, const LoraPlan& p, float* part, hipStream_t st) {
  static std::atomic<uint64_t> attr_done{0};  // LDS above the 64 KB default
  constexpr size_t lds = (size_t)kTWaves / 2 * 16 * kTStrip * 4 + (size_t)kTWaves * 2048;
  const hipError_t e = once_per_device(attr_done, [] {
    return hipFuncSetAttribute((const void*)k_w4a16_back_rows<TX, TS, PW, MB>,
                               hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  });
  if (e != hipSuccess) return e;
  const int64_t tiles = p.strips * p.rows;
  k_w4a16_back_rows<TX, TS, PW, MB>
      <<<dim3((unsigned)(tiles < kTGrid ? tiles : kTGrid), (unsigned)p.parts), 64 * kTWaves, lds, st>>>(
          (const TX*)a.x, a.m, a.n, a.packed, a.scales, a.zeros, a.k, a.g, (int)p.steps, part);
  return hipGetLastError();
}

template <typename TX, typename TS>
static hipError_t back_rows(const TilesArgs& a, const LoraPlan& p, float* part, hipStream_t st) {
  if constexpr (sizeof(TS) == 4) {
    if (p.pw == 3) return back_rows_go<TX, TS, 3, 1>(a, p, part, st);
  }
  if constexpr (sizeof(TX) == 2) {
    if (p.mb == 2) return back_rows_go<TX, TS, 2, 2>(a, p, part, st);
  }
  if constexpr (sizeof(TX) == 2 || sizeof(TS) == 2) return back_rows_go<TX, TS, 2, 1>(a, p, part, st);
  return hipErrorInvalidValue;
}

hipError_t launch_w4a16_lora(const void* x, int x_dtype, const TilesArgs& args, const LoraOut& lo, void* ws,
                             hipStream_t st) {
  const LoraPlan p = lora_plan(args.back, args.m, args.k, args.n, args.g, x_dtype, args.sz_dtype, args.y_dtype);
  TilesArgs a = args;
  a.x = x;
  a.mi = p.mi, a.pw = p.pw, a.parts = (int)p.parts, a.steps = (int)p.steps, a.row = a.n;
  float* part = (float*)ws;
  hipError_t e;
  if (p.tiles) {
    if (p.parts > 1) a.y = ws, a.y_dtype = W4_F32;
    if (p.pad > 0) {
      uint16_t* rows = (uint16_t*)((uint8_t*)ws + p.sums);
      k_pad_rows<<<dim3((unsigned)(a.m < 16384 ? a.m : 16384)), 256, 0, st>>>((const uint16_t*)x, a.m, a.n, p.pad, rows);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      a.x = rows, a.row = p.pad;
    }
    // With parts, forward the first one's tiles add the low-rank part, back the sum, which low may come to in parts.
    if (!a.back) e = launch_w4a16_lora_gemm(a, lo, st);
    else e = launch_w4a16_tiles(a, p.parts == 1 ? lo : LoraOut{}, st);
    if (p.parts == 1) return e;
  } else if (!a.back) {
    return launch_w4a16_lora_rows(x, x_dtype, a.m, a.k, a.packed, a.scales, a.zeros, a.sz_dtype, a.n, a.g, a.y,
                                  a.y_dtype, lo, st);
  } else if (x_dtype == W4_F32) {
    e = a.sz_dtype == W4_F16 ? back_rows<float, _Float16>(a, p, part, st) : back_rows<float, float>(a, p, part, st);
  } else {
    e = a.sz_dtype == W4_F16 ? back_rows<uint16_t, _Float16>(a, p, part, st) : back_rows<uint16_t, float>(a, p, part, st);
  }
  if (e != hipSuccess) return e;
  const Adapters ad = adapters_of(lo);
  if (a.back) return sum_go<true, 4>(part, (int)p.parts, a.m, a.k, ad, args.y, args.y_dtype, st);
  if (a.n % 4 == 0) return sum_go<false, 4>(part, (int)p.parts, a.m, a.n, ad, args.y, args.y_dtype, st);
  return sum_go<false, 1>(part, (int)p.parts, a.m, a.n, ad, args.y, args.y_dtype, st);
}

}  // namespace w4
