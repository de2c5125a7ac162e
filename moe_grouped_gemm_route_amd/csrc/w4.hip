// moe_w4_gemv: a few rows times 4-bit integer weights with a scale, and
// optionally a zero point, per group of G weights along K:
//     y[t, n] = sum_k s[n, k/G] (c[n, k] - z[n, k/G]) x[t, k],
// dense, per chosen expert of a token, or those summed with the router's
// weights, optionally through the SiLU-gated activation.  The codes are read
// as they lie ([N, K/2], the even k in the low nibble): for a handful of rows
// the product is one pass over the weights, and nothing else is large.
//
// The integer part runs on the bf16 matrix unit, exactly.  A nibble c, read as
// an E4M3 byte, is c 2^-9 for every c of 0 .. 15 (the subnormals and the first
// normal binade join linearly), so one scaled convert with scale 2^9 turns two
// bytes into two exact bf16 integers.  The zero point stays out of the
// product:  sum (c - z) x = sum c x - z sum x  per group, both sums in f32 on
// the matrix unit (the second against a constant operand of ones).  A group's
// sums are then multiplied by its scale and added in f32: no weight is rounded.
//
// Both kernels multiply with v_mfma_f32_16x16x32_bf16, which adds over the lane
// groups of a column of codes, while groups with different scales must stay
// apart.  So x is laid out block-diagonally: a row of the first operand holds x
// of one 32-block (one row of x: w4_lane_kernel) or of one token's blocks with
// one scale (several: w4_few_kernel) and zeros elsewhere, and every result is a
// whole sum under one scale.
//
// Bound by memory: 4 bits a weight and the scales.  Matrices in the caches' reach
// and small ones are bound by the start and end of a stream: the first loads, the
// join over the waves, one launch.
#include "common.h"
#include "launch.h"
#include "lds_load.h"
#include "wave.h"

namespace moe {

struct W4Args {
  const uint8_t* codes;
  const void* scales;
  const uint8_t* zeros;      // NULL: 8 everywhere
  const uint16_t* x;
  const int32_t* ids;        // NULL: dense
  const float* weights;      // NULL: a row per pair
  void* y;
  int64_t N, K, groups;      // columns, depth, scale groups of a column
  int E, T, k;
  int gshift;                // log2 G
  int x_pairs;               // x has a row per pair
  int scale_bf16, y_bf16;
  int col_groups;
};

// Eight codes of a word as bf16 integers, in the order k = 0 2 4 6 1 3 5 7
// (x_order puts eight x in the same order).
__device__ __forceinline__ u32x4_t codes_to_bf16(uint32_t q) {
  const uint32_t even = q & 0x0F0F0F0Fu, odd = (q >> 4) & 0x0F0F0F0Fu;
  u32x4_t r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, true));
  return r;
}

__device__ __forceinline__ u32x4_t x_order(u32x4_t x) {
  u32x4_t r;
  r[0] = __builtin_amdgcn_perm(x[1], x[0], 0x05040100u);
  r[1] = __builtin_amdgcn_perm(x[3], x[2], 0x05040100u);
  r[2] = __builtin_amdgcn_perm(x[1], x[0], 0x07060302u);
  r[3] = __builtin_amdgcn_perm(x[3], x[2], 0x07060302u);
  return r;
}

__device__ __forceinline__ f32x4_t w4_mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t w4_rsrc(const void* base, int64_t offset, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(static_cast<const uint8_t*>(base)) + offset, 0,
                                           (int)bytes, 0x00020000);
}

// S groups' scales (SB: bf16) as words; VEC: in one load.
template <int S, bool SB, bool VEC>
__device__ __forceinline__ void w4_load_scales(__amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t off, int left,
                                               uint32_t (&q)[S]) {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < S; ++i) q[i] = 0;
  if constexpr (S == 1) {
    q[0] = SB ? __builtin_amdgcn_raw_buffer_load_b16(r, vo, off, 0) : __builtin_amdgcn_raw_buffer_load_b32(r, vo, off, 0);
  } else if constexpr (VEC && SB && S == 2) {
    q[0] = __builtin_amdgcn_raw_buffer_load_b32(r, vo, off, 0);
  } else if constexpr (VEC && (SB ? S == 4 : S == 2)) {
    const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(r, vo, off, 0);
    q[0] = v[0];
    q[1] = v[1];
  } else if constexpr (VEC) {
    const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, vo, off, 0);
#pragma unroll
    for (int i = 0; i < S; ++i) q[i] = v[i];
  } else {
    // groups past the column's last (K ends inside the chunk) count as 0: what
    // lies there is another column's
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const uint32_t at = i < left ? vo : kLaneOob;
      if (SB) q[i >> 1] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, off + 2 * i, 0) << (16 * (i & 1));
      else q[i] = __builtin_amdgcn_raw_buffer_load_b32(r, at, off + 4 * i, 0);
    }
  }
}

template <int S, bool VEC>
__device__ __forceinline__ uint32_t w4_load_zeros(__amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t off) {
  if constexpr (S == 4 && VEC) return __builtin_amdgcn_raw_buffer_load_b32(r, vo, off, 0);
  if constexpr (S == 2 && VEC) return __builtin_amdgcn_raw_buffer_load_b16(r, vo, off, 0);
  uint32_t q = 0;
#pragma unroll
  for (int i = 0; i < S; ++i) q |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r, vo, off + i, 0) << (8 * i);
  return q;
}

// ---------------------------------------------------------------------------
// Few tokens: a lane's own 32 codes
// ---------------------------------------------------------------------------

// A value that every lane reads and no kernel writes, by a scalar load: a vector
// one would wait for the ring.
template <typename V>
__device__ __forceinline__ V scalar_load(const V* p) {
  return *(const __attribute__((address_space(4))) V*)(uintptr_t)p;
}

// A wave multiplies 4 rows x 512 k of codes at a time, 1 KiB in one load of whole
// 256-byte runs (loads in the matrix unit's order would be 64 cache accesses a
// KiB instead of 16, and the L1 takes one a cycle).  Lane l holds 32 codes of one
// row, r = (l & 15) >> 2, and one 32-block, b = 4 (l >> 4) + (l & 3), and needs
// the sum over just these.  The matrix unit adds over the four lanes of a column
// and shares x between columns, so x is laid out with a row per block: row 4 g + s
// of the first operand holds x of block 4 g + s in lane group g and zeros
// elsewhere.  Result register i of lane l is then block 4 (l >> 4) + i against the
// codes of column l & 15, of which the lane's own is i = l & 3.  The lane's scale
// and zero point are those of the block, loaded as it loads the codes; x and its
// block sums stay in registers for all rows.
//
// Waves of a workgroup take units of 512 k (of a token's experts one after the
// other: SUM) of the same rows, blocks of 8 row quads after one another (with
// ACT 4 quads of gate rows and the 4 of up rows).  A wave's loads run through
// all of its blocks and units in a ring; a block's sums over the lanes of a row
// and over the waves are joined in LDS, in order, while the next block's loads
// are on their way.
//
// Measured, one row, groups of 128: 131,072 x 4,096 46 to 48 us (5.8 TB/s of codes
// and scales, above a copy's 5.1: nothing is written), 8,192 x 8,192 10.5, 4,096
// x 4,096 5.4 (1.7 at a copy's rate: the launch and the stream's two ends are the
// rest).  Six experts of one token (57 MB) 13.9, 42 pairs summed per token (231 MB)
// 39.5 to 44.
constexpr int W4_NT = 2;       // non-temporal: codes are read once
constexpr int W4_WAVES = 8;
constexpr int W4_RING = 8;     // loads of 1 KiB in flight per wave, and row quads of a block

struct W4LaneArgs {
  W4Args a;
  int blocks;                  // of a workgroup
  int row_blocks;              // of the rows of x (w4_few_kernel)
};

template <bool ACT, bool SUM, bool SB, bool Z>
__global__ __launch_bounds__(W4_WAVES * 64) void w4_lane_kernel(W4LaneArgs la) {
  const W4Args& p = la.a;
  constexpr int SZ = SB ? 2 : 4;
  constexpr int HALF = ACT ? W4_RING / 2 : W4_RING;   // quads of a block that are rows of y
  __shared__ __attribute__((aligned(16))) float s_sum[2][W4_RING][W4_WAVES][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;                // a unit each at least
  const int g = lane >> 4, q4 = lane & 3, r = (lane & 15) >> 2;
  const int block = g * 4 + q4;
  const int K = (int)p.K, groups = (int)p.groups;
  const int64_t N = p.N;
  const int cols = (int)(ACT ? N / 2 : N);
  const int cg = blockIdx.x % (uint32_t)p.col_groups;
  const int rb = blockIdx.x / (uint32_t)p.col_groups;
  const bool pairs = p.ids != nullptr;

  const int row0 = cg * la.blocks * HALF * 4;
  const int rows = min(la.blocks * HALF * 4, cols - row0);
  const int blocks = (rows + HALF * 4 - 1) / (HALF * 4);
  const int per = (K + 511) >> 9;                   // units of a matrix
  const int total = (SUM ? p.k : 1) * per;

  // lane offsets; lanes off the block diagonal of x read zeros
  const uint32_t cvo = (uint32_t)r * (uint32_t)(K / 2) + block * 16;
  const uint32_t srow = (uint32_t)(r * groups);
  const bool diag = g == r;
  const int gsh = p.gshift - 5;

  const f32x4_t zero4 = {0.f, 0.f, 0.f, 0.f};
  const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  auto own = [&](const f32x4_t& d) __attribute__((always_inline)) {
    const float lo = q4 & 1 ? d[1] : d[0], hi = q4 & 1 ? d[3] : d[2];
    return q4 & 2 ? hi : lo;
  };

  // A unit: 512 k of one matrix, or nothing.
  struct Unit {
    int64_t e, xrow;
    int c;
    bool live;
    float factor;
  };
  auto unit = [&](int u) __attribute__((always_inline)) {
    const int j = SUM ? u / per : 0;
    const int pair = SUM ? rb * p.k + j : rb;
    Unit n = {0, 0, SUM ? u - j * per : u, u < total, 1.f};
    if (pairs) {
      const int id = u < total ? scalar_load(p.ids + pair) : -1;
      n.live = (uint32_t)id < (uint32_t)p.E;
      n.e = n.live ? id : 0;
      n.xrow = p.x_pairs ? pair : pair / p.k;
      if (SUM) n.factor = n.live ? scalar_load(p.weights + pair) : 0.f;
    }
    return n;
  };

  // (scale and zero point as wide as they are loaded: to widen them on the way
  // into the loop would wait for them)
  struct Row {
    u32x4_t codes;
    std::conditional_t<SB, uint16_t, uint32_t> scale;
    uint8_t zero;
  };
  Row ring[W4_RING];
  // The next load: quad `li` (its place in the ring) of unit lu of block lb.
  int lu = wave, lb = 0;
  Unit ln = unit(lu);
  uint32_t lsvo = 0;
  auto offsets = [&]() __attribute__((always_inline)) {
    lsvo = ln.c * 512 + block * 32 < K ? srow + ((ln.c * 16 + block) >> gsh) : kLaneOob / SZ;
  };
  offsets();
  auto load = [&](int li, Row& q) __attribute__((always_inline)) {
    const bool up = ACT && li >= HALF;
    const int at = (lb * HALF + (up ? li - HALF : li)) * 4;   // row of the workgroup's
    const int64_t base = ln.e * N + (up ? N / 2 : 0) + row0;
    const int have = ln.live && lb < blocks ? rows : 0;
    q.codes = __builtin_amdgcn_raw_buffer_load_b128(w4_rsrc(p.codes, base * (K / 2), (int64_t)have * (K / 2)), cvo,
                                                    at * (K / 2) + ln.c * 256, W4_NT);
    const __amdgpu_buffer_rsrc_t sr = w4_rsrc(p.scales, base * groups * SZ, (int64_t)have * groups * SZ);
    if constexpr (SB) q.scale = __builtin_amdgcn_raw_buffer_load_b16(sr, lsvo * SZ, at * groups * SZ, 0);
    else q.scale = __builtin_amdgcn_raw_buffer_load_b32(sr, lsvo * SZ, at * groups * SZ, 0);
    q.zero = 8;
    if constexpr (Z)
      q.zero = __builtin_amdgcn_raw_buffer_load_b8(w4_rsrc(p.zeros, base * groups, (int64_t)have * groups), lsvo,
                                                   at * groups, 0);
  };
  auto next_unit = [&]() __attribute__((always_inline)) {
    lu += waves;
    if (lu >= total) {
      lu = wave;
      ++lb;
    }
    if (total > waves) {
      ln = unit(lu);
      offsets();
    }
  };

  u32x4_t x[4], xn[4];
  float sx, factor = 1.f, nfactor = 1.f;
  auto load_x = [&](const Unit& n, u32x4_t (&to)[4], float& f) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t xr = w4_rsrc(p.x, n.xrow * K * 2, n.live ? (int64_t)K * 2 : 0);
    const uint32_t xvo = n.c * 512 + block * 32 < K && diag ? (uint32_t)(n.c * 1024 + block * 64) : kLaneOob;
#pragma unroll
    for (int s = 0; s < 4; ++s) to[s] = __builtin_amdgcn_raw_buffer_load_b128(xr, xvo + s * 16, 0, 0);
    f = n.factor;
  };
  auto sum_x = [&]() __attribute__((always_inline)) {
    f32x4_t d = zero4;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      x[s] = x_order(x[s]);
      d = w4_mfma(x[s], ones, d);
    }
    sx = own(d);
  };

  // x of the first unit, then the ring, in the order of use (a load waits for
  // all before it)
  load_x(ln, x, factor);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < W4_RING; ++i) {
    load(i, ring[i]);
    __builtin_amdgcn_sched_barrier(0);
  }
  next_unit();
  sum_x();

  for (int b = 0; b < blocks; ++b) {
    float (*sums)[W4_WAVES][16] = s_sum[b & 1];
    for (int u = wave; u < total; u += waves) {
      // the next unit's x (the last one's: the first of the next block) comes
      // ahead of the loads that follow it
      if (total > waves) load_x(unit(u + waves < total ? u + waves : wave), xn, nfactor);
#pragma unroll
      for (int i = 0; i < W4_RING; ++i) {
        const Row& q = ring[i];
        u32x4_t w[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) w[s] = codes_to_bf16(q.codes[s]);
        float sc = SB ? bf16_lo(q.scale) : __uint_as_float(q.scale);
        if (SUM) sc *= factor;
        const float z = (float)q.zero;
        __builtin_amdgcn_sched_barrier(0);
        load(i, ring[i]);
        __builtin_amdgcn_sched_barrier(0);
        f32x4_t d = zero4;
#pragma unroll
        for (int s = 0; s < 4; ++s) d = w4_mfma(x[s], w[s], d);
        // over the four lanes of the row's 64 bytes
        float f = sc * fmaf(-z, sx, own(d));
        f += dpp_from<0xB1>(f);
        f += dpp_from<0x4E>(f);
        if (q4 == 0) {
          float* to = &sums[i][wave][r * 4 + g];
          *to = u == wave ? f : *to + f;
        }
      }
      next_unit();
      if (total > waves) {
#pragma unroll
        for (int s = 0; s < 4; ++s) x[s] = xn[s];
        factor = nfactor;
        sum_x();
      }
    }
    lds_barrier();

    // eight lanes add up a row, one a wave
    const int w = threadIdx.x & 7;
    const int live = min(rows - b * HALF * 4, HALF * 4);    // rows of y of the block
    auto total_of = [&](int quad, int row) __attribute__((always_inline)) {
      float f = 0.f;
      if (w < waves) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&sums[quad][w][row * 4]);
        f = (v[0] + v[1]) + (v[2] + v[3]);
      }
      f += dpp_from<0xB1>(f);
      f += dpp_from<0x4E>(f);
      return f + dpp_from<0x141>(f);                        // the other quad of eight lanes
    };
    for (int row = threadIdx.x >> 3; row < HALF * 4; row += blockDim.x >> 3) {
      float f = total_of(row >> 2, row & 3);
      if (ACT) f = f / (1.0f + __expf(-f)) * total_of(HALF + (row >> 2), row & 3);
      if (w != 0 || row >= live) continue;
      const int64_t at = (int64_t)rb * cols + row0 + b * HALF * 4 + row;
      if (p.y_bf16) reinterpret_cast<uint16_t*>(p.y)[at] = f32_to_bf16_rne(f);
      else reinterpret_cast<float*>(p.y)[at] = f;
    }
  }
}

// Blocks of `rows` columns of a workgroup, at most as many as keep its codes
// within 2^30 bytes, which its loads address with 32-bit offsets.
static int64_t w4_hold(int64_t blocks, int rows, int64_t K) {
  const int64_t most = (int64_t(1) << 30) / (K / 2) / rows;   // K <= 2^23: 4 at least
  return blocks < most ? blocks : most;
}

template <bool ACT, bool SUM, bool SB, bool Z>
static hipError_t launch_w4_lane_t(const W4Args& a, int64_t row_blocks, hipStream_t stream) {
  W4LaneArgs la = {a, 0, 1};
  const int64_t cols = ACT ? a.N / 2 : a.N;
  constexpr int ROWS = 4 * (ACT ? W4_RING / 2 : W4_RING);
  const int64_t blocks = (cols + ROWS - 1) / ROWS;
  const int64_t units = (a.K + 511) / 512 * (SUM ? a.k : 1);
  const int waves = units < W4_WAVES ? (int)units : W4_WAVES;
  // two workgroups of 8 waves to a CU, where there are as many blocks (28,672 x
  // 4,096: 14.3 us, one to a CU 13.8, four 15.0; 131,072: 48.3, 48.9, 48.1)
  constexpr int ROOM = 512;
  const int64_t per = (blocks * row_blocks + ROOM - 1) / ROOM;
  la.blocks = (int)w4_hold(per < blocks ? per : blocks, ROWS, a.K);
  la.a.col_groups = (int)((blocks + la.blocks - 1) / la.blocks);
  hipLaunchKernelGGL((w4_lane_kernel<ACT, SUM, SB, Z>), dim3((unsigned)(row_blocks * la.a.col_groups)),
                     dim3(waves * 64), 0, stream, la);
  return hipGetLastError();
}

template <bool SB, bool Z>
static hipError_t launch_w4_lane(const W4Args& a, int act, hipStream_t stream) {
  if (a.weights) return launch_w4_lane_t<false, true, SB, Z>(a, a.T, stream);
  const int64_t rows = a.ids ? (int64_t)a.T * a.k : 1;
  return act ? launch_w4_lane_t<true, false, SB, Z>(a, rows, stream)
             : launch_w4_lane_t<false, false, SB, Z>(a, rows, stream);
}

// ---------------------------------------------------------------------------
// A few more tokens: x in registers, 16 columns at a time
// ---------------------------------------------------------------------------

// 16 / S tokens of a dense product, S = 128 / G scale groups of a chunk of 128 k
// (at least 1); more tokens are more row blocks.  In a chunk lane l holds the 16
// bytes of column n = l & 15 and 32-block g = l >> 4, and one of four matrix
// instructions multiplies 8 k of all four blocks.  Row r of the first operand is
// token r / S with the lane groups of scale group r % S alone, the rest zero; a
// lane's four results are whole group sums of one column.
//
// ALL: 16 tokens, also where a chunk has several scale groups.  A matrix
// instruction takes 32 consecutive k, lane group g the 8 k from 8 g, so that its
// results, or a chain's of G / 32, are whole group sums with no zeros laid out:
// 4 / S as many converts a token, S as many sums to scale a chunk.  The sums of x
// (S times as many too) lie in LDS, and with S = 4 chunks are finished one by one;
// what does not fit the registers then is a few addresses.
//
// The walk is w4_lane_kernel's: a wave keeps x of its 512 k (four chunks) in
// registers, with the sums of x per group, and goes through 16-column tiles, BT to
// a block (with ACT half of them gate and half up tiles).  Codes are loaded in
// runs of 256 bytes and turned into the operand's order through LDS of the wave's
// own; a tile's scales and zero points are loaded by lane group g for chunk g and
// handed to the lanes that need them through the LDS crossbar.
//
// Measured (us; 131,072 x 4,096): groups of 128, 2 rows 53, 16 rows 60, 64 rows
// 170; groups of 32, 2 to 4 rows 51 to 54, 5 to 8 (two row blocks) 77, 9 to 16
// (ALL) 78, 64 258 (509 by blocks of 4).  4,096 x 4,096: groups of 32, 2 to 8 rows
// 6.2, 16 rows 9, 64 rows 15; groups of 128, 64 rows 11.8.  One row block is bound
// by memory (5.2 TB/s at 2 rows); with more the codes come from L2 and each is
// converted and multiplied again for every row block, which bounds it then: that
// product is for few rows.
template <int S, bool ALL, bool ACT, bool SB, bool VEC, bool Z, int BT>
__global__ __launch_bounds__(W4_WAVES * 64) void w4_few_kernel(W4LaneArgs la) {
  const W4Args& p = la.a;
  constexpr int SZ = SB ? 2 : 4;
  constexpr int SW = SB ? (S + 1) / 2 : S;            // scale words of a chunk
  constexpr int D = ALL ? 1 : S;                      // rows of the operand that a token takes
  constexpr int R = 4 / D;                            // tokens a lane holds
  constexpr int HALF = ACT ? BT / 2 : BT;             // tiles of a block that are columns of y
  __shared__ float s_sum[2][BT * R][W4_WAVES][64];
  __shared__ __attribute__((aligned(256))) uint8_t s_codes[W4_WAVES][4096];
  __shared__ __attribute__((aligned(16))) float s_sx[ALL ? W4_WAVES : 1][ALL ? 4 * S : 1][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;                  // a unit each at least
  const int n16 = lane & 15, g = lane >> 4;
  const int K = (int)p.K, groups = (int)p.groups;
  const int64_t N = p.N;
  const int cols = (int)(ACT ? N / 2 : N);

  // the row blocks of one column group follow one another on an XCD (workgroup
  // ids go round them), so that its codes come from memory once
  const int id = blockIdx.x >> 3;
  const int cg = id / la.row_blocks * 8 + (blockIdx.x & 7), rb = id % la.row_blocks;
  if (cg >= p.col_groups) return;
  const int t0 = rb * (16 / D);                          // first token
  const int row0 = cg * la.blocks * HALF * 16;           // first column of y
  const int rows = min(la.blocks * HALF * 16, cols - row0);
  const int blocks = (rows + HALF * 16 - 1) / (HALF * 16);
  const int total = (K + 511) >> 9;

  // load c of a tile: rows 4 c + g, their 256 bytes; through LDS, row n's
  // 16-byte segment s at place s ^ n
  const uint32_t cvo = (uint32_t)g * (uint32_t)(K / 2) + n16 * 16;
  uint8_t* own = s_codes[wave];
  const uint32_t srow = (uint32_t)(n16 * groups);
  const bool mine = D == 1 || (S == 2 ? (g >> 1) == (n16 & 1) : g == (n16 & 3));
  constexpr int XG = ALL ? 8 : 32, XS = ALL ? 32 : 8;    // k from a lane group, and a step, to the next
  const uint32_t xrow = mine && t0 + n16 / D < p.T ? (uint32_t)(n16 / D * K * 2 + g * XG * 2) : kLaneOob;

  const f32x4_t zero4 = {0.f, 0.f, 0.f, 0.f};
  const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};

  struct Tile {
    u32x4_t codes[4];
    uint32_t scale[S];
    uint32_t zero;
  };
  Tile ring[BT];
  int lu = wave, lb = 0;               // unit and block of the next load
  auto load = [&](int li, Tile& q) __attribute__((always_inline)) {
    const bool up = ACT && li >= HALF;
    const int at = (lb * HALF + (up ? li - HALF : li)) * 16;
    const int64_t base = (up ? N / 2 : 0) + row0;
    const int have = lb < blocks ? rows : 0;
    const __amdgpu_buffer_rsrc_t cr = w4_rsrc(p.codes, base * (K / 2), (int64_t)have * (K / 2));
#pragma unroll
    for (int c = 0; c < 4; ++c)
      q.codes[c] = __builtin_amdgcn_raw_buffer_load_b128(cr, cvo, (at + c * 4) * (K / 2) + lu * 256, W4_NT);
    const int kc = lu * 4 + g;         // the chunk whose scales this lane loads
    const int gi = S > 1 ? kc * S : (int)(((int64_t)kc * 128) >> p.gshift);
    const uint32_t so = kc * 128 < K ? srow + gi : kLaneOob / SZ;
    w4_load_scales<S, SB, VEC>(w4_rsrc(p.scales, base * groups * SZ, (int64_t)have * groups * SZ), so * SZ,
                               at * groups * SZ, groups - gi, q.scale);
    if (Z)
      q.zero = w4_load_zeros<S, VEC>(w4_rsrc(p.zeros, base * groups, (int64_t)have * groups), so, at * groups);
  };
  auto next_unit = [&]() __attribute__((always_inline)) {
    lu += waves;
    if (lu >= total) {
      lu = wave;
      ++lb;
    }
  };

  u32x4_t x[4][4];
  constexpr int SX = ALL ? S : 1, CH = 4 / SX;           // sums of a chunk, and steps to each
  f32x4_t sx[4];                                          // (not ALL: they lie in LDS)
  const int64_t x0 = (int64_t)t0 * K * 2, xbytes = (int64_t)min(16 / D, p.T - t0) * K * 2;
  auto load_x = [&](int u) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bool in = u * 512 + c * 128 + (ALL ? s : g) * 32 < K;
        x[c][s] = __builtin_amdgcn_raw_buffer_load_b128(w4_rsrc(p.x, x0, !ALL || in ? xbytes : 0),
                                                        (ALL || in ? xrow : kLaneOob) + s * XS * 2, u * 1024 + c * 256, 0);
      }
    }
  };
  auto sum_x = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      f32x4_t v[SX];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        x[c][s] = x_order(x[c][s]);
        v[s / CH] = w4_mfma(x[c][s], ones, s % CH ? v[s / CH] : zero4);
      }
      if constexpr (ALL) {
        if (n16 == 0) {
#pragma unroll
          for (int o = 0; o < S; ++o) *reinterpret_cast<f32x4_t*>(&s_sx[wave][c * S + o][g * 4]) = v[o];
        }
      } else {
        sx[c] = v[0];
      }
    }
    if (ALL) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };

  load_x(wave);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < BT; ++i) {
    load(i, ring[i]);
    __builtin_amdgcn_sched_barrier(0);
  }
  next_unit();
  sum_x();

  for (int b = 0; b < blocks; ++b) {
    float (*sums)[W4_WAVES][64] = s_sum[b & 1];
    for (int u = wave; u < total; u += waves) {
#pragma unroll
      for (int i = 0; i < BT; ++i) {
        uint32_t sw[4][S], zw[4];
        auto scales_of = [&](int c) __attribute__((always_inline)) {
          const int from = (n16 | c << 4) << 2;
#pragma unroll
          for (int j = 0; j < SW; ++j) sw[c][j] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)ring[i].scale[j]);
          zw[c] = Z ? (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)ring[i].zero) : 0x08080808u;
        };
        if constexpr (!(ALL && S == 4))
#pragma unroll
          for (int c = 0; c < 4; ++c) scales_of(c);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<u32x4_t*>(own + (c * 4 + g) * 256 + ((n16 ^ (c * 4 + g)) << 4)) = ring[i].codes[c];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float acc[R];
#pragma unroll
        for (int j = 0; j < R; ++j) acc[j] = 0.f;
        f32x4_t d[4][SX];
        auto products = [&](int c) __attribute__((always_inline)) {
          u32x4_t q;
          if constexpr (ALL) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              q[s] = *reinterpret_cast<const uint32_t*>(own + n16 * 256 + (((c * 4 + s) ^ n16) << 4) + g * 4);
          } else {
            q = *reinterpret_cast<const u32x4_t*>(own + n16 * 256 + (((c * 4 + g) ^ n16) << 4));
          }
#pragma unroll
          for (int s = 0; s < 4; ++s)
            d[c][s / CH] = w4_mfma(x[c][s], codes_to_bf16(q[s]), s % CH ? d[c][s / CH] : zero4);
        };
        auto add = [&](int c) __attribute__((always_inline)) {
#pragma unroll
          for (int o = 0; o < S; ++o) {
            const float sc = SB ? ((o & 1) ? bf16_hi(sw[c][o >> 1]) : bf16_lo(sw[c][o >> 1])) : __uint_as_float(sw[c][o]);
            const float z = (float)((zw[c] >> (8 * o)) & 0xFFu);
            f32x4_t v;
            if constexpr (ALL) v = *reinterpret_cast<const f32x4_t*>(&s_sx[wave][c * S + o][g * 4]);
            else v = sx[c];
            // result j: token j and every group's own sum, or token j / S and group j % S
#pragma unroll
            for (int j = 0; j < R; ++j) {
              const int k = ALL ? j : j * S + o, e = ALL ? o : 0;
              acc[j] = fmaf(sc, fmaf(-z, v[k], d[c][e][k]), acc[j]);
            }
          }
        };
        if constexpr (ALL && S == 4) {
          // chunk by chunk: all sums of a tile do not fit the registers
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            __builtin_amdgcn_sched_barrier(0);
            scales_of(c);
            products(c);
            add(c);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          }
          __builtin_amdgcn_sched_barrier(0);
          load(i, ring[i]);
          __builtin_amdgcn_sched_barrier(0);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) products(c);
          __builtin_amdgcn_sched_barrier(0);
          load(i, ring[i]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int c = 0; c < 4; ++c) add(c);
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
          float* to = &sums[i * R + j][wave][lane];
          *to = u == wave ? acc[j] : *to + acc[j];
        }
      }
      next_unit();
      if (total > waves) {
        load_x(u + waves < total ? u + waves : wave);
        sum_x();
      }
    }
    lds_barrier();

    const int live = min(rows - b * HALF * 16, HALF * 16);
    for (int o = threadIdx.x; o < HALF * R * 64; o += blockDim.x) {
      const int l = o & 63, j = (o >> 6) % R, c = (o >> 6) / R;
      const int t = t0 + (l >> 4) * R + j, col = c * 16 + (l & 15);
      if (t >= p.T || col >= live) continue;
      float f = 0.f, h = 0.f;
      for (int w = 0; w < waves; ++w) {
        f += sums[c * R + j][w][l];
        if (ACT) h += sums[(c + HALF) * R + j][w][l];
      }
      if (ACT) f = f / (1.0f + __expf(-f)) * h;
      const int64_t at = (int64_t)t * cols + row0 + b * HALF * 16 + col;
      if (p.y_bf16) reinterpret_cast<uint16_t*>(p.y)[at] = f32_to_bf16_rne(f);
      else reinterpret_cast<float*>(p.y)[at] = f;
    }
  }
}

template <int S, bool ALL, bool ACT, bool SB, bool VEC, bool Z, int BT>
static hipError_t launch_w4_few_t(const W4Args& a, hipStream_t stream) {
  constexpr int PER = ALL ? 16 : 16 / S;
  W4LaneArgs la = {a, 0, (a.T + PER - 1) / PER};
  const int64_t cols = ACT ? a.N / 2 : a.N;
  constexpr int COLS = 16 * (ACT ? BT / 2 : BT);
  const int64_t blocks = (cols + COLS - 1) / COLS;
  const int64_t units = (a.K + 511) / 512;
  const int waves = units < W4_WAVES ? (int)units : W4_WAVES;
  // a workgroup per CU at a time, its column groups in eights
  const int64_t room = la.row_blocks > 32 ? 8 : 32 / la.row_blocks * 8;
  la.blocks = (int)w4_hold((blocks + room - 1) / room, COLS, a.K);
  la.a.col_groups = (int)((blocks + la.blocks - 1) / la.blocks);
  const int64_t groups = ((int64_t)la.a.col_groups + 7) / 8 * 8 * la.row_blocks;
  hipLaunchKernelGGL((w4_few_kernel<S, ALL, ACT, SB, VEC, Z, BT>), dim3((unsigned)groups), dim3(waves * 64), 0, stream, la);
  return hipGetLastError();
}

template <int S, bool ALL, bool SB, bool VEC, bool Z>
static hipError_t launch_w4_few_rows(const W4Args& a, int act, hipStream_t stream) {
  // four tiles a block where that still leaves a block per CU: one join for twice
  // the codes (131,072 x 4,096, 5 rows, groups of 128: 55.7 us, 60.4 with two);
  // else two, so that more CUs have one (4,096 x 4,096: 6.7, 10.1 with four)
  const int64_t rows = ALL ? (a.T + 15) / 16 : (a.T + 16 / S - 1) / (16 / S), wide = a.N / 64 * rows;
  if constexpr (!(ALL && S == 4))
    if (wide >= 256)
      return act ? launch_w4_few_t<S, ALL, true, SB, VEC, Z, 4>(a, stream) : launch_w4_few_t<S, ALL, false, SB, VEC, Z, 4>(a, stream);
  return act ? launch_w4_few_t<S, ALL, true, SB, VEC, Z, 2>(a, stream) : launch_w4_few_t<S, ALL, false, SB, VEC, Z, 2>(a, stream);
}

template <int S, bool SB, bool VEC, bool Z>
static hipError_t launch_w4_few_z(const W4Args& a, int act, hipStream_t stream) {
  if constexpr (S > 1) {
    // ALL where it saves row blocks enough and its blocks leave no CU idle, or
    // where it saves many (us with and without; groups of 32: 16,384 x 8,192, 8
    // rows 31.7, 26.8, 16 rows 36, 44; 8,192 x 8,192, 9 rows 20, 25, 64 rows 58,
    // 78; 4,096 x 4,096, 16 rows 10.7, 9.3, 32 rows 11.2, 13.3; groups of 64:
    // 16,384 x 4,096, 9 rows 13.3, 15.1; 4,096 x 4,096, 16 rows 8.8, 6.6)
    const int64_t few = (a.T + 16 / S - 1) / (16 / S), all = (a.T + 15) / 16;
    if (few > S / 2 && (a.N / 32 * all >= 256 || few >= 8))
      return launch_w4_few_rows<S, true, SB, VEC, Z>(a, act, stream);
  }
  return launch_w4_few_rows<S, false, SB, VEC, Z>(a, act, stream);
}

template <int S, bool SB, bool VEC>
static hipError_t launch_w4_few(const W4Args& a, int act, hipStream_t stream) {
  return a.zeros ? launch_w4_few_z<S, SB, VEC, true>(a, act, stream) : launch_w4_few_z<S, SB, VEC, false>(a, act, stream);
}

static int w4_groups_per_chunk(int32_t G) { return G >= 128 ? 1 : 128 / G; }

int64_t w4_workgroups(int32_t N, int32_t G, int32_t T, int32_t k, int pairs, int sum, int act) {
  const int per = 16 / w4_groups_per_chunk(G);
  const int64_t rows = pairs ? (sum ? T : (int64_t)T * k) : ((int64_t)T + per - 1) / per;
  return rows * (((int64_t)(act ? N / 2 : N) + 15) / 16 + 8);
}

hipError_t launch_w4_gemv(const uint8_t* codes, const void* scales, int scale_bf16, const uint8_t* zeros, int32_t G,
                          int32_t E, int32_t N, int32_t K, const uint16_t* x, int x_pairs, int32_t T,
                          const int32_t* ids, const float* weights, int32_t k, void* y, int y_bf16, int act,
                          hipStream_t stream) {
  W4Args a;
  a.codes = codes;
  a.scales = scales;
  a.zeros = zeros;
  a.x = x;
  a.ids = ids;
  a.weights = weights;
  a.y = y;
  a.N = N;
  a.K = K;
  a.groups = K / G;
  a.E = E;
  a.T = T;
  a.k = k;
  a.gshift = __builtin_ctz((unsigned)G);
  a.x_pairs = x_pairs;
  a.scale_bf16 = scale_bf16;
  a.y_bf16 = y_bf16;
  a.col_groups = 0;
  // One row: a lane's own codes, the fewest instructions and cache accesses a
  // code (131,072 x 4,096, groups of 128: 48 us, 53 for two rows of the other).
  // More: 16 columns at a time (4,096 x 4,096, 4 rows, groups of 32: 6.1 us; the
  // lane kernel with four rows in registers took 7.6, with eight 11.6).
  if (ids || T == 1) {
    if (scale_bf16) return zeros ? launch_w4_lane<true, true>(a, act, stream) : launch_w4_lane<true, false>(a, act, stream);
    return zeros ? launch_w4_lane<false, true>(a, act, stream) : launch_w4_lane<false, false>(a, act, stream);
  }
  const int S = w4_groups_per_chunk(G);
  const uintptr_t run = S * (scale_bf16 ? 2 : 4);
  const bool vec = a.groups % S == 0 && ((uintptr_t)scales & (run - 1)) == 0 && ((uintptr_t)zeros & (S - 1)) == 0;
#define MOE_W4(SV, VECV) \
  (scale_bf16 ? launch_w4_few<SV, true, VECV>(a, act, stream) : launch_w4_few<SV, false, VECV>(a, act, stream))
  if (S == 4) return vec ? MOE_W4(4, true) : MOE_W4(4, false);
  if (S == 2) return vec ? MOE_W4(2, true) : MOE_W4(2, false);
  return MOE_W4(1, true);
#undef MOE_W4
}

}  // namespace moe
