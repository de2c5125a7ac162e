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
// MFMA mapping (v_mfma_f32_16x16x32_bf16).  A wave takes chunks of 128 k of
// 16 columns: lane l loads the 16 bytes of column n = l & 15 and 32-block
// g = l >> 4, and one of four steps multiplies 8 k of all four blocks.  Summing
// over the lane groups would mix scales, so x is laid out block-diagonally:
// row r of the first operand is token r / S with the lanes of group r % S alone
// (S = 128 / G groups a chunk, at least 1), the rest zero.  The 16 rows hold
// 16 / S tokens, and every lane of the result holds whole group sums of one
// column.
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

// What one chunk of CT column tiles and NB token blocks needs, as it lies in
// memory.
template <int S, int NB, int CT>
struct W4Chunk {
  u32x4_t codes[CT];
  uint32_t scale[CT][S];     // f32 words, or bf16 pairs in the first (S + 1) / 2
  uint32_t zero[CT];         // a byte per group
  u32x4_t x[NB][4];
  float factor;              // router weight of the chunk's expert
};

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

// S: scale groups a 128-k chunk (4, 2, or 1: G >= 128).  NB: blocks of 16 / S
// tokens.  CT: 16-column tiles of a wave, with ACT half of them gate and half
// up columns.  SUM: a row sums the chosen experts of a token, whose chunks
// follow one another.  SB: bf16 scales.  VEC: the scales and zero points of a
// chunk start at whole words.  D: chunks in flight.
//
// Every load is a bounded buffer load: lanes and chunks that do not exist read
// zeros and need no branch, which would make the compiler wait for the loads in
// flight where the paths meet.
template <int S, int NB, int CT, bool ACT, bool SUM, bool SB, bool VEC, int D>
__global__ __launch_bounds__(512) void w4_gemv_kernel(W4Args p) {
  constexpr int R = 4 / S;               // tokens a lane holds of a block
  constexpr int TB = 16 / S * NB;        // tokens of a workgroup
  constexpr int CW = (ACT ? CT / 2 : CT) * 16;
  constexpr int SZ = SB ? 2 : 4;
  extern __shared__ float s_part[];      // [waves][NB * CT * R][64]

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int n16 = lane & 15, g = lane >> 4;
  const int cg = blockIdx.x % (uint32_t)p.col_groups;
  const int rb = blockIdx.x / (uint32_t)p.col_groups;
  const int64_t N = p.N, K = p.K, groups = p.groups;
  const int cols = (int)(ACT ? N / 2 : N);
  const int KC = (int)((K + 127) >> 7);
  const bool pairs = p.ids != nullptr;

  // first column of each tile, and its columns that exist
  int64_t col0[CT];
  int have[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int at = cg * CW + (ACT ? c % (CT / 2) : c) * 16;
    have[c] = max(0, min(16, cols - at));
    col0[c] = at + (ACT && c >= CT / 2 ? N / 2 : 0);
  }
  const uint32_t cvo = (uint32_t)(n16 * (K / 2) + g * 16);
  const uint32_t svo = (uint32_t)(n16 * groups * SZ), zvo = (uint32_t)(n16 * groups);
  uint32_t xvo[NB];                      // the row of x that this lane's operand row takes
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const bool mine = S == 1 || (S == 2 ? (g >> 1) == (n16 & 1) : g == (n16 & 3));
    const int t = b * (16 / S) + n16 / S;
    xvo[b] = mine && (pairs ? t == 0 : rb * TB + t < p.T) ? (uint32_t)(t * K * 2 + g * 64) : kLaneOob;
  }
  const int x_rows = pairs ? 1 : min(TB, p.T - rb * TB);

  float acc[NB][CT][R];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < R; ++i) acc[b][c][i] = 0.f;

  const int total = (SUM ? p.k : 1) * KC;
  const int share = (total + waves - 1) / waves;
  const int first = wave * share, end = min(first + share, total);

  // The next chunk to load: chunk kc of pair `pair`, whose expert is e.
  int v = first, pair = SUM ? rb * p.k + first / KC : rb, kc = SUM ? first % KC : first;
  int64_t e = 0, xrow = pairs ? 0 : (int64_t)rb * TB;
  bool live = true;
  float factor = 1.f;
  auto expert = [&]() __attribute__((always_inline)) {
    const int id = p.ids[pair];
    live = (uint32_t)id < (uint32_t)p.E;
    e = live ? id : 0;
    xrow = p.x_pairs ? pair : pair / p.k;
    if (SUM) factor = live ? p.weights[pair] : 0.f;
  };
  if (pairs && v < end) expert();

  typedef W4Chunk<S, NB, CT> Chunk;
  auto load = [&](Chunk& q) __attribute__((always_inline)) {
    const bool on = live && v < end;
    q.factor = factor;
    const __amdgpu_buffer_rsrc_t xr = w4_rsrc(p.x, xrow * K * 2, on ? x_rows * K * 2 : 0);
    const bool in = kc * 128 + g * 32 < K;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        q.x[b][s] = __builtin_amdgcn_raw_buffer_load_b128(xr, (in ? xvo[b] : kLaneOob) + s * 16, kc * 256, 0);
    const int gi = S > 1 ? kc * S : (int)(((int64_t)kc * 128) >> p.gshift);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int64_t row = e * N + col0[c];
      const int rows = on ? have[c] : 0;
      q.codes[c] = __builtin_amdgcn_raw_buffer_load_b128(w4_rsrc(p.codes, row * (K / 2), rows * (K / 2)), cvo, kc * 64, 0);
      w4_load_scales<S, SB, VEC>(w4_rsrc(p.scales, row * groups * SZ, rows * groups * SZ), svo, gi * SZ,
                                 (int)groups - gi, q.scale[c]);
      q.zero[c] = w4_load_zeros<S, VEC>(w4_rsrc(p.zeros, row * groups, p.zeros ? rows * groups : 0), zvo, gi);
    }
    ++v;
    if (++kc == KC && SUM) {
      kc = 0;
      ++pair;
      if (v < end) expert();
    }
  };
  const float zero_base = p.zeros ? 0.f : 8.f;

  auto use = [&](const Chunk& q) __attribute__((always_inline)) {
    f32x4_t d[NB][CT], sx[NB];
    const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      sx[b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < CT; ++c) d[b][c] = sx[b];
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4_t w[CT];
#pragma unroll
      for (int c = 0; c < CT; ++c) w[c] = codes_to_bf16(q.codes[c][s]);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const u32x4_t x = x_order(q.x[b][s]);
        sx[b] = w4_mfma(x, ones, sx[b]);
#pragma unroll
        for (int c = 0; c < CT; ++c) d[b][c] = w4_mfma(x, w[c], d[b][c]);
      }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      float s[S], z[S];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        s[i] = SB ? ((i & 1) ? bf16_hi(q.scale[c][i >> 1]) : bf16_lo(q.scale[c][i >> 1]))
                  : __uint_as_float(q.scale[c][i]);
        if (SUM) s[i] *= q.factor;
        z[i] = zero_base + (float)((q.zero[c] >> (8 * i)) & 0xFFu);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = fmaf(-z[i % S], sx[b][i], d[b][c][i]);
          acc[b][c][i / S] = fmaf(s[i % S], f, acc[b][c][i / S]);
        }
    }
  };

  Chunk ring[D];
#pragma unroll
  for (int i = 0; i < D; ++i) {
    load(ring[i]);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int u = first; u < end; u += D) {
#pragma unroll
    for (int i = 0; i < D; ++i) {
      use(ring[i]);
      load(ring[i]);
    }
  }

  // the waves' shares, added in the waves' order
  constexpr int V = NB * CT * R;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < R; ++i) s_part[(wave * V + (b * CT + c) * R + i) * 64 + lane] = acc[b][c][i];
  __syncthreads();
  auto total_of = [&](int v, int l) {
    float f = s_part[v * 64 + l];
    for (int w = 1; w < waves; ++w) f += s_part[(w * V + v) * 64 + l];
    return f;
  };
  constexpr int OC = ACT ? CT / 2 : CT;
  for (int o = threadIdx.x; o < NB * OC * R * 64; o += blockDim.x) {
    const int l = o & 63, i = (o >> 6) % R, c = (o >> 6) / R % OC, b = (o >> 6) / R / OC;
    const int t = b * (16 / S) + (l >> 4) * R + i;   // token of the workgroup's
    const int64_t row = pairs ? rb : (int64_t)rb * TB + t;
    const int col = cg * CW + c * 16 + (l & 15);
    if (col >= cols || (pairs ? t != 0 : row >= p.T)) continue;
    float f = total_of((b * CT + c) * R + i, l);
    if (ACT) {
      const float u = total_of((b * CT + c + OC) * R + i, l);
      f = f / (1.0f + __expf(-f)) * u;
    }
    const int64_t at = row * cols + col;
    if (p.y_bf16) reinterpret_cast<uint16_t*>(p.y)[at] = f32_to_bf16_rne(f);
    else reinterpret_cast<float*>(p.y)[at] = f;
  }
}

template <int S, int NB, int CT, bool ACT, bool SUM, bool SB, bool VEC, int D>
static hipError_t launch_w4_t(W4Args a, int64_t row_blocks, hipStream_t stream) {
  const int64_t cols = ACT ? a.N / 2 : a.N;
  constexpr int CW = (ACT ? CT / 2 : CT) * 16;
  a.col_groups = (int)((cols + CW - 1) / CW);
  const int64_t groups = row_blocks * a.col_groups;
  const int64_t chunks = (a.K + 127) / 128 * (SUM ? a.k : 1);
  const int waves = groups * 4 < 2048 && chunks >= 8 ? 8 : 4;
  const size_t lds = (size_t)waves * NB * CT * (4 / S) * 64 * 4;
  hipLaunchKernelGGL((w4_gemv_kernel<S, NB, CT, ACT, SUM, SB, VEC, D>), dim3((unsigned)groups), dim3(waves * 64), lds,
                     stream, a);
  return hipGetLastError();
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

// v of the lane that a quad permutation names.
template <int CTRL>
__device__ __forceinline__ float quad_xor(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

// Lane sums: for up to TT tokens a wave multiplies 4 rows x 512 k of codes at a
// time, 1 KiB in one load of whole 256-byte runs.  Lane l holds 32 codes of one
// row, r = (l & 15) >> 2, and one 32-block, b = 4 (l >> 4) + (l & 3), and needs
// the sum over just these.  The matrix unit adds over the four lanes groups of a
// column and shares x between columns, so x is laid out with a row per block:
// row 4 g + s of the first operand holds x of block 4 g + s in lane group g and
// zeros elsewhere.  Result register i of lane l is then block 4 (l >> 4) + i
// against the codes of column l & 15, of which the lane's own is i = l & 3.  The
// lane's scale and zero point are those of the block, loaded as it loads the
// codes; x and its block sums stay in registers for all rows.
//
// Waves of a workgroup take units of 512 k (of a token's experts one after the
// other: SUM) of the same rows, blocks of 8 row quads after one another (with
// ACT 4 quads of gate rows and the 4 of up rows).  A wave's loads run through
// all of its blocks and units in a ring; a block's sums over the lanes of a row
// and over the waves are joined in LDS, in order, while the next block's loads
// are on their way.
constexpr int W4_NT = 2;       // non-temporal: codes are read once
constexpr int W4_LANE_TOKENS = 16;
constexpr int W4_WAVES = 8;
constexpr int W4_RING = 8;     // loads of 1 KiB in flight per wave, and row quads of a block

struct W4LaneArgs {
  W4Args a;
  int blocks;                  // of a workgroup
};

template <int TT, bool ACT, bool SUM, bool SB, bool Z>
__global__ __launch_bounds__(W4_WAVES * 64) void w4_lane_kernel(W4LaneArgs la) {
  const W4Args& p = la.a;
  constexpr int SZ = SB ? 2 : 4;
  constexpr int HALF = ACT ? W4_RING / 2 : W4_RING;   // quads of a block that are rows of y
  __shared__ __attribute__((aligned(16))) float s_sum[2][W4_RING * TT][W4_WAVES][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int g = lane >> 4, q4 = lane & 3, r = (lane & 15) >> 2;
  const int block = g * 4 + q4;
  const int K = (int)p.K, groups = (int)p.groups;
  const int64_t N = p.N;
  const int cols = (int)(ACT ? N / 2 : N);
  const int cg = blockIdx.x % (uint32_t)p.col_groups;
  const int rb = blockIdx.x / (uint32_t)p.col_groups;
  const bool pairs = p.ids != nullptr;
  const int tokens = pairs ? 1 : min(TT, p.T - rb * TT);

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
    Unit n = {0, pairs ? 0 : (int64_t)rb * TT, SUM ? u - j * per : u, u < total, 1.f};
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

  u32x4_t x[TT][4], xn[TT][4];
  float sx[TT], factor = 1.f, nfactor = 1.f;
  auto load_x = [&](const Unit& n, u32x4_t (&to)[TT][4], float& f) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t xr = w4_rsrc(p.x, n.xrow * K * 2, n.live ? (int64_t)tokens * K * 2 : 0);
    const uint32_t xvo = n.c * 512 + block * 32 < K && diag ? (uint32_t)(n.c * 1024 + block * 64) : kLaneOob;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int s = 0; s < 4; ++s) to[t][s] = __builtin_amdgcn_raw_buffer_load_b128(xr, xvo + s * 16, t * K * 2, 0);
    f = n.factor;
  };
  auto sum_x = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      f32x4_t d = zero4;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        x[t][s] = x_order(x[t][s]);
        d = w4_mfma(x[t][s], ones, d);
      }
      sx[t] = own(d);
    }
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
      // one token: the next unit's x (the last one's: the first of the next
      // block) comes ahead of the loads that follow it
      constexpr bool AHEAD = TT == 1;
      auto next_x = [&]() __attribute__((always_inline)) { return unit(u + waves < total ? u + waves : wave); };
      if (AHEAD && total > waves) load_x(next_x(), xn, nfactor);
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
        // sums of the row's 64 bytes, in all four of their lanes; lane q4 keeps
        // those of token q4 of four.  (Tokens of a call that TT exceeds are
        // zeros: a branch around them would keep the chains of matrix
        // instructions from overlapping.)
#pragma unroll
        for (int t0 = 0; t0 < TT; t0 += 4) {
          constexpr int C = TT < 4 ? TT : 4;
          f32x4_t d[C];
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int t = 0; t < C; ++t)
              if (t0 + t < TT) d[t] = w4_mfma(x[t0 + t][s], w[s], s ? d[t] : zero4);
          float keep = 0.f;
#pragma unroll
          for (int t = 0; t < C; ++t)
            if (t0 + t < TT) {
              float f = sc * fmaf(-z, sx[t0 + t], own(d[t]));
              f += quad_xor<0xB1>(f);
              f += quad_xor<0x4E>(f);
              keep = t == 0 || q4 == t ? f : keep;
            }
          if (t0 + q4 < TT) {
            float* to = &sums[i * TT + t0 + q4][wave][r * 4 + g];
            *to = u == wave ? keep : *to + keep;
          }
        }
      }
      next_unit();
      if (total > waves) {
        if (AHEAD) {
#pragma unroll
          for (int s = 0; s < 4; ++s) x[0][s] = xn[0][s];
          factor = nfactor;
        } else {
          load_x(next_x(), x, factor);
        }
        sum_x();
      }
    }
    lds_barrier();

    // eight lanes add up a row, one a wave
    const int w = threadIdx.x & 7;
    const int live = min(rows - b * HALF * 4, HALF * 4);    // rows of y of the block
    auto total_of = [&](int quad, int t, int row) __attribute__((always_inline)) {
      float f = 0.f;
      if (w < min(waves, total)) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&sums[quad * TT + t][w][row * 4]);
        f = (v[0] + v[1]) + (v[2] + v[3]);
      }
      f += quad_xor<0xB1>(f);
      f += quad_xor<0x4E>(f);
      return f + quad_xor<0x141>(f);                        // the other quad of eight lanes
    };
    for (int o = threadIdx.x >> 3; o < HALF * 4 * TT; o += blockDim.x >> 3) {
      const int t = o % TT, row = o / TT;
      float f = total_of(row >> 2, t, row & 3);
      if (ACT) f = f / (1.0f + __expf(-f)) * total_of(HALF + (row >> 2), t, row & 3);
      if (w != 0 || t >= tokens || row >= live) continue;
      const int64_t at = ((pairs ? rb : (int64_t)rb * TT) + t) * cols + row0 + b * HALF * 4 + row;
      if (p.y_bf16) reinterpret_cast<uint16_t*>(p.y)[at] = f32_to_bf16_rne(f);
      else reinterpret_cast<float*>(p.y)[at] = f;
    }
  }
}

template <int TT, bool ACT, bool SUM, bool SB, bool Z>
static hipError_t launch_w4_lane_t(const W4Args& a, int64_t row_blocks, hipStream_t stream) {
  W4LaneArgs la = {a, 0};
  const int64_t cols = ACT ? a.N / 2 : a.N;
  constexpr int ROWS = 4 * (ACT ? W4_RING / 2 : W4_RING);
  const int64_t blocks = (cols + ROWS - 1) / ROWS;
  const int64_t units = (a.K + 511) / 512 * (SUM ? a.k : 1);
  const int waves = units < W4_WAVES ? (int)units : W4_WAVES;
  // as many workgroups as the CUs hold at once, where there are as many blocks
  const int64_t room = TT == 1 ? 512 : 256;
  const int64_t per = (blocks * row_blocks + room - 1) / room;
  la.blocks = (int)(per < blocks ? per : blocks);
  la.a.col_groups = (int)((blocks + la.blocks - 1) / la.blocks);
  hipLaunchKernelGGL((w4_lane_kernel<TT, ACT, SUM, SB, Z>), dim3((unsigned)(row_blocks * la.a.col_groups)),
                     dim3(waves * 64), 0, stream, la);
  return hipGetLastError();
}

template <bool SB, bool Z>
static hipError_t launch_w4_lane(const W4Args& a, int act, hipStream_t stream) {
  if (a.weights) return launch_w4_lane_t<1, false, true, SB, Z>(a, a.T, stream);
  if (a.ids || a.T == 1) {
    const int64_t rows = a.ids ? (int64_t)a.T * a.k : 1;
    return act ? launch_w4_lane_t<1, true, false, SB, Z>(a, rows, stream)
               : launch_w4_lane_t<1, false, false, SB, Z>(a, rows, stream);
  }
  const int64_t blocks = a.T <= 8 ? 1 : ((int64_t)a.T + 7) / 8;
  switch (a.T <= 8 ? a.T : (int)((a.T + blocks - 1) / blocks)) {
#define MOE_CASE(TT)                                                       \
  return act ? launch_w4_lane_t<TT, true, false, SB, Z>(a, blocks, stream) \
             : launch_w4_lane_t<TT, false, false, SB, Z>(a, blocks, stream)
    case 2: MOE_CASE(2);
    case 3: MOE_CASE(3);
    case 4: MOE_CASE(4);
    case 5: MOE_CASE(5);
    case 6: MOE_CASE(6);
    default: MOE_CASE(8);
#undef MOE_CASE
  }
}

// ---------------------------------------------------------------------------
// A few more tokens: x in registers, 16 columns at a time
// ---------------------------------------------------------------------------

// Up to 16 / S tokens of a dense product.  The operands are laid out as in
// w4_gemv_kernel (one block of tokens), and the walk is w4_lane_kernel's: a wave
// keeps x of its 512 k (four chunks) in registers, with the sums of x per group,
// and goes through 16-column tiles, two to a block (with ACT a gate and an up
// tile).  A tile's scales and zero points are loaded by lane group g for chunk g
// and handed to the lanes that need them through the LDS crossbar.
constexpr int W4_TILES = 4;    // of 4 KiB in flight per wave, and of a block

template <int S, bool ACT, bool SB, bool VEC, bool Z>
__global__ __launch_bounds__(W4_WAVES * 64) void w4_few_kernel(W4LaneArgs la) {
  const W4Args& p = la.a;
  constexpr int SZ = SB ? 2 : 4;
  constexpr int SW = SB ? (S + 1) / 2 : S;            // scale words of a chunk
  constexpr int R = 4 / S;                            // tokens a lane holds
  constexpr int BT = W4_TILES, HALF = ACT ? BT / 2 : BT;   // tiles of a block; of y's columns
  __shared__ float s_sum[2][BT * R][W4_WAVES][64];
  __shared__ __attribute__((aligned(256))) uint8_t s_codes[W4_WAVES][4096];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int n16 = lane & 15, g = lane >> 4;
  const int K = (int)p.K, groups = (int)p.groups;
  const int64_t N = p.N;
  const int cols = (int)(ACT ? N / 2 : N);

  const int row0 = blockIdx.x * la.blocks * HALF * 16;   // first column of y
  const int rows = min(la.blocks * HALF * 16, cols - row0);
  const int blocks = (rows + HALF * 16 - 1) / (HALF * 16);
  const int total = (K + 511) >> 9;

  // load c of a tile: rows 4 c + g, their 256 bytes; through LDS, row n's
  // 16-byte segment s at place s ^ n
  const uint32_t cvo = (uint32_t)g * (uint32_t)(K / 2) + n16 * 16;
  uint8_t* own = s_codes[wave];
  const uint32_t srow = (uint32_t)(n16 * groups);
  const bool mine = S == 1 || (S == 2 ? (g >> 1) == (n16 & 1) : g == (n16 & 3));
  const uint32_t xrow = mine && n16 / S < p.T ? (uint32_t)(n16 / S * K * 2 + g * 64) : kLaneOob;

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
  f32x4_t sx[4];
  const __amdgpu_buffer_rsrc_t xr = w4_rsrc(p.x, 0, (int64_t)p.T * K * 2);
  auto load_x = [&](int u) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool in = u * 512 + c * 128 + g * 32 < K;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        x[c][s] = __builtin_amdgcn_raw_buffer_load_b128(xr, (in ? xrow : kLaneOob) + s * 16, u * 1024 + c * 256, 0);
    }
  };
  auto sum_x = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      sx[c] = zero4;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        x[c][s] = x_order(x[c][s]);
        sx[c] = w4_mfma(x[c][s], ones, sx[c]);
      }
    }
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
        f32x4_t d[4];
        uint32_t sw[4][S], zw[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int from = (n16 | c << 4) << 2;
#pragma unroll
          for (int j = 0; j < SW; ++j) sw[c][j] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)ring[i].scale[j]);
          zw[c] = Z ? (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)ring[i].zero) : 0x08080808u;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<u32x4_t*>(own + (c * 4 + g) * 256 + ((n16 ^ (c * 4 + g)) << 4)) = ring[i].codes[c];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        u32x4_t q[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          q[c] = *reinterpret_cast<const u32x4_t*>(own + n16 * 256 + (((c * 4 + g) ^ n16) << 4));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          d[c] = zero4;
#pragma unroll
          for (int s = 0; s < 4; ++s) d[c] = w4_mfma(x[c][s], codes_to_bf16(q[c][s]), d[c]);
        }
        __builtin_amdgcn_sched_barrier(0);
        load(i, ring[i]);
        __builtin_amdgcn_sched_barrier(0);
        float acc[R];
#pragma unroll
        for (int j = 0; j < R; ++j) acc[j] = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int o = j % S;
            const float sc = SB ? ((o & 1) ? bf16_hi(sw[c][o >> 1]) : bf16_lo(sw[c][o >> 1])) : __uint_as_float(sw[c][o]);
            const float z = (float)((zw[c] >> (8 * o)) & 0xFFu);
            acc[j / S] = fmaf(sc, fmaf(-z, sx[c][j], d[c][j]), acc[j / S]);
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

    const int live_waves = min(waves, total);
    const int live = min(rows - b * HALF * 16, HALF * 16);
    for (int o = threadIdx.x; o < HALF * R * 64; o += blockDim.x) {
      const int l = o & 63, j = (o >> 6) % R, c = (o >> 6) / R;
      const int t = (l >> 4) * R + j, col = c * 16 + (l & 15);
      if (t >= p.T || col >= live) continue;
      float f = 0.f, h = 0.f;
      for (int w = 0; w < live_waves; ++w) {
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

template <int S, bool ACT, bool SB, bool VEC, bool Z>
static hipError_t launch_w4_few_t(const W4Args& a, hipStream_t stream) {
  W4LaneArgs la = {a, 0};
  const int64_t cols = ACT ? a.N / 2 : a.N;
  constexpr int COLS = 16 * (ACT ? W4_TILES / 2 : W4_TILES);
  const int64_t blocks = (cols + COLS - 1) / COLS;
  const int64_t units = (a.K + 511) / 512;
  const int waves = units < W4_WAVES ? (int)units : W4_WAVES;
  const int64_t per = (blocks + 255) / 256;
  la.blocks = (int)per;
  hipLaunchKernelGGL((w4_few_kernel<S, ACT, SB, VEC, Z>), dim3((unsigned)((blocks + per - 1) / per)), dim3(waves * 64),
                     0, stream, la);
  return hipGetLastError();
}

template <int S, bool SB, bool VEC>
static hipError_t launch_w4_few(const W4Args& a, int act, hipStream_t stream) {
  if (a.zeros) return act ? launch_w4_few_t<S, true, SB, VEC, true>(a, stream) : launch_w4_few_t<S, false, SB, VEC, true>(a, stream);
  return act ? launch_w4_few_t<S, true, SB, VEC, false>(a, stream) : launch_w4_few_t<S, false, SB, VEC, false>(a, stream);
}

// Tokens of a workgroup for T rows of a dense product.
static int w4_blocks(int64_t rows, int S) {
  const int64_t need = (rows * S + 15) / 16;
  return need <= 1 ? 1 : need <= 2 ? 2 : 4;
}

static int w4_groups_per_chunk(int32_t G) { return G >= 128 ? 1 : 128 / G; }

int64_t w4_workgroups(int32_t N, int32_t G, int32_t T, int32_t k, int pairs, int sum, int act) {
  const int S = w4_groups_per_chunk(G);
  const int nb = pairs ? 1 : w4_blocks(T, S);
  const int64_t rows = pairs ? (sum ? T : (int64_t)T * k) : ((int64_t)T + 16 / S * nb - 1) / (16 / S * nb);
  return rows * (((act ? N / 2 : N) + 15) / 16);
}

template <int S, bool SB, bool VEC>
static hipError_t launch_w4_s(const W4Args& a, int act, hipStream_t stream) {
  if (a.ids) {
    if (a.weights) return launch_w4_t<S, 1, 2, false, true, SB, VEC, 3>(a, a.T, stream);
    const int64_t rows = (int64_t)a.T * a.k;
    return act ? launch_w4_t<S, 1, 2, true, false, SB, VEC, 3>(a, rows, stream)
               : launch_w4_t<S, 1, 2, false, false, SB, VEC, 3>(a, rows, stream);
  }
  const int nb = w4_blocks(a.T, S);
  const int64_t blocks = ((int64_t)a.T + 16 / S * nb - 1) / (16 / S * nb);
  if (nb == 1)
    return act ? launch_w4_t<S, 1, 2, true, false, SB, VEC, 3>(a, blocks, stream)
               : launch_w4_t<S, 1, 2, false, false, SB, VEC, 3>(a, blocks, stream);
  if (nb == 2)
    return act ? launch_w4_t<S, 2, 2, true, false, SB, VEC, 2>(a, blocks, stream)
               : launch_w4_t<S, 2, 2, false, false, SB, VEC, 2>(a, blocks, stream);
  return act ? launch_w4_t<S, 4, 2, true, false, SB, VEC, 1>(a, blocks, stream)
             : launch_w4_t<S, 4, 2, false, false, SB, VEC, 1>(a, blocks, stream);
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
  const int S = w4_groups_per_chunk(G);
  const uintptr_t run = S * (scale_bf16 ? 2 : 4);
  const bool vec = a.groups % S == 0 && ((uintptr_t)scales & (run - 1)) == 0 && ((uintptr_t)zeros & (S - 1)) == 0;
  if (!ids && T > 1 && T <= 16 / S) {
#define MOE_W4(SV, VECV) \
  (scale_bf16 ? launch_w4_few<SV, true, VECV>(a, act, stream) : launch_w4_few<SV, false, VECV>(a, act, stream))
    if (S == 4) return vec ? MOE_W4(4, true) : MOE_W4(4, false);
    if (S == 2) return vec ? MOE_W4(2, true) : MOE_W4(2, false);
    return MOE_W4(1, true);
#undef MOE_W4
  }
  if (ids || T <= W4_LANE_TOKENS) {
    if (scale_bf16) return zeros ? launch_w4_lane<true, true>(a, act, stream) : launch_w4_lane<true, false>(a, act, stream);
    return zeros ? launch_w4_lane<false, true>(a, act, stream) : launch_w4_lane<false, false>(a, act, stream);
  }
#define MOE_W4(SV, VECV) \
  (scale_bf16 ? launch_w4_s<SV, true, VECV>(a, act, stream) : launch_w4_s<SV, false, VECV>(a, act, stream))
  if (S == 4) return vec ? MOE_W4(4, true) : MOE_W4(4, false);
  if (S == 2) return vec ? MOE_W4(2, true) : MOE_W4(2, false);
  return MOE_W4(1, true);
#undef MOE_W4
}

}  // namespace moe
