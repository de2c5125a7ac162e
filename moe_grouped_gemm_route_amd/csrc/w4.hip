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

// Eight codes of a word, k ascending, as bf16 integers.
__device__ __forceinline__ u32x4_t codes_to_bf16(uint32_t q) {
  const uint32_t even = q & 0x0F0F0F0Fu, odd = (q >> 4) & 0x0F0F0F0Fu;
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u);   // k 0 1 2 3
  const uint32_t hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);   // k 4 5 6 7
  u32x4_t r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
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

// S: scale groups a 128-k chunk (4, 2, or 1: G >= 128).  NB: blocks of 16 / S
// tokens.  CT: 16-column tiles of a wave, with ACT half of them gate and half
// up columns.  D: chunks in flight.
template <int S, int NB, int CT, bool ACT, int D>
__global__ __launch_bounds__(512) void w4_gemv_kernel(W4Args p) {
  constexpr int R = 4 / S;               // tokens a lane holds of a block
  constexpr int TB = 16 / S * NB;        // tokens of a workgroup
  constexpr int CW = (ACT ? CT / 2 : CT) * 16;
  extern __shared__ float s_part[];      // [waves][NB * CT * R][64]

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int n16 = lane & 15, g = lane >> 4;
  const int cg = blockIdx.x % (uint32_t)p.col_groups;
  const int rb = blockIdx.x / (uint32_t)p.col_groups;
  const int64_t N = p.N, K = p.K;
  const int cols = (int)(ACT ? N / 2 : N);
  const int KC = (int)((K + 127) >> 7);

  // rows of x: a block of tokens, the one of a pair, or those of a token's pairs
  const bool pairs = p.ids != nullptr, sum = p.weights != nullptr;
  const int per_row = sum ? p.k : 1;     // experts that add up to the row

  int64_t row_of[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int tile = ACT ? c % (CT / 2) : c;
    const int n = min(cg * CW + tile * 16 + n16, cols - 1);
    row_of[c] = n + (ACT && c >= CT / 2 ? N / 2 : 0);
  }
  int token[NB];                         // row of x that this lane's operand row takes, or -1
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int r = lane & 15;
    const bool mine = S == 1 || (S == 2 ? (g >> 1) == (r & 1) : g == (r & 3));
    const int t = pairs ? r / S : rb * TB + b * (16 / S) + r / S;
    token[b] = mine && (pairs ? t == 0 && b == 0 : t < p.T) ? t : -1;
  }

  float acc[NB][CT][R];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int i = 0; i < R; ++i) acc[b][c][i] = 0.f;

  const int total = per_row * KC;
  const int share = (total + waves - 1) / waves;
  const int first = wave * share, count = min(share, total - first);

  typedef W4Chunk<S, NB, CT> Chunk;
  auto load = [&](int v, Chunk& q) __attribute__((always_inline)) {
    v += first;
    const int j = per_row == 1 ? 0 : v / KC;
    const int kc = v - j * KC;
    int64_t e = 0, xrow = 0;
    bool live = true;
    q.factor = 1.f;
    if (pairs) {
      const int pair = rb * per_row + j;
      const int id = p.ids[pair];
      live = (uint32_t)id < (uint32_t)p.E;
      e = live ? id : 0;
      xrow = p.x_pairs ? pair : pair / p.k;
      if (sum) q.factor = live ? p.weights[pair] : 0.f;
    }
    const int64_t k0 = (int64_t)kc * 128 + g * 32;
    const bool in = live && k0 < K;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const bool on = in && token[b] >= 0;
      const u32x4_t* xp = reinterpret_cast<const u32x4_t*>(p.x + (xrow + (on ? token[b] : 0)) * K + (on ? k0 : 0));
#pragma unroll
      for (int s = 0; s < 4; ++s) q.x[b][s] = on ? xp[s] : u32x4_t{0, 0, 0, 0};
    }
    const int64_t gi = S > 1 ? (int64_t)kc * S : ((int64_t)kc * 128) >> p.gshift;
    const bool whole = S == 1 || (int64_t)kc * 128 + 128 <= K;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int64_t row = e * N + row_of[c];
      q.codes[c] = in ? *reinterpret_cast<const u32x4_t*>(p.codes + row * (K / 2) + (k0 >> 1)) : u32x4_t{0, 0, 0, 0};
      const uint8_t* sp = reinterpret_cast<const uint8_t*>(p.scales) + (row * p.groups + gi) * (p.scale_bf16 ? 2 : 4);
      const uint8_t* zp = p.zeros + row * p.groups + gi;
#pragma unroll
      for (int i = 0; i < S; ++i) q.scale[c][i] = 0;
      q.zero[c] = 0x08080808u;
      if (live && whole) {
        // the runs of a chunk's groups start anywhere: whole words of any alignment
        if (p.scale_bf16) __builtin_memcpy(q.scale[c], sp, 2 * S);
        else __builtin_memcpy(q.scale[c], sp, 4 * S);
        if (p.zeros) {
          q.zero[c] = 0;
          __builtin_memcpy(&q.zero[c], zp, S);
        }
      } else if (live) {
        const int left = (int)(p.groups - gi);       // groups of the last, short chunk
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int at = min(i, left - 1);
          if (p.scale_bf16) {
            const uint32_t h = reinterpret_cast<const uint16_t*>(sp)[at];
            q.scale[c][i >> 1] |= h << (16 * (i & 1));
          } else {
            q.scale[c][i] = reinterpret_cast<const uint32_t*>(sp)[at];
          }
          if (p.zeros) q.zero[c] = (q.zero[c] & ~(0xFFu << (8 * i))) | ((uint32_t)zp[at] << (8 * i));
        }
      }
    }
  };

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
        sx[b] = w4_mfma(q.x[b][s], ones, sx[b]);
#pragma unroll
        for (int c = 0; c < CT; ++c) d[b][c] = w4_mfma(q.x[b][s], w[c], d[b][c]);
      }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      float s[S], z[S];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const float f = p.scale_bf16 ? ((i & 1) ? bf16_hi(q.scale[c][i >> 1]) : bf16_lo(q.scale[c][i >> 1]))
                                     : __uint_as_float(q.scale[c][i]);
        s[i] = f * q.factor;
        z[i] = (float)((q.zero[c] >> (8 * i)) & 0xFFu);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = fmaf(-z[i % S], sx[b][i], d[b][c][i]);
          acc[b][c][i / S] = fmaf(s[i % S], v, acc[b][c][i / S]);
        }
    }
  };

  Chunk ring[D];
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (i < count) load(i, ring[i]);
  for (int v = 0; v < count; v += D) {
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (v + i < count) {
        use(ring[i]);
        if (v + i + D < count) load(v + i + D, ring[i]);
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

template <int S, int NB, int CT, bool ACT, int D>
static hipError_t launch_w4_t(W4Args a, int64_t row_blocks, hipStream_t stream) {
  const int64_t cols = ACT ? a.N / 2 : a.N;
  constexpr int CW = (ACT ? CT / 2 : CT) * 16;
  a.col_groups = (int)((cols + CW - 1) / CW);
  const int64_t groups = row_blocks * a.col_groups;
  const int64_t chunks = (a.K + 127) / 128 * (a.weights ? a.k : 1);
  const int waves = groups * 4 < 2048 && chunks >= 8 ? 8 : 4;
  const size_t lds = (size_t)waves * NB * CT * (4 / S) * 64 * 4;
  hipLaunchKernelGGL((w4_gemv_kernel<S, NB, CT, ACT, D>), dim3((unsigned)groups), dim3(waves * 64), lds, stream, a);
  return hipGetLastError();
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

template <int S, bool ACT>
static hipError_t launch_w4_s(const W4Args& a, hipStream_t stream) {
  if (a.ids) return launch_w4_t<S, 1, ACT ? 2 : 1, ACT, 4>(a, a.weights ? a.T : (int64_t)a.T * a.k, stream);
  const int nb = w4_blocks(a.T, S);
  const int64_t blocks = ((int64_t)a.T + 16 / S * nb - 1) / (16 / S * nb);
  if (nb == 1) return launch_w4_t<S, 1, ACT ? 2 : 1, ACT, 4>(a, blocks, stream);
  if (nb == 2) return launch_w4_t<S, 2, 2, ACT, 2>(a, blocks, stream);
  return launch_w4_t<S, 4, 2, ACT, 2>(a, blocks, stream);
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
  switch (w4_groups_per_chunk(G)) {
    case 4: return act ? launch_w4_s<4, true>(a, stream) : launch_w4_s<4, false>(a, stream);
    case 2: return act ? launch_w4_s<2, true>(a, stream) : launch_w4_s<2, false>(a, stream);
    default: return act ? launch_w4_s<1, true>(a, stream) : launch_w4_s<1, false>(a, stream);
  }
}

}  // namespace moe
