// moe_gmm_dgrad: gradient of the grouped matmul's input through the packed
// 4-bit weights,
//     dx[r, k] = sum_n dy[r, n] W_e[n, k]     for every row r of band e,
// on bf16 MFMA with f32 accumulation, from the same pack that moe_gmm reads.
//
// The transposed operand.  The sum runs over n, so a lane of the MFMA needs
// several n of one k; the pack holds, per lane, 32 k of one n (a 16-byte run:
// one scale block).  The runs of a chunk (16 n x 128 k) go to LDS as they lie
// in memory, by direct-to-LDS loads: [k block 0..3][n 0..15][16 bytes].  One
// ds_read_b64_tr_b8 of 16 lanes reads eight runs (eight n of one k block, 128
// contiguous bytes) as an 8 x 16 byte matrix and returns its transpose: lane
// c gets byte c of each run, the codes of k = 2c and 2c + 1 for eight n.  So
// the transposition moves 4-bit codes, a quarter of the decoded bytes, and
// costs one LDS read of 8 bytes per lane per 32 columns.  Each byte is then
// decoded with its own block scale (two bf16, exact: one scaled convert), and
// a byte permute per pair of n sorts the words into two MFMA operands, the
// even k and the odd k.
//
// The scales of a lane's eight n are the same for the 16 lanes of a group, so
// they are laid out in LDS as bf16 bit patterns (E8M0 and E4M3 values are
// exact in bf16), eight consecutive n per 16-byte read.
//
// MFMA mapping (v_mfma_f32_16x16x32_bf16; lane l supplies one row of each
// operand for eight slots of the sum, picked by g = l >> 4): the weights are
// the first operand (row = byte column c), dy the second (row = band row), so
// lane l of the result holds band row l & 15 and c = 4g .. 4g + 3: together
// with the even/odd pair, eight consecutive columns, stored as whole 16-byte
// words.
#include "common.h"
#include "launch.h"
#include "wave.h"

namespace moe {

constexpr int DG_BM = 128;                     // band rows per workgroup
constexpr int DG_MS = DG_BM / 16;              // 16-row subtiles
constexpr int DG_BK = 256;                     // output columns per workgroup: two chunks of the pack
constexpr int DG_BN = 64;                      // n per stage
constexpr int DG_WAVES = 4;                    // 64 output columns each
constexpr int DG_A_BYTES = DG_BM * DG_BN * 2;  // dy rows of 128 bytes
constexpr int DG_C_BYTES = DG_BN * DG_BK / 2;  // eight chunks of 1 KiB
constexpr int DG_NV_HALVES = 2;                // NVFP4: two scales per 32-block

typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_void_t;
typedef __attribute__((address_space(3))) i32x2_t* lds_i32x2_t;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// Rows [m0, m0 + rows) of expert e's band, or rows = 0 past the last tile.
struct BandTile {
  int e, m0, rows;
};

// Tile t of the list "for each expert, its band cut into ceil(rows / BM) even
// tiles", found
// by the whole wave from the band offsets: lane l covers experts
// [l per, l per + per), whose offsets it loads in one batch; a wave prefix sum
// of the lanes' tile counts picks the lane, which then finds its expert.
// (E <= 1024, so per <= 16.)
// The workgroup's tile and its column group nb of NB.  Workgroup ids are dealt
// round-robin to the 8 XCDs; they are remapped so that each XCD takes a
// contiguous run of the (tile, column group) list: the column groups of a
// tile then read its dy rows from one L2.
template <int BM>
__device__ __forceinline__ BandTile find_tile(const int32_t* __restrict__ off, int E, int NB, int& nb) {
  constexpr int PER = 16;
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) >> 6;
  const int e0 = lane * per;
  int o[PER + 1];
#pragma unroll
  for (int i = 0; i <= PER; ++i) o[i] = (i <= per && e0 + i <= E) ? off[e0 + i] : 0;
  int mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i < per && e0 + i < E) mine += (o[i + 1] - o[i] + BM - 1) / BM;
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  const int items = __builtin_amdgcn_readlane(incl, 63) * NB;
  const int bx = blockIdx.x, x = bx & 7;
  const int item = x * (items >> 3) + min(x, items & 7) + (bx >> 3);
  const int t = bx < items ? item / NB : -1;
  nb = item - t * NB;
  int left = t - (incl - mine);   // tile t's place among this lane's tiles
  const uint64_t hit = __ballot(t >= 0 && left >= 0 && left < mine);
  BandTile b = {0, 0, 0};
  if (hit == 0) return b;
  const int src = __ffsll((unsigned long long)hit) - 1;
  bool found = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (i < per && e0 + i < E && !found) {
      const int c = o[i + 1] - o[i];
      const int n = (c + BM - 1) / BM;
      if (left < n) {
        // an even share of the band, in whole 16-row subtiles
        const int share = ((c + n - 1) / n + 15) & ~15;
        b.e = e0 + i;
        b.m0 = o[i] + left * share;
        b.rows = min(share, c - left * share);
        found = true;
      }
      left -= n;
    }
  }
  b.e = __builtin_amdgcn_readlane(b.e, src);
  b.m0 = __builtin_amdgcn_readlane(b.m0, src);
  b.rows = __builtin_amdgcn_readlane(b.rows, src);
  return b;
}

// bf16 bit patterns of one lane's block scales, from its packed scale word.
__device__ __forceinline__ uint16_t e8m0_bf16(uint32_t b) { return (uint16_t)(b << 7); }
template <int SEL>
__device__ __forceinline__ uint16_t e4m3_bf16(uint32_t w) {
  return (uint16_t)(__float_as_uint(e4m3_to_f32<SEL>(w)) >> 16);
}

// Eight n of two k columns: byte j of q (codes of k even, k odd at n = j),
// scaled by the bf16 pattern j of s, sorted into the even-k and odd-k MFMA
// operands.  ANY: scales that are not powers of two take the exact product
// in f32 (at most six significant bits, so its upper half is the bf16 value).
template <bool ANY>
__device__ __forceinline__ void decode_pair(i32x2_t q, u32x4_t s, u32x4_t& even, u32x4_t& odd) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w = (uint32_t)q[h];
#define MOE_TWO(b0, b1, m)                                                                          \
  {                                                                                                 \
    const uint32_t sw = s[2 * h + m];                                                               \
    const float s0 = __uint_as_float(sw << 16), s1 = __uint_as_float(sw & 0xFFFF0000u);             \
    if constexpr (ANY) {                                                                            \
      const f32x2_t v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, b0);                     \
      const f32x2_t v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, b1);                     \
      even[2 * h + m] = __builtin_amdgcn_perm(__float_as_uint(v1[0] * s1), __float_as_uint(v0[0] * s0), 0x07060302u); \
      odd[2 * h + m] = __builtin_amdgcn_perm(__float_as_uint(v1[1] * s1), __float_as_uint(v0[1] * s0), 0x07060302u);  \
    } else {                                                                                        \
      const uint32_t p0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s0, b0)); \
      const uint32_t p1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s1, b1)); \
      even[2 * h + m] = __builtin_amdgcn_perm(p1, p0, 0x05040100u);                                 \
      odd[2 * h + m] = __builtin_amdgcn_perm(p1, p0, 0x07060302u);                                  \
    }                                                                                               \
  }
    MOE_TWO(0, 1, 0) MOE_TWO(2, 3, 1)
#undef MOE_TWO
  }
}

__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return (uint32_t)f32_to_bf16_rne(a) | ((uint32_t)f32_to_bf16_rne(b) << 16);
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ void load8(const void* p, bool bf16, int64_t i, float (&v)[8]) {
  if (bf16) {
    const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[2 * c] = bf16_lo(w[c]);
      v[2 * c + 1] = bf16_hi(w[c]);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// Gradients of h = silu(g) u for eight columns: dg = dh u s (1 + g (1 - s)),
// du = dh g s with s = 1 / (1 + e^-g).
__device__ __forceinline__ void silu_mul_grads(const float (&dh)[8], const float (&g)[8], const float (&u)[8],
                                               float (&dg)[8], float (&du)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = 1.0f / (1.0f + __expf(-g[i]));
    dg[i] = dh[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
    du[i] = dh[i] * g[i] * s;
  }
}

struct DgradArgs {
  const uint8_t* packed;
  Layout L;
  const uint16_t* dy;
  const int32_t* off;
  int E, NB;            // experts, 256-column groups
  const void* pre;      // [M, 2K] gate and up sums, or NULL (act 0)
  int pre_bf16;
  void* dx;
};

// Ends a step: this wave's LDS operations are done, then the workgroup
// barrier.  Loads into registers stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((63 & 15) | ((63 >> 4) << 14) | (7 << 4));   // vmcnt 63, expcnt 7, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int FMT, bool OBF16, int ACT>
__global__ __launch_bounds__(DG_WAVES * 64, 2) void dgrad_kernel(DgradArgs p) {
  constexpr int S_BYTES = (FMT == 1 ? DG_NV_HALVES : 1) * DG_BN * (DG_BK / 32) * 2;
  constexpr int STAGE = DG_A_BYTES + DG_C_BYTES + S_BYTES;
  __shared__ __attribute__((aligned(1024))) uint8_t s_stage[2 * STAGE];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, g = lane >> 4;
  int nb;
  const BandTile tile = find_tile<DG_BM>(p.off, p.E, p.NB, nb);
  if (tile.rows == 0) return;
  const Layout& L = p.L;
  const int N = (int)L.N, K = (int)L.K, KC = (int)L.KC;
  const int kc0 = nb * 2;                      // first chunk column of the workgroup
  const int kc2 = wave >> 1;                   // this wave's chunk column
  const int kb0 = (wave & 1) * 2;              // and first k block in it

  // dy rows of the tile: rows past the band do not exist in the range, so
  // they read zeros
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(p.dy + (int64_t)tile.m0 * N, (uint32_t)tile.rows * N * 2);
  const int64_t et = (int64_t)tile.e * L.NT;
  const __amdgpu_buffer_rsrc_t cr = make_rsrc(p.packed + ((et * KC) << 10), (uint32_t)((int64_t)N * K / 2));
  const __amdgpu_buffer_rsrc_t sr =
      make_rsrc(p.packed + L.scales_off + et * L.groups * 256, (uint32_t)(L.NT * L.groups * 256));
  const int rec = FMT == 0 ? kc0 >> 2 : kc0 >> 1;
  const int groups = (int)L.groups;

  // source offsets of this lane's staging loads: 1 KiB (8 rows of 128 bytes)
  // each, lane l landing in row l / 8 at segment l & 7, which holds the row's
  // segment (l & 7) ^ (row / 2 & 7): the 16 rows of a fragment read then fall
  // into 16 different 16-byte bank groups
  uint32_t avo[4], cvo[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = (wave * 4 + j) * 8 + (lane >> 3);
    avo[j] = row < tile.rows ? (uint32_t)row * N * 2 + (((lane & 7) ^ ((row >> 1) & 7)) << 4) : kLaneOob;
  }
  // chunk column (wave >> 1) of the workgroup, 16-row blocks (wave & 1)*2 + j
#pragma unroll
  for (int j = 0; j < 2; ++j)
    cvo[j] = kc0 + kc2 < KC ? (uint32_t)((((kb0 + j) * KC + kc0 + kc2) << 10) + lane * 16) : kLaneOob;

  f32x4_t acc[DG_MS][2][2];
#pragma unroll
  for (int ms = 0; ms < DG_MS; ++ms)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[ms][i >> 1][i & 1] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  bool any = false;
  if (FMT == 1) {
    const uint32_t* flags = reinterpret_cast<const uint32_t*>(p.packed + L.flags_off) + et;
    uint32_t f = 0;
    for (int i = lane; i < L.NT; i += 64) f |= flags[i];
    any = __ballot(f != 0) != 0;
  }

  const int steps = N / DG_BN;
  // A step's 4 KiB of dy, 2 KiB of codes and 256 bytes of scale words per
  // wave, loaded into registers one step ahead and written to LDS once the
  // step before is computed.  Past the last step the lane offsets lie outside
  // the buffers, so the loads fetch nothing.
  u32x4_t ra[4], rc[2];
  uint32_t rw;
  auto load = [&](int i) {
    const bool live = i < steps;
    const uint32_t q = live ? (uint32_t)i : 0u;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      rc[j] = __builtin_amdgcn_raw_buffer_load_b128(cr, live ? cvo[j] : kLaneOob, (q * (DG_BN / 16) * KC) << 10, 0);
    rw = __builtin_amdgcn_raw_buffer_load_b32(sr, live ? lane * 4 : kLaneOob,
                                              ((q * (DG_BN / 16) + wave) * groups + rec) * 256, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      ra[j] = __builtin_amdgcn_raw_buffer_load_b128(ar, live ? avo[j] : kLaneOob, q * DG_BN * 2, 0);
  };
  // Writes them to a stage: dy and codes as they are, the scale word (16-row
  // block `wave`, row c16, k block g of both chunk columns) as bf16 patterns,
  // [block][half][n].
  auto put = [&](uint8_t* st) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<u32x4_t*>(st + (wave * 4 + j) * 1024 + lane * 16) = ra[j];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<u32x4_t*>(st + DG_A_BYTES + (wave * 2 + j) * 1024 + lane * 16) = rc[j];
    uint16_t* s = reinterpret_cast<uint16_t*>(st + DG_A_BYTES + DG_C_BYTES) + wave * 16 + c16;
    if (FMT == 0) {
      s[g * 64] = e8m0_bf16((rw >> (8 * (kc0 & 3))) & 0xFFu);
      s[(4 + g) * 64] = e8m0_bf16((rw >> (8 * (kc0 & 3) + 8)) & 0xFFu);
    } else {
      s[(g * 2) * 64] = e4m3_bf16<0>(rw);
      s[(g * 2 + 1) * 64] = e4m3_bf16<1>(rw);
      s[((4 + g) * 2) * 64] = e4m3_bf16<2>(rw);
      s[((4 + g) * 2 + 1) * 64] = e4m3_bf16<3>(rw);
    }
  };
  auto compute = [&](auto nsub, const uint8_t* a) {
    constexpr int NSUB = decltype(nsub)::value;
    const uint8_t* c = a + DG_A_BYTES;
    const uint8_t* sp = c + DG_C_BYTES;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4_t w[2][2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int kb = kb0 + b;
        const i32x2_t q = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (lds_i32x2_t)(c + (kc2 * 4 + 2 * s + (g >> 1)) * 1024 + kb * 256 + (g & 1) * 128 + c16 * 8));
        const int blk = FMT == 0 ? kc2 * 4 + kb : (kc2 * 4 + kb) * 2 + (c16 >> 3);
        const u32x4_t sc = *reinterpret_cast<const u32x4_t*>(sp + (blk * 64 + s * 32 + g * 8) * 2);
        if (FMT == 1 && any) decode_pair<true>(q, sc, w[b][0], w[b][1]);
        else decode_pair<false>(q, sc, w[b][0], w[b][1]);
      }
#pragma unroll
      for (int ms = 0; ms < NSUB; ++ms) {
        const int row = ms * 16 + c16;
        const u32x4_t x =
            *reinterpret_cast<const u32x4_t*>(a + row * 128 + (((s * 4 + g) ^ ((row >> 1) & 7)) << 4));
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          acc[ms][b][0] = mfma16(w[b][0], x, acc[ms][b][0]);
          acc[ms][b][1] = mfma16(w[b][1], x, acc[ms][b][1]);
        }
      }
    }
  };

  // step i + 1 loads while step i computes; the walk of a tile with fewer
  // rows leaves out the subtiles it does not have
  load(0);
  put(s_stage);
  lds_barrier();
  auto walk = [&](auto nsub) {
    for (int i = 0; i < steps; ++i) {
      load(i + 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(nsub, s_stage + (i & 1) * STAGE);
      put(s_stage + (~i & 1) * STAGE);
      lds_barrier();
    }
  };
  switch ((tile.rows + 15) >> 4) {
    case 1: walk(std::integral_constant<int, 1>{}); break;
    case 2: walk(std::integral_constant<int, 2>{}); break;
    case 3: walk(std::integral_constant<int, 3>{}); break;
    case 4: walk(std::integral_constant<int, 4>{}); break;
    case 5: walk(std::integral_constant<int, 5>{}); break;
    case 6: walk(std::integral_constant<int, 6>{}); break;
    case 7: walk(std::integral_constant<int, 7>{}); break;
    default: walk(std::integral_constant<int, 8>{}); break;
  }

  if (kc0 + kc2 >= KC) return;
  const float post = FMT == 1 ? reinterpret_cast<const float*>(p.packed + L.tscale_off)[tile.e] : 1.0f;
#pragma unroll
  for (int ms = 0; ms < DG_MS; ++ms) {
    const int rl = ms * 16 + c16;
    if (rl >= tile.rows) continue;
    const int64_t row = tile.m0 + rl;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int col = (kc0 + kc2) * 128 + (kb0 + b) * 32 + g * 8;
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = acc[ms][b][0][i] * post;
        v[2 * i + 1] = acc[ms][b][1][i] * post;
      }
      if (ACT == 1) {
        float gate[8], up[8], dg[8], du[8];
        load8(p.pre, p.pre_bf16, row * 2 * K + col, gate);
        load8(p.pre, p.pre_bf16, row * 2 * K + K + col, up);
        silu_mul_grads(v, gate, up, dg, du);
        store8<OBF16>(p.dx, row * 2 * K + col, dg);
        store8<OBF16>(p.dx, row * 2 * K + K + col, du);
      } else {
        store8<OBF16>(p.dx, row * K + col, v);
      }
    }
  }
}

// Workgroups: an upper bound on the row tiles (a band of c rows has at most
// c / BM + 1) times the column groups.
int64_t dgrad_workgroups(int32_t E, int32_t K, int32_t M) {
  const int64_t tiles = (int64_t)M / DG_BM + (E < M ? E : M);
  return tiles * ((K + DG_BK - 1) / DG_BK);
}

template <int FMT, bool OBF16, int ACT>
static void launch_dgrad_t(const DgradArgs& a, int64_t groups, hipStream_t stream) {
  hipLaunchKernelGGL((dgrad_kernel<FMT, OBF16, ACT>), dim3((unsigned)groups), dim3(DG_WAVES * 64), 0, stream, a);
}

hipError_t launch_dgrad(const uint8_t* packed, int fmt, int32_t E, int32_t N, int32_t K, const uint16_t* dy,
                        const int32_t* group_offsets, int32_t M, const void* preact, int preact_bf16, void* dx,
                        int dx_bf16, int act, hipStream_t stream) {
  DgradArgs a;
  a.packed = packed;
  a.L = make_layout(fmt, E, N, K);
  a.dy = dy;
  a.off = group_offsets;
  a.E = E;
  a.NB = (K + DG_BK - 1) / DG_BK;
  a.pre = preact;
  a.pre_bf16 = preact_bf16;
  a.dx = dx;
  const int64_t groups = dgrad_workgroups(E, K, M);
  if (fmt == 0) {
    if (dx_bf16) act ? launch_dgrad_t<0, true, 1>(a, groups, stream) : launch_dgrad_t<0, true, 0>(a, groups, stream);
    else act ? launch_dgrad_t<0, false, 1>(a, groups, stream) : launch_dgrad_t<0, false, 0>(a, groups, stream);
  } else {
    if (dx_bf16) act ? launch_dgrad_t<1, true, 1>(a, groups, stream) : launch_dgrad_t<1, true, 0>(a, groups, stream);
    else act ? launch_dgrad_t<1, false, 1>(a, groups, stream) : launch_dgrad_t<1, false, 0>(a, groups, stream);
  }
  return hipGetLastError();
}

}  // namespace moe
