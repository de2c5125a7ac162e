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
// The scales of a lane's eight n are the same for the 16 lanes of a group (of
// its halves, NVFP4); they are converted once per workgroup and laid out in
// LDS as f32, eight consecutive n to two 16-byte reads.
//
// MFMA mapping (v_mfma_f32_16x16x32_bf16; lane l supplies one row of each
// operand for eight slots of the sum, picked by g = l >> 4): the weights are
// the first operand (row = byte column c), dy the second (row = band row), so
// lane l of the result holds band row l & 15 and c = 4g .. 4g + 3: together
// with the even/odd pair, eight consecutive columns, stored as whole 16-byte
// words.
//
// What bounds it, measured (one MI355X, 256 experts top-6):
//   w13 (4,096 x 4,096), 4,096 tokens: 772-797 us, 1.03-1.07 PFLOP/s of useful
//     products (a bf16 library product of 8,192^3 reaches 1.39 on this card,
//     the forward tiled kernel on the same bands, in turn, 731 us to 773).  The
//     matrix pipes are busy 61 % of the time at 1.9 GHz, LDS 30 %, VALU 44 %;
//     time goes with the power that the code stream, the LDS reads and the
//     decode draw: of 815 us, before the last steps, the loop without its loads
//     ran in 589, without the decode in 712.
//   the same at 64 tokens: 288-299 us, 6.0-6.2 TB/s of codes: HBM (6.6 TB/s reads).
//   w2 (4,096 x 2,048) NVFP4 with general scales, 256 tokens Zipf: 209-214 us,
//     4.5-4.7 TB/s: the general decode (twice the instructions) keeps the VALU busy
//     74 % and the matrix pipes 16 %.
//   w13 at 1 token (6 experts): 23.4 us on 192 CUs, one workgroup each, of which
//     the loads take 7 (16.5 without them) and the decode 1 (22.8; 14.8 without
//     both): a stage ends when the loads that it issued itself have landed, 16
//     times one after the other, and nothing else on the CU covers that.  32
//     experts of 1,024 x 1,024, 256 tokens top-4: 17.3 us, 13.0 without the
//     loads, 17.0 without the decode.
// Steps that brought it there (w13, 4,096 tokens): one stage, loaded and then
// computed, 988 us; walks per number of 16-row subtiles, staged one ahead, 915;
// column groups of a tile on one XCD 881; decode among the matrix instructions
// 834; direct-to-LDS loads 815; tiles dealt to the XCDs, one convert per bf16
// pair 788; wave priorities 801 -> 790, on another card.  Tried and dropped:
// 512-column workgroups of eight waves (856) or of four waves with 128 columns
// each (1,249); the largest tiles first (+2 %).
#include <utility>

#include "common.h"
#include "launch.h"
#include "wave.h"

namespace moe {

constexpr int DG_BN = 64;                      // n per stage
constexpr int DG_WAVES = 4;                    // waves per group
constexpr int DG_CUS = 256;

typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) uint8_t* lds_u8_t;
typedef __attribute__((address_space(3))) i32x2_t* lds_i32x2_t;

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// Raw buffer resource over [base, base + bytes), in scalar registers: loads
// past the end read zeros.
__device__ __forceinline__ u32x4_t make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  return u32x4_t{uniform((uint32_t)a), uniform((uint32_t)(a >> 32) & 0xFFFFu), uniform(bytes), 0x00020000u};
}

// The same range, or an empty one.
__device__ __forceinline__ u32x4_t only_if(bool live, u32x4_t rsrc) {
  rsrc[2] = live ? rsrc[2] : 0u;
  return rsrc;
}

__device__ __forceinline__ uint32_t lds_addr(const uint8_t* p) { return (uint32_t)(uintptr_t)(lds_u8_t)p; }

// 16 bytes per active lane straight to LDS: lane l's at lds + 16 l.  Written
// as an instruction of its own (it has no result register) so that the
// compiler, which cannot tell the stages apart, does not make every LDS read
// wait for every such load; vm_wait does the waiting.  NT: non-temporal, for
// the codes, which are read once.
//
// A vector memory instruction may read a scalar register only 5 wait states
// after a vector instruction wrote it, which the hardware does not see to and
// the compiler does not either around an asm statement.  The v_readfirstlane
// of uniform() are such writes and can come directly before, so the statement
// holds the whole distance itself (s_nop 4 is 5 wait states; it also covers
// the 1 after the write of M0, which the compiler places).
template <bool NT>
__device__ __forceinline__ void load_lds16(uint32_t lds, u32x4_t rsrc, uint32_t lane_off, uint32_t off) {
  lds = uniform(lds);
  off = uniform(off);
  rsrc = u32x4_t{uniform(rsrc[0]), uniform(rsrc[1]), uniform(rsrc[2]), 0x00020000u};
  if (NT)
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                 :: "{m0}"(lds), "v"(lane_off), "s"(rsrc), "s"(off) : "memory");
  else
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "{m0}"(lds), "v"(lane_off), "s"(rsrc), "s"(off) : "memory");
}

// All vector loads of this wave have landed.
__device__ __forceinline__ void vm_wait() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));   // vmcnt 0, expcnt 7, lgkmcnt 15
  asm volatile("" ::: "memory");
}

// Rows [m0, m0 + rows) of expert e's band, or rows = 0 past the last tile.
struct BandTile {
  int e, m0, rows;
};

// The workgroup's tile and its column group nb of NB, found by the whole wave
// from the band offsets.  A band of c rows is cut into ceil(c / BM) even tiles
// (of whole 16-row subtiles, the last one of the rows left).  Lane l covers
// experts [l per, l per + per) (E <= 1024, so per <= 16), whose offsets it
// loads in one batch; a wave prefix sum of the lanes' tile counts picks the
// lane, which then finds its expert.  (Offsets are held to [0, M] and bands to
// 0 rows, so that no offsets lead outside dy and dx.)
//
// Workgroup ids are dealt round-robin to the 8 XCDs.  Tiles are dealt to the
// XCDs in turn, each with all its column groups in a row, so that these read
// its dy rows from one L2; the groups of the last (tiles mod 8) tiles are
// spread over all XCDs.  (Contiguous runs of tiles per XCD, which give one XCD
// a whole tile more, cost 3 % on w2 at 4,096 tokens.)
template <int BM>
__device__ __forceinline__ BandTile find_tile(const int32_t* __restrict__ off, int E, int M, int NB, int& nb) {
  constexpr int PER = 16;
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) >> 6;
  const int e0 = lane * per;
  int o[PER + 1];
#pragma unroll
  for (int i = 0; i <= PER; ++i) o[i] = i <= per ? min(max(off[min(e0 + i, E)], 0), M) : 0;
  int mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i < per) mine += (max(o[i + 1] - o[i], 0) + BM - 1) / BM;
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d, 64);
    if (lane >= d) incl += v;
  }
  const int tiles = __builtin_amdgcn_readlane(incl, 63);
  const int x = blockIdx.x & 7, k = blockIdx.x >> 3;
  const int whole = (tiles >> 3) * NB;
  int t;
  if (k < whole) {
    t = (k / NB) * 8 + x;
    nb = k % NB;
  } else {
    const int r = (k - whole) * 8 + x;
    t = (tiles & ~7) + r / NB;
    nb = r % NB;
  }
  BandTile b = {0, 0, 0};
  if (t >= tiles) return b;
  int left = t - (incl - mine);   // tile t's place among this lane's tiles
  const int src = __ffsll((unsigned long long)__ballot(left >= 0 && left < mine)) - 1;
  bool found = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (i < per && !found) {
      const int c = max(o[i + 1] - o[i], 0);
      const int n = (c + BM - 1) / BM;
      if (left < n) {
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

// Codes and scales of eight n of two k columns, as they come from LDS, and the
// two MFMA operands they decode to.
struct RawWeights {
  i32x2_t q;       // byte j: the codes of k even, k odd at n = j
  f32x4_t s[2];    // scale of n = j at s[j / 4][j % 4]
};
struct Weights {
  u32x4_t even, odd;
};

// Word M of both operands (n = 2M, 2M + 1).  ANY: scales that are not powers of
// two take the exact product in f32 (at most six significant bits, so its
// upper half is the bf16 value).
template <bool ANY, int M>
__device__ __forceinline__ void decode_word(const RawWeights& r, Weights& w) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  const uint32_t q = (uint32_t)r.q[M / 2];
  const float sa = r.s[M / 2][(M & 1) * 2], sb = r.s[M / 2][(M & 1) * 2 + 1];
  constexpr int B = (M & 1) * 2;
  if constexpr (ANY) {
    const f32x2_t v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, B);
    const f32x2_t v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, B + 1);
    w.even[M] = __builtin_amdgcn_perm(__float_as_uint(v1[0] * sb), __float_as_uint(v0[0] * sa), 0x07060302u);
    w.odd[M] = __builtin_amdgcn_perm(__float_as_uint(v1[1] * sb), __float_as_uint(v0[1] * sa), 0x07060302u);
  } else {
    const uint32_t p0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sa, B));
    const uint32_t p1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sb, B + 1));
    w.even[M] = __builtin_amdgcn_perm(p1, p0, 0x05040100u);
    w.odd[M] = __builtin_amdgcn_perm(p1, p0, 0x07060302u);
  }
}

// Words [LO, HI) of the 4 words of each of a wave's KB k blocks.
template <bool ANY, int LO, int HI, int KB>
__device__ __forceinline__ void decode_words(const RawWeights (&r)[KB], Weights (&w)[KB]) {
  if constexpr (LO < HI) {
    decode_word<ANY, LO % 4>(r[LO / 4], w[LO / 4]);
    decode_words<ANY, LO + 1, HI, KB>(r, w);
  }
}

__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

__device__ __forceinline__ void store8(void* p, bool bf16, int64_t i, const float (&v)[8]) {
  if (bf16) {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Eight values as they lie in memory (PRE 1: bf16, 2: f32), and as f32.
template <int PRE>
struct Raw8 {
  u32x4_t w[PRE];
};

template <int PRE>
__device__ __forceinline__ Raw8<PRE> load_raw8(const void* p, int64_t i) {
  Raw8<PRE> r;
  const u32x4_t* q = reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint8_t*>(p) + i * (2 * PRE));
#pragma unroll
  for (int c = 0; c < PRE; ++c) r.w[c] = q[c];
  return r;
}

template <int PRE>
__device__ __forceinline__ void unpack8(const Raw8<PRE>& r, float (&v)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    v[c] = PRE == 2 ? __uint_as_float(r.w[(c >> 2) * (PRE - 1)][c & 3]) : c & 1 ? bf16_hi(r.w[0][c >> 1]) : bf16_lo(r.w[0][c >> 1]);
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

// N times one matrix instruction and VALU vector instructions behind it.
template <int N, int VALU>
__device__ __forceinline__ void interleave() {
  if constexpr (N > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (VALU > 0) __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    interleave<N - 1, VALU>();
  }
}

// One 32-n step: the NSUB row subtiles against the operands w, with the next
// step's operands decoded from r into v on the way.  Each group is a subtile's
// matrix instructions, the LDS read of the subtile after next, and a share of
// the decode, which issues in the shadow of the matrix instructions.  The last
// group has no decode where there are others: it issues the LDS reads that the
// next step starts with (next).
template <bool ANY, int NSUB, int MAX, int KB, int... MS, typename ROWS, typename NEXT>
__device__ __forceinline__ void dgrad_step(std::integer_sequence<int, MS...>, u32x4_t (&x)[2], ROWS rows, NEXT next,
                                           const Weights (&w)[KB], const RawWeights (&r)[KB], Weights (&v)[KB],
                                           f32x4_t (&acc)[MAX][KB][2]) {
  constexpr int DEC = NSUB > 1 ? NSUB - 1 : 1;   // groups that decode
  auto group = [&](auto mc) __attribute__((always_inline)) {
    constexpr int ms = decltype(mc)::value;
    const u32x4_t xa = x[ms & 1];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      acc[ms][b][0] = mfma16(w[b].even, xa, acc[ms][b][0]);
      acc[ms][b][1] = mfma16(w[b].odd, xa, acc[ms][b][1]);
    }
    if constexpr (ms + 2 < NSUB) x[ms & 1] = rows(ms + 2);
    if constexpr (ms < DEC) {
      constexpr int LO = 4 * KB * ms / DEC, HI = 4 * KB * (ms + 1) / DEC;
      decode_words<ANY, LO, HI, KB>(r, v);
      interleave<2 * KB - 1, (ANY ? 8 : 4) * (HI - LO) / (2 * KB)>();
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (ms == NSUB - 1) next();
  };
  (group(std::integral_constant<int, MS>{}), ...);
}

// f(0), f(1), ... with constants.
template <int... I, typename F>
__device__ __forceinline__ void for_each(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>{}), ...);
}

struct DgradArgs {
  const uint8_t* packed;
  Layout L;
  const uint16_t* dy;
  const int32_t* off;
  int E, M, NB;         // experts, rows, column groups
  const void* pre;      // [M, 2K] gate and up sums, or NULL (no activation)
  int pre_bf16;
  void* dx;
  int dx_bf16;
};

// Ends a stage: this wave's LDS operations are done, then the workgroup
// barrier.  Vector loads are vm_wait's.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((63 & 15) | ((63 >> 4) << 14) | (7 << 4));   // vmcnt 63, expcnt 7, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Four waves take KB k blocks (32 output columns) each.  NS groups of four
// waves share a workgroup; each walks its share of n (in whole stages, the
// last share padded with empty ones) through LDS of its own, and the first
// adds up the partial sums in order.
//
// Stages.  All operands go straight to LDS.  While stage i is multiplied, dy
// of stage i + 1, codes of stage i + 2 and scale words of stage i + 3 are
// loaded; the operands of stage i + 1 are decoded from its codes, which have
// landed, and the scale words of stage i + 2 are spread out as f32.  A stage
// ends when all loads of the wave have landed, then the barrier.  Counted
// waits that leave the newest loads on their way (with a third stage of codes)
// gained 1 % at most on large grids and 1.6 us on small ones; direct-to-LDS
// loads of 4 bytes have been seen on MI355X to land later than such a count
// said, so nothing here hangs on their order (370,000 runs with counted waits
// on loads of 16 bytes gave the bits of the full wait).
template <int FMT, int MS, int KB, int OCC, int NS>
__global__ __launch_bounds__(DG_WAVES * 64 * NS, OCC) void dgrad_kernel(DgradArgs p) {
  constexpr int BM = MS * 16;                            // band rows per workgroup
  constexpr int KCW = KB;                                // chunk columns (128 k) per workgroup
  constexpr int A_BYTES = BM * DG_BN * 2;                // dy rows of 128 bytes
  constexpr int A_LOADS = A_BYTES / 1024 / DG_WAVES;     // 1 KiB loads per wave
  constexpr int C_BYTES = KCW * DG_BN / 16 * 1024;
  constexpr int H = FMT == 1 ? 2 : 1;                    // scales per 32-block
  constexpr int R_BYTES = DG_BN / 16 * 256;              // scale words: a record per 16 n, one a wave
  constexpr int S_BYTES = H * DG_BN * KCW * 4 * 4;       // the same as f32
  constexpr int GROUP_BYTES = 2 * A_BYTES + 2 * C_BYTES + 3 * R_BYTES + 2 * S_BYTES;
  constexpr int PART_BYTES = DG_WAVES * MS * KB * 2 * 64 * 16;   // a group's accumulators
  static_assert(DG_BN / 16 == DG_WAVES && A_LOADS >= 1, "whole loads per wave");
  static_assert((NS - 1) * PART_BYTES <= NS * GROUP_BYTES, "the partial sums fit the stages");
  __shared__ __attribute__((aligned(1024))) uint8_t s_all[NS * GROUP_BYTES];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % DG_WAVES);
  const int part = NS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / (DG_WAVES * 64)) : 0;
  uint8_t* s_dy = s_all + part * GROUP_BYTES;
  uint8_t* s_codes = s_dy + 2 * A_BYTES;
  uint8_t* s_words = s_codes + 2 * C_BYTES;
  uint8_t* s_scale = s_words + 3 * R_BYTES;
  const int c16 = lane & 15, g = lane >> 4;
  int nb;
  const BandTile tile = find_tile<BM>(p.off, p.E, p.M, p.NB, nb);
  if (tile.rows == 0) return;
  const Layout& L = p.L;
  const int N = (int)L.N, K = (int)L.K, KC = (int)L.KC;
  const int kc0 = nb * KCW;                    // first chunk column of the workgroup
  const int kcw = wave * KB / 4;               // this wave's chunk column
  const int kb0 = wave * KB % 4;               // and first k block in it

  // dy rows of the tile: rows past the band do not exist in the range, so
  // they read zeros
  const u32x4_t ar = make_rsrc(p.dy + (int64_t)tile.m0 * N, (uint32_t)tile.rows * N * 2);
  const int64_t et = (int64_t)tile.e * L.NT;
  const u32x4_t cr = make_rsrc(p.packed + ((et * KC) << 10), (uint32_t)((int64_t)N * K / 2));
  const int groups = (int)L.groups;
  const u32x4_t sr = make_rsrc(p.packed + L.scales_off + et * groups * 256, (uint32_t)(L.NT * groups * 256));

  // source offsets of this lane's staging loads: 1 KiB (8 rows of 128 bytes)
  // each, lane l landing in row l / 8 at segment l & 7, which holds the row's
  // segment (l & 7) ^ (row / 2 & 7): the 16 rows of a fragment read then fall
  // into 16 different 16-byte bank groups
  uint32_t avo[A_LOADS];
#pragma unroll
  for (int j = 0; j < A_LOADS; ++j) {
    const int row = (wave * A_LOADS + j) * 8 + (lane >> 3);
    avo[j] = row < tile.rows ? (uint32_t)row * N * 2 + (((lane & 7) ^ ((row >> 1) & 7)) << 4) : kLaneOob;
  }
  // the wave's KB code chunks: its chunk column, 16-n blocks kb0, kb0 + 1, ...
  const uint32_t cvo = kc0 + kcw < KC ? (uint32_t)(((kb0 * KC + kc0 + kcw) << 10) + lane * 16) : kLaneOob;
  // and its scale words: the records of 16-n block `wave`
  const uint32_t rvo = (uint32_t)((wave * groups + (FMT == 0 ? kc0 >> 2 : kc0 >> 1)) * 256 + lane * 16);

  f32x4_t acc[MS][KB][2];
#pragma unroll
  for (int ms = 0; ms < MS; ++ms)
#pragma unroll
    for (int i = 0; i < 2 * KB; ++i) acc[ms][i >> 1][i & 1] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // stages [first, end) of this group; every group runs `steps`
  const int steps = (N / DG_BN + NS - 1) / NS;
  const int first = part * steps, end = min(N / DG_BN, first + steps);
  // Past the last stage the buffers are empty, so the loads fetch nothing and
  // write zeros.
  const uint32_t l_dy = lds_addr(s_dy) + wave * A_LOADS * 1024, l_codes = lds_addr(s_codes) + wave * KB * 1024,
                 l_words = lds_addr(s_words) + wave * 256;
  auto load_dy = [&](int i) {
    const bool live = first + i < end;
    const uint32_t q = live ? (uint32_t)(first + i) : 0u;
#pragma unroll
    for (int j = 0; j < A_LOADS; ++j)
      load_lds16<false>(l_dy + (i & 1) * A_BYTES + j * 1024, only_if(live, ar), avo[j], q * DG_BN * 2);
  };
  auto load_words = [&](int i, uint32_t slot) {
    const bool live = first + i < end;
    const uint32_t q = live ? (uint32_t)(first + i) * (DG_BN / 16) : 0u;
    if (lane < 16)
      load_lds16<false>(l_words + slot * R_BYTES, only_if(live, sr), rvo, q * groups * 256);
  };
  auto load_codes = [&](int i) {
    const bool live = first + i < end;
    const uint32_t q = live ? (uint32_t)(first + i) * (DG_BN / 16) : 0u;
#pragma unroll
    for (int j = 0; j < KB; ++j)
      load_lds16<true>(l_codes + (i & 1) * C_BYTES + j * 1024, only_if(live, cr), cvo, ((q + j) * KC) << 10);
  };
  // This wave's scale words of stage i (n = c16 of 16-n block `wave`, k block
  // g of the record's chunk columns), from LDS and back to it as f32,
  // [k block][half][n]; the high halves' n (NVFP4) are turned by 32, so that
  // the lanes of the two halves read different banks (NVFP4 w2 at 128 tokens:
  // 222 -> 216 us).
  auto scale_word = [&](uint32_t slot) {
    return *reinterpret_cast<const uint32_t*>(s_words + slot * R_BYTES + wave * 256 + lane * 4);
  };
  auto spread_scales = [&](uint32_t w, int i) {
    float* s = reinterpret_cast<float*>(s_scale + (i & 1) * S_BYTES) + wave * 16 + c16;
    float* hi = s + ((wave ^ 2) - wave) * 16;
    if (FMT == 0) {
#pragma unroll
      for (int j = 0; j < KCW; ++j) s[(j * 4 + g) * 64] = e8m0_to_f32((w >> (8 * ((kc0 & 3) + j))) & 0xFFu);
    } else {
      if (KCW == 1) w >>= 16 * (kc0 & 1);
      s[(g * 2) * 64] = e4m3_to_f32<0>(w);
      hi[(g * 2 + 1) * 64] = e4m3_to_f32<1>(w);
      if (KCW == 2) {
        s[((4 + g) * 2) * 64] = e4m3_to_f32<2>(w);
        hi[((4 + g) * 2 + 1) * 64] = e4m3_to_f32<3>(w);
      }
    }
  };

  // Step s (32 n) of a stage: codes and scales of this wave's k blocks,
  // and the band rows of subtile ms.
  const uint32_t q_off = (kcw * 4 + (g >> 1)) * 1024 + kb0 * 256 + (g & 1) * 128 + c16 * 8;
  const uint32_t half = H == 2 ? c16 >> 3 : 0;
  const uint32_t s_off = (((kcw * 4 + kb0) * H + half) * 64 + g * 8) << 2;
  const uint32_t s_turn = half * 128;
  const uint32_t a_off = c16 * 128 + ((g ^ ((c16 >> 1) & 7)) << 4);
  auto raw = [&](int i, int s, RawWeights (&r)[KB]) {
    const uint8_t* st = s_codes + (i & 1) * C_BYTES;
    const uint8_t* sc = s_scale + (i & 1) * S_BYTES;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      r[b].q = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2_t)(st + q_off + s * 2048 + b * 256));
      const f32x4_t* f = reinterpret_cast<const f32x4_t*>(sc + s_off + ((s * 128) ^ s_turn) + b * 256 * H);
      r[b].s[0] = f[0];
      r[b].s[1] = f[1];
    }
  };
  auto rows = [&](const uint8_t* a, int s, int ms) {
    return *reinterpret_cast<const u32x4_t*>(a + (a_off ^ (s * 64)) + ms * 2048);
  };

  // The walk of a tile with nsub 16-row subtiles: the operands of a step are
  // decoded among the matrix instructions of the step before.  (Inlined, so
  // that the accumulators stay in registers.)
  auto walk = [&](auto any, auto nsub) __attribute__((always_inline)) {
    constexpr bool any_v = decltype(any)::value;
    constexpr int NSUB = decltype(nsub)::value;
    load_words(0, 0);
    load_words(1, 1);
    load_words(2, 2);
    load_codes(0);
    load_codes(1);
    load_dy(0);
    vm_wait();
    spread_scales(scale_word(0), 0);
    spread_scales(scale_word(1), 1);
    lds_barrier();
    RawWeights r[KB];
    Weights w[KB], v[KB];
    raw(0, 0, r);
    decode_words<any_v, 0, 4 * KB, KB>(r, w);
    raw(0, 1, r);
    lds_barrier();                             // stage 0's codes and f32 scales make room
    uint32_t slot = 0;                         // of the scale words: i mod 3
    for (int i = 0; i < steps; ++i) {
      const uint8_t* a = s_dy + (i & 1) * A_BYTES;
      u32x4_t x[2];
      auto first_rows = [&](int s) {
        x[0] = rows(a, s, 0);
        if constexpr (NSUB > 1) x[1] = rows(a, s, 1);
      };
      first_rows(0);
      __builtin_amdgcn_sched_barrier(0);
      load_dy(i + 1);
      load_codes(i + 2);
      load_words(i + 3, slot);
      // the waves at their products before those between stages (128-row tiles:
      // 801 -> 790 us; thin ones lose)
      if (MS == 8) __builtin_amdgcn_s_setprio(1);
      __builtin_amdgcn_sched_barrier(0);
      dgrad_step<any_v, NSUB, MS, KB>(std::make_integer_sequence<int, NSUB>{}, x, [&](int ms) { return rows(a, 0, ms); },
                                  [&] { first_rows(1); raw(i + 1, 0, r); }, w, r, v, acc);
      const uint32_t word = scale_word(slot == 0 ? 2 : slot - 1);
      dgrad_step<any_v, NSUB, MS, KB>(std::make_integer_sequence<int, NSUB>{}, x, [&](int ms) { return rows(a, 1, ms); },
                                  [&] { raw(i + 1, 1, r); }, v, r, w, acc);
      __builtin_amdgcn_sched_barrier(0);
      if (MS == 8) __builtin_amdgcn_s_setprio(0);
      spread_scales(word, i + 2);
      vm_wait();
      lds_barrier();
      slot = slot == 2 ? 0 : slot + 1;
    }
  };
  auto walk_any = [&](auto any) __attribute__((always_inline)) {
    const int nsub = (tile.rows + 15) >> 4;
    if constexpr (MS == 8) {
      switch (nsub) {
        case 1: walk(any, std::integral_constant<int, 1>{}); break;
        case 2: walk(any, std::integral_constant<int, 2>{}); break;
        case 3: walk(any, std::integral_constant<int, 3>{}); break;
        case 4: walk(any, std::integral_constant<int, 4>{}); break;
        case 5: walk(any, std::integral_constant<int, 5>{}); break;
        case 6: walk(any, std::integral_constant<int, 6>{}); break;
        case 7: walk(any, std::integral_constant<int, 7>{}); break;
        default: walk(any, std::integral_constant<int, 8>{}); break;
      }
    } else if constexpr (MS == 4) {
      switch (nsub) {
        case 1: walk(any, std::integral_constant<int, 1>{}); break;
        case 2: walk(any, std::integral_constant<int, 2>{}); break;
        case 3: walk(any, std::integral_constant<int, 3>{}); break;
        default: walk(any, std::integral_constant<int, 4>{}); break;
      }
    } else {
      if (nsub == 1) walk(any, std::integral_constant<int, 1>{});
      else walk(any, std::integral_constant<int, 2>{});
    }
  };
  bool any = false;
  if (FMT == 1) {
    const uint32_t* flags = reinterpret_cast<const uint32_t*>(p.packed + L.flags_off) + et;
    uint32_t f = 0;
    for (int i = lane; i < L.NT; i += 64) f |= flags[i];
    any = __ballot(f != 0) != 0;
  }
  if (FMT == 1 && any) walk_any(std::true_type{});
  else walk_any(std::false_type{});

  if constexpr (NS > 1) {
    // accumulators of groups 1 .. NS - 1, a float4 per lane and register quad
    lds_barrier();   // no load is on its way to any group's stages
    f32x4_t* sum = reinterpret_cast<f32x4_t*>(s_all) + (wave * MS * KB * 2) * 64 + lane;
    if (part > 0) {
#pragma unroll
      for (int j = 0; j < MS * KB * 2; ++j)
        sum[(part - 1) * (PART_BYTES / 16) + j * 64] = acc[j / (2 * KB)][j / 2 % KB][j & 1];
    }
    lds_barrier();
    if (part > 0) return;
#pragma unroll 1
    for (int q = 0; q < NS - 1; ++q)
#pragma unroll
      for (int j = 0; j < MS * KB * 2; ++j)
        acc[j / (2 * KB)][j / 2 % KB][j & 1] += sum[q * (PART_BYTES / 16) + j * 64];
  }

  if (kc0 + kcw >= KC) return;
  const float post = FMT == 1 ? reinterpret_cast<const float*>(p.packed + L.tscale_off)[tile.e] : 1.0f;
  // Unit u = ms * KB + b: eight columns (k block b) of this lane's row of
  // subtile ms.  Constants all the way, so that the accumulators are never
  // indexed at run time.
  const int64_t col0 = (int64_t)(kc0 + kcw) * 128 + kb0 * 32 + g * 8;
  auto sums = [&](auto uc, float (&v)[8]) __attribute__((always_inline)) {
    constexpr int u = decltype(uc)::value;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = acc[u / KB][u % KB][0][i] * post;
      v[2 * i + 1] = acc[u / KB][u % KB][1][i] * post;
    }
  };
  if (!p.pre) {
    for_each(std::make_integer_sequence<int, MS * KB>{}, [&](auto uc) __attribute__((always_inline)) {
      constexpr int u = decltype(uc)::value;
      const int rl = u / KB * 16 + c16;
      float v[8];
      sums(uc, v);
      if (rl < tile.rows) store8(p.dx, p.dx_bf16, (int64_t)(tile.m0 + rl) * K + col0 + u % KB * 32, v);
    });
    return;
  }
  // Through the activation: the gate and up values of G units are loaded while
  // the G before them are computed (rows past the tile read its last row).
  auto activation = [&](auto prec) __attribute__((always_inline)) {
    constexpr int PRE = decltype(prec)::value;
    constexpr int G = PRE == 1 && MS == 8 ? 4 : 2;
    constexpr int GROUPS = MS * KB / G;
    Raw8<PRE> gate[2][G], up[2][G];
    auto load_group = [&](auto jc) __attribute__((always_inline)) {
      constexpr int j = decltype(jc)::value;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int u = j * G + i;
        const int64_t at = (int64_t)(tile.m0 + min(u / KB * 16 + c16, tile.rows - 1)) * 2 * K + col0 + u % KB * 32;
        gate[j & 1][i] = load_raw8<PRE>(p.pre, at);
        up[j & 1][i] = load_raw8<PRE>(p.pre, at + K);
      }
    };
    load_group(std::integral_constant<int, 0>{});
    for_each(std::make_integer_sequence<int, GROUPS>{}, [&](auto jc) __attribute__((always_inline)) {
      constexpr int j = decltype(jc)::value;
      if constexpr (j + 1 < GROUPS) load_group(std::integral_constant<int, j + 1>{});
      __builtin_amdgcn_sched_barrier(0);
      for_each(std::make_integer_sequence<int, G>{}, [&](auto ic) __attribute__((always_inline)) {
        constexpr int i = decltype(ic)::value, u = j * G + i;
        const int rl = u / KB * 16 + c16;
        float v[8], gt[8], ut[8], dg[8], du[8];
        sums(std::integral_constant<int, u>{}, v);
        unpack8<PRE>(gate[j & 1][i], gt);
        unpack8<PRE>(up[j & 1][i], ut);
        silu_mul_grads(v, gt, ut, dg, du);
        if (rl < tile.rows) {
          const int64_t at = (int64_t)(tile.m0 + rl) * 2 * K + col0 + u % KB * 32;
          store8(p.dx, p.dx_bf16, at, dg);
          store8(p.dx, p.dx_bf16, at + K, du);
        }
      });
    });
  };
  if (p.pre_bf16) activation(std::integral_constant<int, 1>{});
  else activation(std::integral_constant<int, 2>{});
}

// The kernel for E experts and M rows: row subtiles of a tile, k blocks of a
// wave (128 columns of a workgroup each), workgroups (an upper bound: a band
// of c rows has at most c / BM + 1 tiles), and groups of waves per workgroup.
struct DgradPlan {
  int subtiles, blocks, parts;
  int64_t groups;
};

static DgradPlan dgrad_plan(int32_t E, int32_t K, int32_t M) {
  DgradPlan pl;
  // By the mean band: 32-row tiles up to 24 rows (w13, 4,096 x 4,096, at 24
  // rows a band: 429 us against 442 with 64-row tiles), 64-row tiles to 72
  // (at 48: 544 against 802 with 32 and 604 with 128), then 128 (at 96: 775
  // against 1,034 with 64).  Those are of uniform routing; with Zipf routing
  // the choice at 24 rows costs 4 % (w2, 4,096 x 2,048: 290 against 277).
  pl.subtiles = (int64_t)M <= 24 * (int64_t)E ? 2 : (int64_t)M < 72 * (int64_t)E ? 4 : 8;
  const int64_t tiles = (int64_t)M / (16 * pl.subtiles) + (E < M ? E : M);
  pl.blocks = 2;
  pl.parts = 1;
  pl.groups = tiles * ((K + 255) / 256);
  if (pl.subtiles == 2) {
    // A CU runs four groups of waves at a time, and a short grid is bound by
    // how fast a wave decodes its stages.  Where the groups have room, n is
    // shared by several (w13, 1 token: 50 -> 30 us with four), and where half
    // the CUs would idle, a workgroup takes 128 columns (28 -> 23 us).
    if (pl.groups <= DG_CUS) pl.parts = 4;
    else if (pl.groups <= 2 * DG_CUS) pl.parts = 2;
    if (pl.groups * 2 <= DG_CUS) {
      pl.blocks = 1;
      pl.groups = tiles * (K / 128);
    }
  }
  return pl;
}

int64_t dgrad_workgroups(int32_t E, int32_t K, int32_t M) { return dgrad_plan(E, K, M).groups; }

template <int FMT, int MS, int KB, int OCC, int NS>
static void launch_dgrad_t(DgradArgs a, int64_t groups, hipStream_t stream) {
  a.NB = (int)((a.L.K + 128 * KB - 1) / (128 * KB));
  hipLaunchKernelGGL((dgrad_kernel<FMT, MS, KB, OCC, NS>), dim3((unsigned)groups), dim3(DG_WAVES * 64 * NS), 0,
                     stream, a);
}

template <int FMT>
static void launch_dgrad_plan(const DgradArgs& a, const DgradPlan& pl, hipStream_t stream) {
  if (pl.subtiles == 8) launch_dgrad_t<FMT, 8, 2, 2, 1>(a, pl.groups, stream);
  else if (pl.subtiles == 4) launch_dgrad_t<FMT, 4, 2, 3, 1>(a, pl.groups, stream);
  else if (pl.blocks == 1) launch_dgrad_t<FMT, 2, 1, 4, 4>(a, pl.groups, stream);
  else if (pl.parts == 4) launch_dgrad_t<FMT, 2, 2, 4, 4>(a, pl.groups, stream);
  else if (pl.parts == 2) launch_dgrad_t<FMT, 2, 2, 4, 2>(a, pl.groups, stream);
  else launch_dgrad_t<FMT, 2, 2, 4, 1>(a, pl.groups, stream);
}

hipError_t launch_dgrad(const uint8_t* packed, int fmt, int32_t E, int32_t N, int32_t K, const uint16_t* dy,
                        const int32_t* group_offsets, int32_t M, const void* preact, int preact_bf16, void* dx,
                        int dx_bf16, hipStream_t stream) {
  DgradArgs a;
  a.packed = packed;
  a.L = make_layout(fmt, E, N, K);
  a.dy = dy;
  a.off = group_offsets;
  a.E = E;
  a.M = M;
  a.pre = preact;
  a.pre_bf16 = preact_bf16;
  a.dx = dx;
  a.dx_bf16 = dx_bf16;
  const DgradPlan pl = dgrad_plan(E, K, M);
  if (fmt == 0) launch_dgrad_plan<0>(a, pl, stream);
  else launch_dgrad_plan<1>(a, pl, stream);
  return hipGetLastError();
}

}  // namespace moe
