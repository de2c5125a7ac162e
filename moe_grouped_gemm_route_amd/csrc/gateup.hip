// moe_gate_up and moe_gate_up_bwd: the gated feed-forward block of the tokens'
// shared expert (or of a dense layer), bf16 weights [N, K] with the gate rows
// first and the up rows behind them:
//     [g u] = x w13^T,   h = silu(g) u,   silu(z) = z / (1 + e^-z),
// and backwards, with s = 1 / (1 + e^-g),
//     dg = dh u s (1 + g (1 - s)),   du = dh g s,   d = [dg du],
//     dx = d w13,   dw13 = d^T x.
//
// All three products run on one tile kernel, out[i, j] = sum_r A(i, r) B(j, r)
// on bf16 MFMA with f32 sums.  An operand lies in memory either with r
// contiguous (x and w13 forwards, d for dx) or with r as the row (w13 for dx;
// d and x for dw13); the second kind goes to LDS as it lies and is transposed
// by the reads (ds_read_b64_tr_b16), so nothing is transposed in memory.
#include "common.h"
#include "launch.h"
#include "lds_load.h"
#include "wave.h"

namespace moe {

constexpr int GU_BK = 64;      // r per stage
constexpr int GU_CUS = 256;

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4_t* lds_i16x4_t;

__device__ __forceinline__ f32x4_t gu_mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

// 1 / (1 + e^-z) by the reciprocal instruction (1 ulp; the division's correct
// rounding costs ten more instructions, 8 us of 4,096 x 4,096 sums' epilogue).
__device__ __forceinline__ float gu_sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }
__device__ __forceinline__ float gu_silu(float z) { return z * gu_sigmoid(z); }

__device__ __forceinline__ void gu_store8(void* p, bool bf16, int64_t i, const float (&v)[8]) {
  if (bf16) {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
    float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t gu_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

__device__ __forceinline__ void gu_store4(void* p, bool bf16, int64_t i, f32x4_t v) {
  if (bf16)
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + i) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  else
    *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(p) + i) = v;
}

// ---------------------------------------------------------------------------
// The tile kernel
// ---------------------------------------------------------------------------

struct TileArgs {
  const uint16_t* a;       // r contiguous: [I, lda]; r as the row: [R, lda]
  const uint16_t* b;       // likewise with J
  int64_t lda, ldb;
  int I, J, R;             // J: columns of out (with GATE: of h)
  int64_t part_stride;     // PARTS matrices, this far apart, add up to A (of f32 results)
  int splits, steps;       // shares of the sum over r, and stages of a share
  int tiles_i, tiles_j;
  void* out;               // [I, J]; with splits > 1 f32 [splits, I, J]
  int out_bf16;
  void* pre;               // GATE: [I, 2J] sums, or NULL
  int pre_bf16;
};

// One operand's tile of DIM rows (or columns) x 64 r in LDS, DIM * 128 bytes.
//
// r contiguous: rows of 128 bytes, 16-byte segment c of row q at place
// c ^ swizzle(q), so that the eight lanes that are served together read eight
// different segments of the 128 bytes that their rows share in the banks.
// r as the row: rows of DIM * 2 bytes, segment c of row r at c ^ swizzle(r): 32
// lanes of a transposing read take 32 bytes of eight rows, r = 0 .. 3 and 8 .. 11
// of a step, which then lie in different banks.
//
// PAIR (the B operand with r contiguous): the columns of out that two
// neighbouring 16-column subtiles cover are dealt so that a lane's results are
// eight consecutive ones: subtile s, row q of the operand is column
// (q >> 2) * 8 + s * 4 + (q & 3) of the pair's 32.
template <bool RROW, int DIM, int WAVES, bool PAIR>
struct Operand {
  static constexpr int BYTES = DIM * GU_BK * 2;
  static constexpr int LOADS = BYTES / 1024 / WAVES;        // 1 KiB loads of a wave
  static constexpr int SEGS = RROW ? DIM / 8 : GU_BK / 8;   // 16-byte segments of an LDS row
  static constexpr int ROWS = 64 / SEGS;                    // LDS rows of a load
  static_assert(LOADS >= 1 && LOADS * WAVES * 1024 == BYTES, "whole loads per wave");
  static_assert(!RROW || (DIM >= 128 && DIM <= 512), "rows of 256 bytes at least, a load per two rows at most");

  static __device__ __forceinline__ int swizzle(int row) {
    return RROW ? ((row & 3) | ((row >> 3) & 1) << 2) << 1 : PAIR ? (row & 3) | ((row >> 3) & 1) << 2 : row & 7;
  }
  // LDS row and source segment of this lane in load j of a wave
  static __device__ __forceinline__ int row(int wave, int j) {
    return (wave * LOADS + j) * ROWS + (threadIdx.x & 63) / SEGS;
  }
  static __device__ __forceinline__ int seg(int row) { return ((threadIdx.x & 63) % SEGS) ^ swizzle(row); }

  // The MFMA operand of 32 r (step ks) and 16 rows: subtile `sub` of the wave's
  // `base`; lane l holds row l & 15, r = 8 (l >> 4) .. + 7.
  static __device__ __forceinline__ u32x4_t read(const uint8_t* tile, int base, int sub, int ks) {
    const int lane = threadIdx.x & 63, q = lane & 15, g = lane >> 4;
    if constexpr (!RROW) {
      const int r = base + (PAIR ? (sub >> 1) * 32 + (q >> 2) * 8 + (sub & 1) * 4 + (q & 3) : sub * 16 + q);
      return *reinterpret_cast<const u32x4_t*>(tile + r * 128 + (((ks * 4 + g) ^ swizzle(r)) << 4));
    } else {
      // 16 lanes read four r of 16 columns, lane q four columns of row q / 4,
      // and get one column's four r
      const int seg = base / 8 + sub * 2 + ((q & 3) >> 1);
      const int half = q & 1;
      u32x4_t v;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = ks * 32 + g * 8 + h * 4 + (q >> 2);
        const uint8_t* at = tile + r * (DIM * 2) + ((seg ^ swizzle(r)) << 4) + half * 8;
        const uint2 w = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)at));
        v[2 * h] = w.x;
        v[2 * h + 1] = w.y;
      }
      return v;
    }
  }
};

// Tile t of the grid, or of a share of it: tiles are dealt to the 8 XCDs
// (workgroup ids go round them) in contiguous runs, which walk bands of four
// tile rows column by column, so that the workgroups that run together on an
// XCD share rows of both operands in its L2.
__device__ __forceinline__ void tile_of(int id, int tiles, int ti, int tj, int& i, int& j) {
  const int x = id & 7, k = id >> 3;
  const int per = tiles >> 3, rest = tiles & 7;
  const int t = x * per + min(x, rest) + k;
  const int band = t / (4 * tj), in = t - band * 4 * tj;
  const int h = min(4, ti - band * 4);
  j = in / h;
  i = band * 4 + in - j * h;
}

// WI x WJ waves of SI x SJ 16 x 16 subtiles each, KG such groups of waves that
// take every KG-th 64 r; two stages in LDS, or three (TURNS).  PARTS: A comes as
// that many bf16 matrices, each multiplied with the same B.
//
// PARTS and infinities.  The second and third part of a value are zero or of the
// other sign as often as not, so an infinite B makes the sum NaN (0 inf, inf - inf)
// where A B is an infinity.  A tile of which a result is NaN is therefore walked a
// second time, with the first part in place of all three, and the results that were
// NaN are written again: each has a term that is not finite, so the first parts'
// sum is the infinity or the NaN that the whole values' is.  Finite tiles pay for
// the comparison and a barrier (us without and with: dx of 64 rows 21.8, 22.1; dw13
// of 64 rows of 4,096 x 4,096 24.7, 25.1; dx and dw13 of 1,237 rows 89, 90; the two
// walks as one loop 0.3 to 1 more on the small ones).
//
// The walk.  A stage's 2 SI PARTS operand groups (one A subtile, SJ matrix
// instructions) run in order; operands are read from LDS two groups ahead.
// The last quarter of the groups has all of its operands in registers, and the
// barrier stands before it: there every wave has read the stage to the end and
// the next stage has landed.  Behind the barrier the loads of the stage after
// next start into the buffer just read, the next stage's first operands are
// read, and the last quarter's matrix instructions cover both.  So a stage's
// loads have a whole stage to land in, and the matrix pipes do not run dry at
// the barrier.  The wait before it is a full one: direct-to-LDS loads are not
// counted as still on their way.
//
// TURNS: half of the waves load the even stages and half the odd ones, each wave
// twice as much, into three buffers.  A wave waits, fully, at every other barrier,
// so that two stages are on their way at a time and a stage has two stages' time
// to land.  Tiles of which three stages fit LDS do this (us with and without, K
// 4,096, 2,048 columns of h: 64 rows in 32 x 64 tiles 14.7, 19.0; 256 rows in 64
// x 64 19.6, 27.4; 512 rows in 64 x 128 26.8, 33.4; 2,048 rows in 128 x 256 59.5,
// 63.6; dx of 1,237 rows of 2,560, a sum over 2,832, in 128 x 128 30.1, 36.1).
// Loads alone, without products, take 0.67 us a stage of 128 x 128 tiles with one
// stage on its way, 0.41 with two, 0.47 with four: one more half of the waves and
// one more buffer are worth it, three more are not.
//
// What bounds it.  256 x 256 tiles: the matrix pipes, 1.16 to 1.21 PFLOP/s forward at
// 4,096 rows with the sums kept, 1.22 to 1.29 at 16,384, and 1.18 to 1.26 backward at
// 4,096, where a library product reaches 1.22 to 1.26; 60 % of the pipes' busy cycles
// at the clock that the chip holds.  Of 116 us of
// such a product 88 are left without the loads, 91 without the LDS reads and 71
// without the matrix instructions.  Smaller tiles: the loads from L2 (14 to 18 TB/s
// over the chip with two stages on their way), since with fewer rows each weight
// meets less work.  Tried and not faster: 4 waves of 128 x 128
// (116 to 124 for 110), half or three eighths of the groups behind the barrier,
// loads between single matrix instructions.
template <bool AROW, bool BROW, int WI, int WJ, int SI, int SJ, int KG, int PARTS, bool GATE, bool TURNS, int OCC>
__global__ __launch_bounds__(WI * WJ * KG * 64, OCC) void gu_tile_kernel(TileArgs p) {
  constexpr int NW = WI * WJ;
  constexpr int LW = TURNS ? NW / 2 : NW;          // waves that load a slice
  constexpr int BUFS = TURNS ? 3 : 2;
  constexpr int BM = WI * SI * 16, BN = WJ * SJ * 16;
  typedef Operand<AROW, BM, LW, false> OpA;
  typedef Operand<BROW, BN, LW, !BROW> OpB;
  constexpr int A_BYTES = PARTS * OpA::BYTES;
  constexpr int SLICE = A_BYTES + OpB::BYTES;
  constexpr int STAGE = KG * SLICE;
  constexpr int JOIN = (KG - 1) * BM * BN * 4;
  constexpr int FLAGS = PARTS > 1 && TURNS ? NW * 4 : 0;
  constexpr int LDS = BUFS * STAGE + FLAGS > JOIN ? BUFS * STAGE + FLAGS : JOIN;
  static_assert(!GATE || !BROW, "w13's rows are columns of out");
  static_assert(!GATE || SJ == 4, "a wave holds a pair of gate and a pair of up subtiles");
  __shared__ __attribute__((aligned(1024))) uint8_t s_all[LDS];

  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG > 1 ? wid / NW : 0;
  const int wi = wid % NW / WJ, wj = wid % NW % WJ;
  // what this wave loads: share `wave` of group lg's slice, with TURNS of the
  // stages of parity `turn` (each SIMD holds waves of both)
  const int turn = TURNS ? wid / (LW * KG) : 0;
  const int lg = TURNS ? wid % (LW * KG) / LW : kg;
  const int wave = wid % LW;

  const int tiles = p.tiles_i * p.tiles_j;
  const int split = blockIdx.x / (uint32_t)tiles;
  int ti, tj;
  tile_of(blockIdx.x - split * tiles, tiles, p.tiles_i, p.tiles_j, ti, tj);
  const int i0 = ti * BM;
  const int j0 = tj * (GATE ? BN / 2 : BN);

  // Source offsets of this lane's loads from the tile's base; lanes outside the
  // matrix read zeros.
  uint32_t avo[OpA::LOADS], bvo[OpB::LOADS];
  int aseg[OpA::LOADS], bseg[OpB::LOADS];
#pragma unroll
  for (int j = 0; j < OpA::LOADS; ++j) {
    const int row = OpA::row(wave, j), seg = OpA::seg(row);
    aseg[j] = seg * 8;
    if (AROW) avo[j] = i0 + seg * 8 < p.I ? (uint32_t)(row * p.lda * 2) + seg * 16 : kLaneOob;
    else avo[j] = i0 + row < p.I ? (uint32_t)(row * p.lda * 2) + seg * 16 : kLaneOob;
  }
  bool up[OpB::LOADS];             // GATE: the load's rows are up rows
#pragma unroll
  for (int j = 0; j < OpB::LOADS; ++j) {
    const int row = OpB::row(wave, j), seg = OpB::seg(row);
    bseg[j] = seg * 8;
    up[j] = false;
    if (BROW) {
      bvo[j] = j0 + seg * 8 < p.J ? (uint32_t)(row * p.ldb * 2) + seg * 16 : kLaneOob;
    } else if (GATE) {
      // pairs of 32 rows: gate, up, gate, up ...; a load's eight rows lie in one
      const int pair = row >> 5, col = (pair >> 1) * 32 + (row & 31);
      up[j] = (((wave * OpB::LOADS + j) * OpB::ROWS) >> 5) & 1;
      bvo[j] = j0 + col < p.J ? (uint32_t)(col * p.ldb * 2) + seg * 16 : kLaneOob;
    } else {
      bvo[j] = j0 + row < p.J ? (uint32_t)(row * p.ldb * 2) + seg * 16 : kLaneOob;
    }
  }

  // The next stage to load: this group's KG stages on from its last.
  const int stages = (p.R + GU_BK - 1) / GU_BK;
  const int begin = (split * p.steps + turn) * KG + lg;
  int at = begin;
  int64_t part_stride = p.part_stride;
  const uint32_t l0 = lds_addr(s_all) + lg * SLICE;
  constexpr uint32_t OPEN = 0x7FFE0000u;   // lanes outside are marked: the range need not end anywhere
  auto load_a = [&](int buf) __attribute__((always_inline)) {
    const bool live = at < stages;
    const int r0 = live ? at * GU_BK : 0;
    const int left = p.R - r0;             // r of the stage that exist, or more
    const uint32_t bytes = AROW ? (uint32_t)((min(left, GU_BK) * p.lda - i0) * 2) : OPEN;
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
      const uint16_t* base = p.a + q * part_stride + (AROW ? (int64_t)r0 * p.lda + i0 : (int64_t)i0 * p.lda + r0);
      const u32x4_t rs = only_if(live, make_rsrc(base, bytes));
#pragma unroll
      for (int j = 0; j < OpA::LOADS; ++j) {
        const uint32_t vo = AROW || aseg[j] < left ? avo[j] : kLaneOob;
        load_lds16<false>(l0 + buf * STAGE + q * OpA::BYTES + (wave * OpA::LOADS + j) * 1024, rs, vo, 0);
      }
    }
  };
  auto load_b = [&](int buf) __attribute__((always_inline)) {
    const bool live = at < stages;
    const int r0 = live ? at * GU_BK : 0;
    const int left = p.R - r0;
    const uint16_t* base = p.b + (BROW ? (int64_t)r0 * p.ldb + j0 : (int64_t)j0 * p.ldb + r0);
    const uint32_t bytes = BROW ? (uint32_t)((min(left, GU_BK) * p.ldb - j0) * 2) : OPEN;
    const u32x4_t rs = only_if(live, make_rsrc(base, bytes));
    const u32x4_t ru = GATE ? only_if(live, make_rsrc(base + (int64_t)p.J * p.ldb, bytes)) : rs;
#pragma unroll
    for (int j = 0; j < OpB::LOADS; ++j) {
      const uint32_t vo = BROW || bseg[j] < left ? bvo[j] : kLaneOob;
      load_lds16<false>(l0 + buf * STAGE + A_BYTES + (wave * OpB::LOADS + j) * 1024, up[j] ? ru : rs, vo, 0);
    }
  };
  auto load_stage = [&](int buf) __attribute__((always_inline)) {
    load_a(buf);
    load_b(buf);
    at += (TURNS ? 2 : 1) * KG;
  };
  f32x4_t acc[SI][SJ];

  constexpr int SP = SI * PARTS;
  constexpr int NQ = 2 * SP;                       // operand groups of a stage
  constexpr int HOLD = NQ >= 4 ? NQ / 4 : 1;       // behind the barrier
  constexpr int CA = SP >= 2 ? 2 : 1;              // A operands read a stage ahead
  u32x4_t fa[NQ], fb[2][SJ];
  auto read_a = [&](int buf, int q) __attribute__((always_inline)) {
    fa[q] = OpA::read(s_all + buf * STAGE + kg * SLICE + q % PARTS * OpA::BYTES, wi * SI * 16, q % SP / PARTS, q / SP);
  };
  auto read_b = [&](int buf, int ks, int s) __attribute__((always_inline)) {
    fb[ks][s] = OpB::read(s_all + buf * STAGE + kg * SLICE + A_BYTES, wj * SJ * 16, s, ks);
  };
  auto mults = [&](int q) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < SJ; ++s)
      acc[q % SP / PARTS][s] = gu_mfma(fb[q / SP][s], fa[q], acc[q % SP / PARTS][s]);
  };

  const int steps = p.steps;
  auto first = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < SJ; ++s) read_b(0, 0, s);
#pragma unroll
    for (int q = 0; q < CA; ++q) read_a(0, q);
  };

  // Stage st, from buffer buf; stage st + 1 is in buffer `after`.  `mine`: this
  // wave's loads are of stage st + 1, and then of the one that takes st's place.
  auto step = [&](int buf, int after, bool mine) __attribute__((always_inline)) {
    // reads in the order of need: A of the first half and B of the second
    // between them, then A of the second
    constexpr int READS = NQ - CA + SJ;
    constexpr int FRONT = NQ - HOLD;               // groups before the barrier
    int done = 0;
#pragma unroll
    for (int q = 0; q < FRONT; ++q) {
      __builtin_amdgcn_sched_barrier(0);
      constexpr int FIRST = SP - CA;               // A reads of the first half
      const int upto = q == FRONT - 1 ? READS : (READS * (q + 1) + FRONT - 1) / FRONT;
#pragma unroll
      for (int k = 0; k < READS; ++k) {
        if (k < done || k >= upto) continue;
        constexpr int MIX = FIRST < SJ ? FIRST : SJ;
        if (k < 2 * MIX) {
          if (k & 1) read_b(buf, 1, k >> 1);
          else read_a(buf, CA + (k >> 1));
        } else {
          const int rest = k - 2 * MIX;            // one of the two is done
          if (FIRST > SJ) read_a(buf, CA + MIX + rest);
          else if (rest < SJ - MIX) read_b(buf, 1, MIX + rest);
          else read_a(buf, SP + rest - (SJ - MIX));
        }
      }
      done = upto;
      mults(q);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (mine) vm_wait();
    lds_barrier();
    u32x4_t na[CA], nb[SJ];
    {
      const uint8_t* nx = s_all + after * STAGE + kg * SLICE;
#pragma unroll
      for (int s = 0; s < SJ; ++s) nb[s] = OpB::read(nx + A_BYTES, wj * SJ * 16, s, 0);
#pragma unroll
      for (int q = 0; q < CA; ++q) na[q] = OpA::read(nx + q % PARTS * OpA::BYTES, wi * SI * 16, q / PARTS, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = NQ - HOLD; q < NQ; ++q) {
      mults(q);
      __builtin_amdgcn_sched_barrier(0);
      if (q == NQ - HOLD && mine) {
        load_a(buf);
        if (HOLD == 1) load_b(buf);
      }
      if (q == NQ - HOLD + 1 && mine) load_b(buf);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (mine) at += (TURNS ? 2 : 1) * KG;
#pragma unroll
    for (int s = 0; s < SJ; ++s) fb[0][s] = nb[s];
#pragma unroll
    for (int q = 0; q < CA; ++q) fa[q] = na[q];
  };
  auto walk = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int a = 0; a < SI; ++a)
#pragma unroll
      for (int s = 0; s < SJ; ++s) acc[a][s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if constexpr (TURNS) {
      int st = 0, buf = 0;
      auto one = [&](bool mine) __attribute__((always_inline)) {
        const int after = buf == 2 ? 0 : buf + 1;
        step(buf, after, mine);
        buf = after;
        return ++st < steps;
      };
      // Stage 1 is the other half's: the waves that have loaded stage 0 begin with a
      // step without loads.  From there on a step with and one without follow one
      // another for every wave.
      bool more = true;
      if (turn == 0) {
        load_stage(0);
        vm_wait();
        lds_barrier();
        load_stage(2);
        first();
        more = one(false);
      } else {
        load_stage(1);
        lds_barrier();
        first();
      }
#pragma unroll 1
      while (more) {
        more = one(true);
        if (!more) break;
        more = one(false);
      }
    } else {
      load_stage(0);
      load_stage(1);
      vm_wait();
      lds_barrier();
      first();
#pragma unroll 1
      for (int st = 0; st < steps; ++st) step(st & 1, (st & 1) ^ 1, true);
    }
    vm_wait();      // the loads past the last stage land before LDS is used again
  };

  const int c16 = lane & 15, g = lane >> 4;
  if constexpr (PARTS > 1) {
    static_assert(KG == 1 && !GATE && SI * SJ * 4 <= 64, "a bit per result of a lane");
    uint64_t nan = 0;                      // the first walk's results that were
    // A word of wave w's, where nothing is read or on its way once its own loads have
    // landed: with two buffers in the last stage's, where its loads past the end went.
    auto flag = [&](int w) __attribute__((always_inline)) {
      return reinterpret_cast<uint32_t*>(s_all + (TURNS ? BUFS * STAGE + w * 4 : ((steps - 1) & 1) * STAGE + w * OpA::LOADS * 1024));
    };
    walk();
    const int64_t row0 = (int64_t)split * p.I + i0 + wi * SI * 16 + c16;
    const int rows = p.I - i0 - wi * SI * 16 - c16, col0 = j0 + wj * SJ * 16 + g * 4;
    float* const out = static_cast<float*>(p.out) + row0 * p.J + col0;
#pragma unroll
    for (int a = 0; a < SI; ++a) {
      if (a * 16 >= rows) continue;
#pragma unroll
      for (int c = 0; c < SJ; ++c)
        if (col0 + c * 16 < p.J) gu_store4(out, false, (int64_t)a * 16 * p.J + c * 16, acc[a][c]);
    }
    bool bad = false;
#pragma unroll
    for (int q = 0; q < SI * SJ * 2; ++q)
      bad |= __builtin_isunordered(acc[q / SJ / 2][q / 2 % SJ][q % 2 * 2], acc[q / SJ / 2][q / 2 % SJ][q % 2 * 2 + 1]);
    const uint64_t any = __ballot(bad);
    if (lane == 0) *flag(wid) = any != 0;
    lds_barrier();
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) all |= *flag(w);
    if (__builtin_expect(uniform(all) == 0, 1)) return;
#pragma unroll
    for (int q = 0; q < SI * SJ * 4; ++q) {
      const float v = acc[q / SJ / 4][q / 4 % SJ][q % 4];
      nan |= (uint64_t)(v != v) << q;
    }
    lds_barrier();
    part_stride = 0;
    at = begin;
    walk();
#pragma unroll
    for (int q = 0; q < SI * SJ * 4; ++q) {
      const int a = q / SJ / 4, c = q / 4 % SJ;
      if (nan >> q & 1 && a * 16 < rows && col0 + c * 16 < p.J) out[(int64_t)a * 16 * p.J + c * 16 + q % 4] = acc[a][c][q % 4];
    }
    return;
  } else {
    walk();
  }

  if constexpr (KG > 1) {
    lds_barrier();
    f32x4_t* sum = reinterpret_cast<f32x4_t*>(s_all) + wid % NW * SI * SJ * 64 + lane;
    constexpr int GROUP = NW * SI * SJ * 64;
    if (kg > 0) {
#pragma unroll
      for (int q = 0; q < SI * SJ; ++q) sum[(kg - 1) * GROUP + q * 64] = acc[q / SJ][q % SJ];
    }
    lds_barrier();
    if (kg > 0) return;
#pragma unroll 1
    for (int k = 0; k < KG - 1; ++k)
#pragma unroll
      for (int q = 0; q < SI * SJ; ++q) acc[q / SJ][q % SJ] += sum[k * GROUP + q * 64];
  }

#pragma unroll
  for (int a = 0; a < SI; ++a) {
    const int row = i0 + wi * SI * 16 + a * 16 + c16;
    if (row >= p.I) continue;
    if constexpr (GATE) {
      const int col = j0 + wj * 32 + g * 8;
      if (col >= p.J) continue;
      float gt[8], ut[8], h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        gt[i] = acc[a][i >> 2][i & 3];
        ut[i] = acc[a][2 + (i >> 2)][i & 3];
        h[i] = gu_silu(gt[i]) * ut[i];
      }
      gu_store8(p.out, p.out_bf16, (int64_t)row * p.J + col, h);
      if (p.pre) {
        gu_store8(p.pre, p.pre_bf16, (int64_t)row * 2 * p.J + col, gt);
        gu_store8(p.pre, p.pre_bf16, (int64_t)row * 2 * p.J + p.J + col, ut);
      }
    } else {
#pragma unroll
      for (int c = 0; c < SJ; ++c) {
        const int col = j0 + wj * SJ * 16 + c * 16 + g * 4;
        if (col < p.J) gu_store4(p.out, p.out_bf16, ((int64_t)split * p.I + row) * p.J + col, acc[a][c]);
      }
    }
  }
}

template <bool AROW, bool BROW, int WI, int WJ, int SI, int SJ, int KG, int PARTS, bool GATE, bool TURNS, int OCC>
static hipError_t launch_tiles(TileArgs a, hipStream_t stream) {
  constexpr int BM = WI * SI * 16, BN = WJ * SJ * 16, CN = GATE ? BN / 2 : BN;
  a.tiles_i = (a.I + BM - 1) / BM;
  a.tiles_j = (a.J + CN - 1) / CN;
  const int stages = ((a.R + GU_BK - 1) / GU_BK + KG - 1) / KG;
  a.steps = (stages + a.splits - 1) / a.splits;
  const int64_t groups = (int64_t)a.tiles_i * a.tiles_j * a.splits;
  hipLaunchKernelGGL((gu_tile_kernel<AROW, BROW, WI, WJ, SI, SJ, KG, PARTS, GATE, TURNS, OCC>), dim3((unsigned)groups),
                     dim3(WI * WJ * KG * 64), 0, stream, a);
  return hipGetLastError();
}

constexpr int GS_NT = 2;       // non-temporal: weights are read once

// ---------------------------------------------------------------------------
// Few rows: the weights stream through registers
// ---------------------------------------------------------------------------

struct StreamArgs {
  const uint16_t* x;
  const uint16_t* w;
  int64_t K;
  int M, F, blocks;        // blocks of 8 columns of h of a workgroup
  void* h;
  int h_bf16;
  void* pre;
  int pre_bf16;
};

// A tile is 8 gate rows of w13 and the 8 up rows that belong to them, 256 k deep:
// 8 KiB, loaded by one wave in runs of 512 bytes and turned into the matrix
// unit's order through LDS of the wave's own (the operand's lanes lie across the
// rows, 16 bytes each: loaded that way, every lane is a cache access of its own,
// and the L1 takes one a cycle).  The 16 rows of x come along with the tiles in
// the same way.  A workgroup's waves share K, in units of 256; blocks of 8
// columns of h follow one another; two tiles in flight per wave.
//
// Bound by memory where the weights come from there, and by the start of the
// stream where they do not (33.6 MB of w13, one row: 10.7 us a call, 8.0 at best,
// for 6.6 at a copy's rate).  Tiles with 17 rows and more: at 16 rows the stream
// takes 11.6 us, at 17 the smallest tiles 15.8; a row more would take a second x.
constexpr int GS_WAVES = 8;
constexpr int GS_ROWS = 16;

__global__ __launch_bounds__(GS_WAVES * 64) void gu_stream_kernel(StreamArgs p) {
  constexpr int D = 2;
  __shared__ __attribute__((aligned(512))) uint8_t s_tile[GS_WAVES][2][8192];
  __shared__ float s_part[2][GS_WAVES][4][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;                        // a unit of every block each at least
  const int n16 = lane & 15, g = lane >> 4;
  const int K = (int)p.K;
  const int total = (K + 255) >> 8;
  const int j0 = blockIdx.x * p.blocks * 8;                 // first column of h
  const int cols = min(p.blocks * 8, p.F - j0);
  const int blocks = (cols + 7) >> 3;

  // load i of a tile: rows 2 i and 2 i + 1, a half of the wave each; segment c of
  // row r at place c ^ r of its 32
  const int half = lane >> 5, seg = lane & 31;
  const uint32_t rvo = (uint32_t)half * (uint32_t)(K * 2) + seg * 16;
  uint8_t* tile = s_tile[wave][0];
  const __amdgpu_buffer_rsrc_t xr = gu_rsrc(p.x, (int64_t)p.M * K * 2);

  struct Slot {
    u32x4_t w[8], x[8];
  };
  Slot ring[D];
  int lu = wave, lb = 0;                                    // unit and block of the next load
  auto load = [&](Slot& q) __attribute__((always_inline)) {
    const int left = lb < blocks ? (cols - lb * 8) : 0;     // columns from here on
    const uint16_t* base = p.w + (int64_t)(j0 + lb * 8) * K;
    const uint32_t bytes = (uint32_t)max(0, min(left, 8)) * (uint32_t)(K * 2);
    const __amdgpu_buffer_rsrc_t gr = gu_rsrc(base, bytes), ur = gu_rsrc(base + (int64_t)p.F * K, bytes);
    const uint32_t vo = lu * 256 + seg * 8 < K ? rvo : kLaneOob;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      q.w[i] = __builtin_amdgcn_raw_buffer_load_b128(i < 4 ? gr : ur, vo, (i & 3) * K * 4 + lu * 512, GS_NT);
#pragma unroll
    for (int i = 0; i < 8; ++i) q.x[i] = __builtin_amdgcn_raw_buffer_load_b128(xr, vo, i * K * 4 + lu * 512, 0);
    lu += waves;
    if (lu >= total) {
      lu = wave;
      ++lb;
    }
  };
#pragma unroll
  for (int i = 0; i < D; ++i) {
    load(ring[i]);
    __builtin_amdgcn_sched_barrier(0);
  }

  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  auto join = [&](int blk) __attribute__((always_inline)) {
    float (*part)[4][64] = s_part[blk & 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][i][lane] = acc[i];
    acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    lds_barrier();
    const int live = min(cols - blk * 8, 8);
    // eight lanes to a column's row: one a wave
    for (int o = threadIdx.x >> 3; o < p.M * 8; o += blockDim.x >> 3) {
      const int w = threadIdx.x & 7, c = o & 7, row = o >> 3;
      float gt = 0.f, ut = 0.f;
      if (w < waves) {
        const float* from = &part[w][row & 3][(row >> 2) * 16 + c];
        gt = from[0];
        ut = from[8];
      }
      gt += dpp_from<0xB1>(gt), ut += dpp_from<0xB1>(ut);
      gt += dpp_from<0x4E>(gt), ut += dpp_from<0x4E>(ut);
      gt += dpp_from<0x141>(gt), ut += dpp_from<0x141>(ut);
      if (w != 0 || c >= live) continue;
      const float h = gu_silu(gt) * ut;
      const int col = j0 + blk * 8 + c;
      const int64_t at = (int64_t)row * p.F + col;
      if (p.h_bf16) reinterpret_cast<uint16_t*>(p.h)[at] = f32_to_bf16_rne(h);
      else reinterpret_cast<float*>(p.h)[at] = h;
      if (p.pre) {
        const int64_t pa = (int64_t)row * 2 * p.F + col;
        if (p.pre_bf16) {
          reinterpret_cast<uint16_t*>(p.pre)[pa] = f32_to_bf16_rne(gt);
          reinterpret_cast<uint16_t*>(p.pre)[pa + p.F] = f32_to_bf16_rne(ut);
        } else {
          reinterpret_cast<float*>(p.pre)[pa] = gt;
          reinterpret_cast<float*>(p.pre)[pa + p.F] = ut;
        }
      }
    }
  };

  // the tiles of this wave: `per` units of each block
  const int per = (total - wave + waves - 1) / waves;
  int u = 0, blk = 0;
  while (blk < blocks) {
#pragma unroll
    for (int i = 0; i < D; ++i) {
      if (i > 0 && blk >= blocks) break;
      Slot& q = ring[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int row = 2 * c + half, place = row * 512 + ((seg ^ row) << 4);
        *reinterpret_cast<u32x4_t*>(tile + place) = q.w[c];
        *reinterpret_cast<u32x4_t*>(tile + 8192 + place) = q.x[c];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint8_t* from = tile + n16 * 512 + (((s * 4 + g) ^ n16) << 4);
        acc = gu_mfma(*reinterpret_cast<const u32x4_t*>(from + 8192), *reinterpret_cast<const u32x4_t*>(from), acc);
      }
      __builtin_amdgcn_sched_barrier(0);
      load(q);
      __builtin_amdgcn_sched_barrier(0);
      if (++u == per) {
        u = 0;
        join(blk++);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The activation's gradient, and sums of shares
// ---------------------------------------------------------------------------

template <bool BF16>
__device__ __forceinline__ void gu_load8(const void* p, int64_t i, float (&v)[8]) {
  if (BF16) {
    const u32x4_t q = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = c & 1 ? bf16_hi(q[c >> 1]) : bf16_lo(q[c >> 1]);
  } else {
    const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// v as the sum of PARTS bf16 values: the nearest one, then the nearest one to
// what is left (24 bits in three).  A value that is not finite is its own first
// part alone.
template <int PARTS>
__device__ __forceinline__ void gu_store_parts(uint16_t* d, int64_t stride, int64_t i, float (&v)[8]) {
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = pack_bf16(v[2 * c], v[2 * c + 1]);
    *reinterpret_cast<uint4*>(d + q * stride + i) = make_uint4(w[0], w[1], w[2], w[3]);
    if (q + 1 < PARTS) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float r = v[c] - (c & 1 ? bf16_hi(w[c >> 1]) : bf16_lo(w[c >> 1]));
        v[c] = fabsf(r) < 3.0e38f ? r : 0.f;
      }
    }
  }
}

// d = [dg du] of [M, 2F] sums and dh [M, F], eight columns of each a thread, in
// bf16 (PARTS 1), or in three bf16 matrices that add up to the f32 value.
template <bool PBF16, bool HBF16, int PARTS>
__global__ __launch_bounds__(256) void gu_act_bwd_kernel(const void* __restrict__ pre, const void* __restrict__ dh,
                                                         int64_t M, int F, uint16_t* __restrict__ d) {
  const int64_t per = F / 8, total = M * per;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t m = i / per;
    const int64_t at = m * 2 * F + (i - m * per) * 8;
    float gt[8], ut[8], hv[8];
    gu_load8<PBF16>(pre, at, gt);
    gu_load8<PBF16>(pre, at + F, ut);
    gu_load8<HBF16>(dh, at - m * F, hv);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float s = gu_sigmoid(gt[c]);
      const float dg = hv[c] * ut[c] * s * (1.0f + gt[c] * (1.0f - s));
      ut[c] = hv[c] * gt[c] * s;
      gt[c] = dg;
    }
    gu_store_parts<PARTS>(d, M * 2 * F, at, gt);
    gu_store_parts<PARTS>(d, M * 2 * F, at + F, ut);
  }
}

// out = sum of `splits` f32 matrices of n values, in order.
__global__ __launch_bounds__(256) void gu_join_kernel(const float* __restrict__ part, int splits, int64_t n,
                                                      void* __restrict__ out, int bf16) {
  for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) * 8; i < n;
       i += (int64_t)gridDim.x * blockDim.x * 8) {
    float v[8];
    gu_load8<false>(part, i, v);
    for (int s = 1; s < splits; ++s) {
      float w[8];
      gu_load8<false>(part + s * n, i, w);
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] += w[c];
    }
    gu_store8(out, bf16, i, v);
  }
}

static unsigned gu_grid(int64_t threads) {
  const int64_t g = (threads + 255) / 256;
  return (unsigned)(g < (int64_t(1) << 22) ? g : (int64_t(1) << 22));
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The smallest tiles that a launch takes (shares of a sum add workgroups only
// where they are few).
int64_t gate_up_workgroups(int32_t M, int32_t N, int32_t K) {
  const int64_t fwd = ceil_div(M, 32) * ceil_div(N / 2, 32), dx = ceil_div(M, 64) * ceil_div(K, 128);
  const int64_t dw = ceil_div(N, 128) * ceil_div(K, 128);
  const int64_t most = fwd > dx ? fwd : dx;
  return most > dw ? most : dw;
}

// The tile kernel's instances, and what a stage of 64 r costs them when all the
// workgroups that fit the CUs run (us, from 4,096 x 4,096 products; a stage of KG
// groups counts KG).  A product takes the instance, and the shares of its sum,
// of the least estimate: whole rounds of workgroups, and for shares the sums
// written, read and added at 4.5 TB/s in one more launch.  The sides measured, us
// (the instance taken first; sN: in N shares, without the launch that adds them):
//   gate/up, K 4,096, 2,048 columns of h: 64 rows 32 x 64 tiles 14.7, 64 x 64
//     18.4, 64 x 128 24.5; 256 rows 64 x 64 19.6, 64 x 128 25.3, 32 x 64 26.4; 512
//     rows 64 x 128 26.8, 64 x 64 34.1, 128 x 128 36.3; 1,024 rows 128 x 128
//     38.5, 64 x 128 47.3, 128 x 256 50.5; 2,048 rows 128 x 256 59.5, 128 x 128
//     75.6, 256 x 256 93.3; 4,096 rows 256 x 256 106.7, 128 x 256 113.4
//   dx of 1,237 rows (2,560 columns, sum over 2,832): 128 x 128 30.1, 128 x 256
//     in s2 30.4, 64 x 128 35.8, 256 x 256 in s4 37.1
//   dx of 64 rows (4,096 columns and sums): 64 x 128 in s8 12.2, s4 13.3, 128 x
//     128 in s8 13.3; from three parts 64 x 128 in s8 15.8, 64 x 256 in s8 19.3
//   dw13 of 2,832 x 2,560 over 1,237 rows: 256 x 128 27.9, 128 x 128 31.9, 256 x
//     256 in s2 33.5, alone 44.7
struct TileConfig {
  int bm, bn, kg, fit;    // rows, columns (gate and up: of w13), groups, workgroups that run at once
  float stage, alone;     // a stage with `fit` workgroups, and with one per CU at most
};

struct TilePlan {
  int config, splits;
};

template <int COUNT>
static TilePlan tile_plan(const TileConfig (&configs)[COUNT], int gate, int64_t I, int64_t J, int64_t R,
                          int most_splits) {
  TilePlan best = {0, 1};
  float least = 0.f;
  for (int c = 0; c < COUNT; ++c) {
    const TileConfig& t = configs[c];
    const int64_t tiles = ceil_div(I, t.bm) * ceil_div(J, gate ? t.bn / 2 : t.bn);
    const int64_t stages = ceil_div(ceil_div(R, GU_BK), t.kg);
    for (int splits = 1; splits <= most_splits && splits <= stages; splits *= 2) {
      if (splits > 1 && tiles * splits > 2 * t.fit) break;
      const float stage = tiles * splits <= GU_CUS ? t.alone : t.stage;
      float us = (float)ceil_div(tiles * splits, t.fit) * (3.f + (float)(ceil_div(stages, splits) * t.kg) * stage);
      if (splits > 1) us += 4.f + (float)splits * (float)I * (float)J * (8.f / 4.5e6f);
      if (least == 0.f || us < least) {
        least = us;
        best = {c, splits};
      }
    }
  }
  return best;
}

static const TileConfig kForward[] = {{256, 256, 1, 256, 1.57f, 1.57f}, {128, 256, 1, 256, .88f, .88f},
                                      {128, 128, 1, 256, .56f, .56f},   {64, 128, 2, 256, .37f, .37f},
                                      {64, 64, 2, 256, .26f, .26f},     {32, 64, 4, 256, .19f, .19f}};
static const TileConfig kDx[] = {{256, 256, 1, 256, 1.65f, 1.65f}, {128, 256, 1, 256, .93f, .93f},
                                 {128, 128, 1, 256, .6f, .6f}, {64, 128, 1, 512, .68f, .4f}};
static const TileConfig kDx3[] = {{128, 256, 1, 256, 2.1f, 2.1f}, {64, 256, 1, 256, 1.3f, 1.3f},
                                  {64, 128, 1, 256, .7f, .7f}};
static const TileConfig kDw[] = {{256, 256, 1, 256, 1.7f, 1.7f}, {256, 128, 1, 256, .93f, .93f},
                                 {128, 128, 1, 256, .6f, .6f}};
static const TileConfig kDw3[] = {{128, 256, 1, 256, 2.2f, 2.2f}};
constexpr int GU_SPLITS = 16;

static hipError_t launch_forward(int config, const TileArgs& a, hipStream_t s) {
  switch (config) {
    case 0: return launch_tiles<false, false, 2, 4, 8, 4, 1, 1, true, false, 2>(a, s);
    case 1: return launch_tiles<false, false, 2, 4, 4, 4, 1, 1, true, true, 2>(a, s);
    case 2: return launch_tiles<false, false, 4, 2, 2, 4, 1, 1, true, true, 2>(a, s);
    case 3: return launch_tiles<false, false, 2, 2, 2, 4, 2, 1, true, true, 2>(a, s);
    case 4: return launch_tiles<false, false, 4, 1, 1, 4, 2, 1, true, true, 2>(a, s);
    default: return launch_tiles<false, false, 2, 1, 1, 4, 4, 1, true, true, 2>(a, s);
  }
}

static hipError_t launch_dx(int parts, int config, const TileArgs& a, hipStream_t s) {
  if (parts == 1) switch (config) {
    case 0: return launch_tiles<false, true, 2, 4, 8, 4, 1, 1, false, false, 2>(a, s);
    case 1: return launch_tiles<false, true, 2, 4, 4, 4, 1, 1, false, true, 2>(a, s);
    case 2: return launch_tiles<false, true, 4, 2, 2, 4, 1, 1, false, true, 2>(a, s);
    default: return launch_tiles<false, true, 4, 2, 1, 4, 1, 1, false, true, 4>(a, s);
  }
  switch (config) {
    case 0: return launch_tiles<false, true, 2, 4, 4, 4, 1, 3, false, false, 2>(a, s);
    case 1: return launch_tiles<false, true, 2, 4, 2, 4, 1, 3, false, false, 2>(a, s);
    default: return launch_tiles<false, true, 4, 2, 1, 4, 1, 3, false, true, 2>(a, s);
  }
}

static hipError_t launch_dw(int parts, int config, const TileArgs& a, hipStream_t s) {
  if (parts == 3) return launch_tiles<true, true, 2, 4, 4, 4, 1, 3, false, false, 2>(a, s);
  switch (config) {
    case 0: return launch_tiles<true, true, 2, 4, 8, 4, 1, 1, false, false, 2>(a, s);
    case 1: return launch_tiles<true, true, 4, 2, 4, 4, 1, 1, false, true, 2>(a, s);
    default: return launch_tiles<true, true, 4, 2, 2, 4, 1, 1, false, true, 2>(a, s);
  }
}

hipError_t launch_gate_up(const uint16_t* x, const uint16_t* w, int32_t M, int32_t N, int32_t K, void* h, int h_bf16,
                          void* pre, int pre_bf16, hipStream_t stream) {
  const int F = N / 2;
  if (M <= GS_ROWS) {
    const int all = (F + 7) / 8, per = (all + GU_CUS - 1) / GU_CUS;
    StreamArgs a = {x, w, K, M, F, per, h, h_bf16, pre, pre_bf16};
    const int units = (K + 255) / 256, waves = units < GS_WAVES ? units : GS_WAVES;
    hipLaunchKernelGGL(gu_stream_kernel, dim3((all + per - 1) / per), dim3(waves * 64), 0, stream, a);
    return hipGetLastError();
  }
  TileArgs a = {};
  a.a = x; a.b = w; a.lda = K; a.ldb = K;
  a.I = M; a.J = F; a.R = K;
  a.splits = 1;
  a.out = h; a.out_bf16 = h_bf16; a.pre = pre; a.pre_bf16 = pre_bf16;
  return launch_forward(tile_plan(kForward, 1, M, F, K, 1).config, a, stream);
}

// The plan of the gradients: bf16 parts of d, and each product's instance and
// shares, whose f32 sums lie behind d (dx's are added up before dw13's begin).
//
// Parts.  A bf16 result takes the first part alone, d rounded to bf16: a bf16 factor
// is multiplied by bf16 only, so that more bits of d are further products, and dh,
// the kept sums and the result are mostly bf16 themselves.  Both sides, 4,096 rows of 4,096 x
// 4,096, both gradients: one part 240 us, 2-norm of the error 2.35e-3 of the
// result's; three parts 630 us, 7e-7, and 1.66e-3 once rounded to bf16.  A mixed call
// does the same, so that a gradient's bits do not depend on the other's type.
struct BwdPlan {
  int parts;
  TilePlan dx, dw;
  int64_t d_bytes, ws_bytes;
};

static BwdPlan bwd_plan(int32_t M, int32_t N, int32_t K, int want_dx, int dx_bf16, int want_dw, int dw_bf16) {
  BwdPlan p = {};
  p.parts = (want_dx && !dx_bf16) || (want_dw && !dw_bf16) ? 3 : 1;
  p.d_bytes = ((int64_t)p.parts * M * N * 2 + 255) / 256 * 256;
  int64_t sums = 0;
  if (want_dx) {
    p.dx = dx_bf16 ? tile_plan(kDx, 0, M, K, N, GU_SPLITS) : tile_plan(kDx3, 0, M, K, N, GU_SPLITS);
    if (p.dx.splits > 1) sums = (int64_t)p.dx.splits * M * K * 4;
  }
  if (want_dw) {
    p.dw = dw_bf16 ? tile_plan(kDw, 0, N, K, M, GU_SPLITS) : tile_plan(kDw3, 0, N, K, M, GU_SPLITS);
    const int64_t bytes = p.dw.splits > 1 ? (int64_t)p.dw.splits * N * K * 4 : 0;
    sums = bytes > sums ? bytes : sums;
  }
  p.ws_bytes = p.d_bytes + sums;
  return p;
}

int64_t gate_up_bwd_ws(int32_t M, int32_t N, int32_t K, int want_dx, int dx_bf16, int want_dw, int dw_bf16) {
  return bwd_plan(M, N, K, want_dx, dx_bf16, want_dw, dw_bf16).ws_bytes;
}

template <bool P, bool H>
static void launch_act_bwd(int parts, const void* pre, const void* dh, int64_t M, int F, uint16_t* d, hipStream_t s) {
  const dim3 grid(gu_grid(M * (F / 8)));
  if (parts == 1) hipLaunchKernelGGL((gu_act_bwd_kernel<P, H, 1>), grid, dim3(256), 0, s, pre, dh, M, F, d);
  else hipLaunchKernelGGL((gu_act_bwd_kernel<P, H, 3>), grid, dim3(256), 0, s, pre, dh, M, F, d);
}

hipError_t launch_gate_up_bwd(const void* dh, int dh_bf16, const uint16_t* x, const uint16_t* w, const void* pre,
                              int pre_bf16, int32_t M, int32_t N, int32_t K, void* dx, int dx_bf16, void* dw,
                              int dw_bf16, void* ws, hipStream_t stream) {
  const BwdPlan pl = bwd_plan(M, N, K, dx != nullptr, dx_bf16, dw != nullptr, dw_bf16);
  uint16_t* d = static_cast<uint16_t*>(ws);
  const int F = N / 2;
  if (pre_bf16) {
    if (dh_bf16) launch_act_bwd<true, true>(pl.parts, pre, dh, M, F, d, stream);
    else launch_act_bwd<true, false>(pl.parts, pre, dh, M, F, d, stream);
  } else {
    if (dh_bf16) launch_act_bwd<false, true>(pl.parts, pre, dh, M, F, d, stream);
    else launch_act_bwd<false, false>(pl.parts, pre, dh, M, F, d, stream);
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  float* sums = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + pl.d_bytes);
  // out of the product, or of its shares
  auto product = [&](TileArgs a, const TilePlan& t, bool is_dx, int parts, void* out, int out_bf16) {
    a.part_stride = (int64_t)M * N;
    a.splits = t.splits;
    a.out = t.splits > 1 ? sums : out;
    a.out_bf16 = t.splits > 1 ? 0 : out_bf16;
    hipError_t e = is_dx ? launch_dx(parts, t.config, a, stream) : launch_dw(parts, t.config, a, stream);
    if (e != hipSuccess || t.splits == 1) return e;
    const int64_t n = (int64_t)a.I * a.J;
    hipLaunchKernelGGL(gu_join_kernel, dim3(gu_grid(n / 8)), dim3(256), 0, stream, sums, t.splits, n, out, out_bf16);
    return hipGetLastError();
  };
  if (dx) {
    TileArgs a = {};
    a.a = d; a.b = w; a.lda = N; a.ldb = K;
    a.I = M; a.J = K; a.R = N;
    err = product(a, pl.dx, true, dx_bf16 ? 1 : 3, dx, dx_bf16);
    if (err != hipSuccess) return err;
  }
  if (dw) {
    TileArgs a = {};
    a.a = d; a.b = x; a.lda = N; a.ldb = K;
    a.I = N; a.J = K; a.R = M;
    err = product(a, pl.dw, false, dw_bf16 ? 1 : 3, dw, dw_bf16);
  }
  return err;
}

}  // namespace moe
