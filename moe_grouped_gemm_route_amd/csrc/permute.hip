// The token permutation's training side (moe_dispatch, moe_dispatch_bwd,
// moe_combine_bwd) and the unfused SiLU-gated activation (moe_silu_mul).
//
// All four move rows and are bound by HBM.  Pair p = t*k + j of token t sits
// at band row pair_row[p] (below 0 or past the last row: a dropped pair, which
// reads and writes nothing).  Every output element is written by one thread
// and sums run in slot order, so no atomics and the same bits on every call.
//
// A wave takes one unit: VEC consecutive columns per lane, 64 VEC columns of
// a row (of a whole row for the dot products of moe_combine_bwd).  VEC is 8
// where rows allow it (N a multiple of 8: 16-byte bf16 accesses), else 4.
//
// Stores are non-temporal: the rows written are larger than the caches where
// it matters (dispatch of 4,096 tokens to 6 experts, 4,096 columns: 46.7 ->
// 40.2 us).  Loads are too in moe_silu_mul, which reads everything once
// (24,576 x 4,096: 53.2 -> 49.3 us), but not in moe_combine_bwd, whose k waves
// of a token share its dout row (92 -> 103 us).
//
// Measured, bf16, 4,096 tokens top-6, 4,096 columns: dispatch 39-40 us for 235
// MB (5.9-6.0 TB/s; a torch copy of 1 GiB runs at 5.2 on this card, reads alone
// at 6.6), combine_bwd 86-90 us for 437 MB (4.9-5.1), silu_mul 49-50 us for 302
// MB (6.1); dispatch_bwd of f32 rows, 1,237 tokens top-8, 2,560 columns, 19 us
// for 108 MB (5.6).
#include "common.h"
#include "launch.h"
#include "wave.h"

namespace moe {

constexpr int ROW_WAVES = 4;                       // waves per workgroup
constexpr int64_t ROW_GRID_CAP = int64_t(1) << 22; // workgroups; larger problems stride

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

template <bool NT, typename V>
__device__ __forceinline__ V load_word(const V* p) {
  return NT ? __builtin_nontemporal_load(p) : *p;
}

// VEC consecutive elements at element offset i, as f32.
template <bool BF16, int VEC, bool NT = false>
__device__ __forceinline__ void load_vec(const void* __restrict__ p, int64_t i, float (&v)[VEC]) {
  if constexpr (BF16) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + i;
    uint32_t w[VEC / 2];
    if constexpr (VEC == 8) {
      const u32x4_t u = load_word<NT>(reinterpret_cast<const u32x4_t*>(q));
      w[0] = u[0]; w[1] = u[1]; w[2] = u[2]; w[3] = u[3];
    } else {
      const u32x2_t u = load_word<NT>(reinterpret_cast<const u32x2_t*>(q));
      w[0] = u[0]; w[1] = u[1];
    }
#pragma unroll
    for (int c = 0; c < VEC / 2; ++c) {
      v[2 * c] = bf16_lo(w[c]);
      v[2 * c + 1] = bf16_hi(w[c]);
    }
  } else {
    const float* q = reinterpret_cast<const float*>(p) + i;
#pragma unroll
    for (int c = 0; c < VEC; c += 4) {
      const f32x4_t u = load_word<NT>(reinterpret_cast<const f32x4_t*>(q + c));
      v[c] = u[0]; v[c + 1] = u[1]; v[c + 2] = u[2]; v[c + 3] = u[3];
    }
  }
}

template <bool BF16, int VEC>
__device__ __forceinline__ void store_vec(void* __restrict__ p, int64_t i, const float (&v)[VEC]) {
  if constexpr (BF16) {
    uint16_t* q = reinterpret_cast<uint16_t*>(p) + i;
    uint32_t w[VEC / 2];
#pragma unroll
    for (int c = 0; c < VEC / 2; ++c)
      w[c] = pack_bf16(v[2 * c], v[2 * c + 1]);
    if constexpr (VEC == 8) __builtin_nontemporal_store(u32x4_t{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4_t*>(q));
    else __builtin_nontemporal_store(u32x2_t{w[0], w[1]}, reinterpret_cast<u32x2_t*>(q));
  } else {
    float* q = reinterpret_cast<float*>(p) + i;
#pragma unroll
    for (int c = 0; c < VEC; c += 4)
      __builtin_nontemporal_store(f32x4_t{v[c], v[c + 1], v[c + 2], v[c + 3]}, reinterpret_cast<f32x4_t*>(q + c));
  }
}

// xs[pair_row[t*k + j]] = x[t]: each element of x is read once and written k
// times, unchanged (V is 16 or 8 bytes of the row).
template <typename V>
__global__ __launch_bounds__(ROW_WAVES * 64) void dispatch_kernel(const V* __restrict__ x,
                                                                  const int32_t* __restrict__ pair_row, int32_t T,
                                                                  int32_t k, int32_t cols, int32_t chunks,
                                                                  int32_t rows, V* __restrict__ xs) {
  const int lane = threadIdx.x & 63;
  const int64_t units = (int64_t)T * chunks;
  for (int64_t u = blockIdx.x * (int64_t)ROW_WAVES + (threadIdx.x >> 6); u < units;
       u += (int64_t)gridDim.x * ROW_WAVES) {
    const int64_t t = u / chunks;
    const int c = (int)(u - t * chunks) * 64 + lane;
    if (c >= cols) continue;
    const V v = x[t * cols + c];
    for (int j = 0; j < k; ++j) {
      const int r = pair_row[t * k + j];
      if (r >= 0 && r < rows) __builtin_nontemporal_store(v, &xs[(int64_t)r * cols + c]);
    }
  }
}

// dx[t] = sum over j, in slot order, of dxs[pair_row[t*k + j]], in f32.
template <bool IBF16, bool OBF16, int VEC>
__global__ __launch_bounds__(ROW_WAVES * 64) void dispatch_bwd_kernel(const void* __restrict__ dxs,
                                                                      const int32_t* __restrict__ pair_row, int32_t T,
                                                                      int32_t k, int32_t N, int32_t chunks,
                                                                      int32_t rows, void* __restrict__ dx) {
  const int lane = threadIdx.x & 63;
  const int64_t units = (int64_t)T * chunks;
  for (int64_t u = blockIdx.x * (int64_t)ROW_WAVES + (threadIdx.x >> 6); u < units;
       u += (int64_t)gridDim.x * ROW_WAVES) {
    const int64_t t = u / chunks;
    const int c = ((int)(u - t * chunks) * 64 + lane) * VEC;
    if (c >= N) continue;
    float a[VEC] = {};
    for (int j = 0; j < k; ++j) {
      const int r = pair_row[t * k + j];
      if (r >= 0 && r < rows) {
        float v[VEC];
        load_vec<IBF16, VEC>(dxs, (int64_t)r * N + c, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) a[i] += v[i];
      }
    }
    store_vec<OBF16, VEC>(dx, t * N + c, a);
  }
}

// One wave per pair: dy[row] = w dout[t] and dweights[p] = <dout[t], y[row]>,
// summed in f32 (a lane's columns ascending, then the wave's lanes).
template <bool GBF16, bool YBF16, bool OBF16, int VEC>
__global__ __launch_bounds__(ROW_WAVES * 64) void combine_bwd_kernel(
    const void* __restrict__ dout, const void* __restrict__ y, const float* __restrict__ w,
    const int32_t* __restrict__ pair_row, int32_t T, int32_t k, int32_t N, int32_t rows, void* __restrict__ dy,
    float* __restrict__ dweights) {
  const int lane = threadIdx.x & 63;
  const int64_t pairs = (int64_t)T * k;
  for (int64_t p = blockIdx.x * (int64_t)ROW_WAVES + (threadIdx.x >> 6); p < pairs;
       p += (int64_t)gridDim.x * ROW_WAVES) {
    const int64_t t = p / k;
    const int r = pair_row[p];
    const bool live = r >= 0 && r < rows;
    float dot = 0.f;
    if (live) {
      const float wp = w[p];
      for (int c = lane * VEC; c < N; c += 64 * VEC) {
        float g[VEC], v[VEC];
        load_vec<GBF16, VEC>(dout, t * N + c, g);
        load_vec<YBF16, VEC>(y, (int64_t)r * N + c, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          dot = fmaf(g[i], v[i], dot);
          g[i] *= wp;
        }
        store_vec<OBF16, VEC>(dy, (int64_t)r * N + c, g);
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) dweights[p] = dot;
  }
}

// h[r, c] = silu(y[r, c]) * y[r, H + c] for the first *n_rows rows (all M
// where n_rows is NULL), silu(z) = z / (1 + e^-z).
template <bool IBF16, bool OBF16, int VEC>
__global__ __launch_bounds__(ROW_WAVES * 64) void silu_mul_kernel(const void* __restrict__ y, int32_t M, int32_t H,
                                                                  int32_t chunks, const int32_t* __restrict__ n_rows,
                                                                  void* __restrict__ h) {
  const int lane = threadIdx.x & 63;
  const int live = n_rows ? min(M, *n_rows) : M;
  const int64_t units = (int64_t)live * chunks;
  for (int64_t u = blockIdx.x * (int64_t)ROW_WAVES + (threadIdx.x >> 6); u < units;
       u += (int64_t)gridDim.x * ROW_WAVES) {
    const int64_t r = u / chunks;
    const int c = ((int)(u - r * chunks) * 64 + lane) * VEC;
    if (c >= H) continue;
    float g[VEC], v[VEC];
    load_vec<IBF16, VEC, true>(y, r * 2 * H + c, g);
    load_vec<IBF16, VEC, true>(y, r * 2 * H + H + c, v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = g[i] / (1.0f + __expf(-g[i])) * v[i];
    store_vec<OBF16, VEC>(h, r * H + c, g);
  }
}

static unsigned row_grid(int64_t units) {
  const int64_t g = (units + ROW_WAVES - 1) / ROW_WAVES;
  return (unsigned)(g < ROW_GRID_CAP ? g : ROW_GRID_CAP);
}

// Calls f with v as a compile-time constant.
template <typename F>
static void with_bool(bool v, F f) {
  if (v) f(std::true_type{});
  else f(std::false_type{});
}

hipError_t launch_dispatch(const void* x, int bf16, const int32_t* pair_row, int32_t T, int32_t k, int32_t N,
                           int32_t rows, void* xs, hipStream_t stream) {
  const int64_t bytes = (int64_t)N * (bf16 ? 2 : 4);
  const bool wide = bytes % 16 == 0;
  const int32_t cols = (int32_t)(bytes / (wide ? 16 : 8)), chunks = (cols + 63) / 64;
  const dim3 grid(row_grid((int64_t)T * chunks)), block(ROW_WAVES * 64);
  if (wide)
    hipLaunchKernelGGL(dispatch_kernel<u32x4_t>, grid, block, 0, stream, reinterpret_cast<const u32x4_t*>(x),
                       pair_row, T, k, cols, chunks, rows, reinterpret_cast<u32x4_t*>(xs));
  else
    hipLaunchKernelGGL(dispatch_kernel<uint64_t>, grid, block, 0, stream, reinterpret_cast<const uint64_t*>(x),
                       pair_row, T, k, cols, chunks, rows, reinterpret_cast<uint64_t*>(xs));
  return hipGetLastError();
}

hipError_t launch_dispatch_bwd(const void* dxs, int in_bf16, const int32_t* pair_row, int32_t T, int32_t k, int32_t N,
                               int32_t rows, void* dx, int out_bf16, hipStream_t stream) {
  with_bool(in_bf16, [&](auto ib) { with_bool(out_bf16, [&](auto ob) { with_bool(N % 8 == 0, [&](auto wide) {
    constexpr int VEC = decltype(wide)::value ? 8 : 4;
    const int32_t chunks = (N + 64 * VEC - 1) / (64 * VEC);
    hipLaunchKernelGGL((dispatch_bwd_kernel<decltype(ib)::value, decltype(ob)::value, VEC>),
                       dim3(row_grid((int64_t)T * chunks)), dim3(ROW_WAVES * 64), 0, stream, dxs, pair_row, T, k, N,
                       chunks, rows, dx);
  }); }); });
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const void* dout, int dout_bf16, const void* y, int y_bf16, const float* w,
                              const int32_t* pair_row, int32_t T, int32_t k, int32_t N, int32_t rows, void* dy,
                              int dy_bf16, float* dweights, hipStream_t stream) {
  with_bool(dout_bf16, [&](auto gb) { with_bool(y_bf16, [&](auto yb) { with_bool(dy_bf16, [&](auto ob) {
    with_bool(N % 8 == 0, [&](auto wide) {
      constexpr int VEC = decltype(wide)::value ? 8 : 4;
      hipLaunchKernelGGL((combine_bwd_kernel<decltype(gb)::value, decltype(yb)::value, decltype(ob)::value, VEC>),
                         dim3(row_grid((int64_t)T * k)), dim3(ROW_WAVES * 64), 0, stream, dout, y, w, pair_row, T, k,
                         N, rows, dy, dweights);
    });
  }); }); });
  return hipGetLastError();
}

hipError_t launch_silu_mul(const void* y, int y_bf16, int32_t M, int32_t N, const int32_t* n_rows, void* h,
                           int h_bf16, hipStream_t stream) {
  const int32_t H = N / 2;
  with_bool(y_bf16, [&](auto ib) { with_bool(h_bf16, [&](auto ob) { with_bool(H % 8 == 0, [&](auto wide) {
    constexpr int VEC = decltype(wide)::value ? 8 : 4;
    const int32_t chunks = (H + 64 * VEC - 1) / (64 * VEC);
    hipLaunchKernelGGL((silu_mul_kernel<decltype(ib)::value, decltype(ob)::value, VEC>),
                       dim3(row_grid((int64_t)M * chunks)), dim3(ROW_WAVES * 64), 0, stream, y, M, H, chunks, n_rows,
                       h);
  }); }); });
  return hipGetLastError();
}

}  // namespace moe
