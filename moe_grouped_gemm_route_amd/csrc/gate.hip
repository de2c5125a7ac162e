// moe_topk_gate / moe_topk_gate_bwd: the router's top-k choice and weights,
// and their gradient.
//
// One wave per token; lane l holds experts l, l + 64, l + 128, ...  The k
// choices are k rounds of "largest key over the wave, lowest index among
// equals": the keys are unsigned integers in the order of the values, the
// maximum is one DPP reduction of six instructions, and because a slot's 64
// experts are consecutive, the lowest index is the first set bit of the first
// non-empty ballot of (key == maximum), slot by slot.  No shuffle of indices
// and no LDS.
//
// Keys.  Without a bias the scores rise with the logits, so the keys are the
// logits themselves and the choice is exact.  With a bias the key is
// score + bias, where two experts can come within an f32 rounding of each
// other; those keys are computed in f64, so the choice does not hang on the
// last bit of an exponential (at 4,096 tokens x 256 experts f32 keys would
// put a pair in another order about once a batch).
//
// Weights are f32.  A renormalised weight is s_j / sum s over the chosen,
// with s scaled by a common factor so that the largest chosen score cannot
// underflow: softmax subtracts the largest chosen logit; for the sigmoid,
//     sigma(l) = e^min(l, 0) / (1 + e^-|l|),
// and the largest chosen min(l, 0) is subtracted in that exponent.
//
// Bound by latency: at 4,096 tokens x 256 experts top-6 the f32 logits are 4
// MB, under a microsecond of HBM; the kernel takes 5.2 us (k rounds of a
// 64-lane reduction one after the other), 9.0 with a bias (f64 exponentials),
// the gradient 4.6, or 6.1 where every expert has one (softmax, not
// renormalised); a call from Python takes 8.1 to 9.9, bound by the host.  At
// 16,384 tokens x 1,024 experts top-16 (67 MB, 13 us at the copy rate): 33 us,
// the instructions of 16 rounds of which each serves one token, and the
// gradient 17 (134 MB).
#include "common.h"
#include "launch.h"
#include "wave.h"

namespace moe {

constexpr int GATE_WAVES = 4;   // tokens per workgroup

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* __restrict__ logits, int64_t i) {
  if (BF16) return bf16_lo(reinterpret_cast<const uint16_t*>(logits)[i]);
  return reinterpret_cast<const float*>(logits)[i];
}

// A row's logits, NaN and places past E as -inf (masked).
template <int VPL, bool BF16>
__device__ __forceinline__ void load_row(const void* __restrict__ logits, int64_t t, int E, float (&x)[VPL]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    x[i] = -INFINITY;
    if (e < E) {
      const float v = load_logit<BF16>(logits, t * E + e);
      if (v == v) x[i] = v;
    }
  }
}

// e^(x - m), 1 at x = m (infinities included), 0 for a masked x.
__device__ __forceinline__ float exp_below(float x, float m) { return x == m && x > -INFINITY ? 1.f : x > -INFINITY ? expf(x - m) : 0.f; }

template <int VPL>
__device__ __forceinline__ float row_max(const float (&x)[VPL]) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = fmaxf(m, x[i]);
  return wave_max(m);
}

template <int VPL>
__device__ __forceinline__ float row_exp_sum(const float (&x)[VPL], float m) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) s += exp_below(x[i], m);
  return wave_sum(s);
}

// The unscaled weights of lanes j < k from the chosen logits (-inf in lanes
// whose slot chose nothing, and in lanes >= k): softmax (score 0) or sigmoid
// (1), over the chosen (renorm) or as they are.  m and z: the row's largest
// logit and sum of exponentials (softmax without renorm only).
__device__ __forceinline__ float chosen_weight(float l, int score, int renorm, float m, float z) {
  const bool live = l > -INFINITY;
  if (score == 0) {
    if (renorm) {
      m = wave_max(l);
      const float s = exp_below(l, m);
      z = wave_sum(s);
      return live ? s / z : 0.f;
    }
    return live ? exp_below(l, m) / z : 0.f;
  }
  const float low = fminf(l, 0.f);
  const float ref = renorm ? wave_max(low) : 0.f;
  const float s = live ? expf(low - (ref > -INFINITY ? ref : 0.f)) / (1.f + expf(-fabsf(l))) : 0.f;
  if (!renorm) return s;
  z = wave_sum(s);
  return live ? s / z : 0.f;
}

// Unsigned keys in the order of the values, 0 for a masked one (below the key
// of every other value); -0 as +0, so that they tie.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return x > -INFINITY ? u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ float order_value(uint32_t key) {
  return key == 0 ? -INFINITY : __uint_as_float(key ^ ((key >> 31) != 0 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return x > -(double)INFINITY ? u ^ ((uint64_t)((int64_t)u >> 63) | (1ull << 63)) : 0ull;
}

// BIAS: the keys are score + bias in f64 (64-bit keys in two words, the high
// one compared first); else the logits.
template <int VPL, bool BF16, bool BIAS>
__global__ __launch_bounds__(GATE_WAVES * 64) void gate_kernel(const void* __restrict__ logits,
                                                               const float* __restrict__ bias, int32_t T, int32_t E,
                                                               int32_t k, int score, int renorm, float scale,
                                                               int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.x * (int64_t)GATE_WAVES + (threadIdx.x >> 6);
  if (t >= T) return;
  float x[VPL];
  load_row<VPL, BF16>(logits, t, E, x);
  float m = -INFINITY, z = 0.f;
  if (score == 0 && !renorm) {
    m = row_max(x);
    z = row_exp_sum(x, m);
  }
  uint32_t hi[VPL], lo[BIAS ? VPL : 1];
  if constexpr (BIAS) {
    double zd = 0.0, p[VPL];
    if (score == 0) {
      const double md = (double)row_max(x);
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        p[i] = x[i] > -INFINITY ? ((double)x[i] == md ? 1.0 : exp((double)x[i] - md)) : 0.0;
        zd += p[i];
      }
      zd = wave_sum(zd);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 64 + lane;
      const double s = score == 0 ? p[i] / zd : 1.0 / (1.0 + exp(-(double)x[i]));
      // a NaN bias compares false in order_key and masks its expert
      const uint64_t key = x[i] > -INFINITY ? order_key(s + (double)bias[e]) : 0ull;
      hi[i] = (uint32_t)(key >> 32);
      lo[i] = (uint32_t)key;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) hi[i] = order_key(x[i]);
  }

  // Each lane keeps the largest key of every GR of its registers (and among
  // equal high words the largest low one), so that a round looks at one group
  // only: the one that holds the chosen key (1,024 experts top-16: 55 -> 33 us; up
  // to 256 experts there is one group and nothing changes).  q0 and e are the same
  // in every lane, so the branches on them are scalar.
  constexpr int GR = VPL < 4 ? VPL : 4, GROUPS = VPL / GR;
  uint32_t top[GROUPS], top_lo[BIAS ? GROUPS : 1];
  auto find_top = [&](int q) __attribute__((always_inline)) {
    uint32_t h = hi[q * GR], l = 0;
#pragma unroll
    for (int i = 1; i < GR; ++i) h = max(h, hi[q * GR + i]);
    top[q] = h;
    if constexpr (BIAS) {
#pragma unroll
      for (int i = 0; i < GR; ++i) l = max(l, hi[q * GR + i] == h ? lo[q * GR + i] : 0u);
      top_lo[q] = l;
    }
  };
#pragma unroll
  for (int q = 0; q < GROUPS; ++q) find_top(q);

  int my_id = -1;
  uint32_t my_key = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = top[0], low = 0;
#pragma unroll
    for (int q = 1; q < GROUPS; ++q) best = max(best, top[q]);
    best = wave_max_u32(best);
    if (best == 0) break;   // uniform: nothing is left to choose
    if constexpr (BIAS) {
#pragma unroll
      for (int q = 0; q < GROUPS; ++q) low = max(low, top[q] == best ? top_lo[q] : 0u);
      low = wave_max_u32(low);
    }
    int q0 = GROUPS - 1;                       // the lowest group that holds the key
#pragma unroll
    for (int q = GROUPS - 2; q >= 0; --q) {
      bool is = top[q] == best;
      if constexpr (BIAS) is = is && top_lo[q] == low;
      if (__ballot(is) != 0) q0 = q;
    }
    int e = 0;
#pragma unroll
    for (int q = 0; q < GROUPS; ++q) {
      if (q != q0) continue;
#pragma unroll
      for (int i = (q + 1) * GR - 1; i >= q * GR; --i) {
        bool is = hi[i] == best;
        if constexpr (BIAS) is = is && lo[i] == low;
        const uint64_t hit = __ballot(is);
        if (hit != 0) e = i * 64 + __ffsll((unsigned long long)hit) - 1;
      }
#pragma unroll
      for (int i = q * GR; i < (q + 1) * GR; ++i) hi[i] = e == i * 64 + lane ? 0u : hi[i];
      find_top(q);
    }
    if (lane == j) {
      my_id = e;
      my_key = best;
    }
  }
  float my_logit;
  if constexpr (BIAS) my_logit = my_id >= 0 ? load_logit<BF16>(logits, t * E + my_id) : -INFINITY;
  else my_logit = order_value(my_key);
  const float w = chosen_weight(my_logit, score, renorm, m, z);
  if (lane < k) {
    ids[t * k + lane] = my_id;
    weights[t * k + lane] = w * scale;
  }
}

// Between LDS writes of a wave's lanes and reads of them by other lanes of the
// wave.  The hardware runs one wave's LDS operations in order; the fences keep
// the compiler from handing a lane's own store on to its later load, past what
// another lane wrote in between (a wave barrier alone orders no memory).
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// dlogits of one token: lane j < k computes the gradient that reaches the
// logit of its slot; slots of one expert (a repeated id) are added up in slot
// order by the first of them, which adds the sum to the expert's place in the
// row.  The row is put together in LDS: with every lane testing every slot
// against its own experts instead, 16,384 tokens x 1,024 experts top-16 took
// 33 us.
template <int VPL, bool BF16>
__global__ __launch_bounds__(GATE_WAVES * 64) void gate_bwd_kernel(const void* __restrict__ logits,
                                                                   const int32_t* __restrict__ ids,
                                                                   const float* __restrict__ dweights, int32_t T,
                                                                   int32_t E, int32_t k, int score, int renorm,
                                                                   float scale, void* __restrict__ dlogits) {
  __shared__ float s_row[GATE_WAVES][VPL * 64];
  const int lane = threadIdx.x & 63;
  const int64_t t = blockIdx.x * (int64_t)GATE_WAVES + (threadIdx.x >> 6);
  if (t >= T) return;
  int id = -1;
  float g = 0.f, l = -INFINITY;
  if (lane < k) {
    id = ids[t * k + lane];
    if (id < 0 || id >= E) id = -1;
    if (id >= 0) {
      g = dweights[t * k + lane] * scale;
      const float v = load_logit<BF16>(logits, t * E + id);
      if (v == v) l = v;
    }
  }
  const bool dense = score == 0 && !renorm;
  float p[VPL];              // the row's exponentials (dense), masked ones 0
  float m = -INFINITY, z = 0.f;
  if (dense) {
    load_row<VPL, BF16>(logits, t, E, p);
    m = row_max(p);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = exp_below(p[i], m);
      z += p[i];
    }
    z = wave_sum(z);
  }
  const float w = chosen_weight(l, score, renorm, m, z);
  // a slot that chose nothing (or a masked expert) has weight 0 whatever its
  // logits, so nothing flows back through it
  const bool live = l > -INFINITY;
  const float gl = live ? g : 0.f;
  const float mean = score == 0 || renorm ? wave_sum(gl * w) : 0.f;
  float d = live ? w * (gl - (dense ? 0.f : mean)) : 0.f;
  if (score == 1 && live) d *= l >= 0.f ? expf(-l) / (1.f + expf(-l)) : 1.f / (1.f + expf(l));   // 1 - sigma
  float total = 0.f;
  bool first = id >= 0;
  for (int j = 0; j < k; ++j) {
    const bool same = read_lane(id, j) == id;
    if (same) total += read_lane(d, j);
    if (same && j < lane) first = false;
  }
  float* row = s_row[threadIdx.x >> 6];
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    row[i * 64 + lane] = dense && p[i] > 0.f ? -mean * (p[i] / z) : 0.f;
  wave_lds_sync();
  if (first) row[id] += total;
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    const float a = row[e];
    if (e < E) {
      if (BF16) reinterpret_cast<uint16_t*>(dlogits)[t * E + e] = f32_to_bf16_rne(a);
      else reinterpret_cast<float*>(dlogits)[t * E + e] = a;
    }
  }
}

// Calls f with the logits per lane, rounded up to the built sizes.
template <typename F>
static void for_vpl(int32_t E, F f) {
  if (E <= 64) f(std::integral_constant<int, 1>{});
  else if (E <= 128) f(std::integral_constant<int, 2>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}

hipError_t launch_topk_gate(const void* logits, int bf16, const float* bias, int32_t T, int32_t E, int32_t k,
                            int score, int renorm, float scale, int32_t* ids, float* weights, hipStream_t stream) {
  const dim3 grid((unsigned)((T + GATE_WAVES - 1) / GATE_WAVES)), block(GATE_WAVES * 64);
  for_vpl(E, [&](auto v) {
    constexpr int VPL = decltype(v)::value;
    if (bf16) {
      if (bias) hipLaunchKernelGGL((gate_kernel<VPL, true, true>), grid, block, 0, stream, logits, bias, T, E, k, score, renorm, scale, ids, weights);
      else hipLaunchKernelGGL((gate_kernel<VPL, true, false>), grid, block, 0, stream, logits, bias, T, E, k, score, renorm, scale, ids, weights);
    } else {
      if (bias) hipLaunchKernelGGL((gate_kernel<VPL, false, true>), grid, block, 0, stream, logits, bias, T, E, k, score, renorm, scale, ids, weights);
      else hipLaunchKernelGGL((gate_kernel<VPL, false, false>), grid, block, 0, stream, logits, bias, T, E, k, score, renorm, scale, ids, weights);
    }
  });
  return hipGetLastError();
}

hipError_t launch_topk_gate_bwd(const void* logits, int bf16, const int32_t* ids, const float* dweights, int32_t T,
                                int32_t E, int32_t k, int score, int renorm, float scale, void* dlogits,
                                hipStream_t stream) {
  const dim3 grid((unsigned)((T + GATE_WAVES - 1) / GATE_WAVES)), block(GATE_WAVES * 64);
  for_vpl(E, [&](auto v) {
    constexpr int VPL = decltype(v)::value;
    if (bf16) hipLaunchKernelGGL((gate_bwd_kernel<VPL, true>), grid, block, 0, stream, logits, ids, dweights, T, E, k, score, renorm, scale, dlogits);
    else hipLaunchKernelGGL((gate_bwd_kernel<VPL, false>), grid, block, 0, stream, logits, ids, dweights, T, E, k, score, renorm, scale, dlogits);
  });
  return hipGetLastError();
}

}  // namespace moe
