// Wave-wide (64-lane) reductions and small conversions for the row kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "common.h"

namespace moe {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two f32 as a word of two bf16 (a in the low half), round to nearest even: one
// v_cvt_pk_bf16_f32 (the integer rounding cost w2's gradient at 4,096 tokens
// 20 of 481 us).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

// v of the lane that the DPP control CTRL names; `other` in lanes that have no
// such source or whose row ROWS leaves out.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or(uint32_t other, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)other, (int)v, CTRL, ROWS, 0xF, false);
}

// v of the lane that the DPP control CTRL names, where every lane has one.
template <int CTRL>
__device__ __forceinline__ float dpp_from(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or(float other, float v) {
  return __uint_as_float(dpp_or<CTRL, ROWS>(__float_as_uint(other), __float_as_uint(v)));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or(double other, double v) {
  const uint64_t o = (uint64_t)__double_as_longlong(other), u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = dpp_or<CTRL, ROWS>((uint32_t)o, (uint32_t)u);
  const uint32_t hi = dpp_or<CTRL, ROWS>((uint32_t)(o >> 32), (uint32_t)(u >> 32));
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

__device__ __forceinline__ int read_lane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float read_lane(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// Reductions over the wave's 64 lanes, every lane active; the result is
// uniform.  row_shr 1, 2, 4, 8 gather a row of 16 lanes in its last lane,
// row_bcast 15 and 31 carry rows 0 -> 1, 2 -> 3, then 1 -> 2, 3; lane 63 holds
// the whole.  A fixed order, so a sum is the same on every call.
template <typename V>
__device__ __forceinline__ V wave_max(V v) {
  V o;
#define MOE_STEP(CTRL, ROWS) o = dpp_or<CTRL, ROWS>(v, v); v = o > v ? o : v;
  MOE_STEP(0x111, 0xF) MOE_STEP(0x112, 0xF) MOE_STEP(0x114, 0xF) MOE_STEP(0x118, 0xF)
  MOE_STEP(0x142, 0xA) MOE_STEP(0x143, 0xC)
#undef MOE_STEP
  return read_lane(v, 63);
}

// The same for unsigned integers, where 0 stands in for a lane without a
// source and each step folds into one v_max_u32.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#define MOE_STEP(CTRL, ROWS) v = max(v, dpp_or<CTRL, ROWS>(0u, v));
  MOE_STEP(0x111, 0xF) MOE_STEP(0x112, 0xF) MOE_STEP(0x114, 0xF) MOE_STEP(0x118, 0xF)
  MOE_STEP(0x142, 0xA) MOE_STEP(0x143, 0xC)
#undef MOE_STEP
  return (uint32_t)read_lane((int)v, 63);
}

template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#define MOE_STEP(CTRL, ROWS) v += dpp_or<CTRL, ROWS>(V(0), v);
  MOE_STEP(0x111, 0xF) MOE_STEP(0x112, 0xF) MOE_STEP(0x114, 0xF) MOE_STEP(0x118, 0xF)
  MOE_STEP(0x142, 0xA) MOE_STEP(0x143, 0xC)
#undef MOE_STEP
  return read_lane(v, 63);
}

}  // namespace moe
