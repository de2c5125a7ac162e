// Direct-to-LDS loads and the waits around them, for the kernels that stage
// their operands in LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace moe {

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

// Ends a stage: this wave's LDS operations are done, then the workgroup
// barrier.  Vector loads are vm_wait's.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((63 & 15) | ((63 >> 4) << 14) | (7 << 4));   // vmcnt 63, expcnt 7, lgkmcnt 0
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace moe
