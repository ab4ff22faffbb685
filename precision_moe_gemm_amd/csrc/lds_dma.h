// Direct-to-LDS loads and the workgroup barrier that goes with them.
#pragma once

#include "common.h"

namespace nvfp4moe {

typedef __attribute__((address_space(3))) void lds_void;

// LDS byte address of a wave-uniform pointer into LDS
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void*)p);
}

// Each lane's 16 (or 4) bytes at base + voff land at lds + 16 (4) * lane.  Issued through
// inline assembly so that the compiler, which cannot tell which LDS bytes such a load
// writes, does not make every later LDS read wait for all of them; a kernel waits itself
// (vmcnt) before the barrier that publishes a stage.  The compiler does not count these
// loads, so its own vmcnt waits only become stricter.
//
// Nor does it look into the assembly for the wait states that the hardware asks of the
// program, so the block holds them itself: one between the write of M0 and the load that
// takes its LDS address from it, and five between a vector instruction that may have
// written `base` just before (v_readfirstlane, v_readlane) and the load that reads it.
// s_mov is the first of the five, s_nop 3 the other four.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
#define LDS_DMA(LOAD) "s_mov_b32 m0, %0\n\ts_nop 3\n\t" LOAD
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile(LDS_DMA("global_load_lds_dwordx4 %1, %2") :: "s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void lds_dma4(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile(LDS_DMA("global_load_lds_dword %1, %2") :: "s"(lds), "v"(voff), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void lds_dma16(const void* p, uint32_t lds) {   // each lane's own 64-bit address
  asm volatile(LDS_DMA("global_load_lds_dwordx4 %1, off") :: "s"(lds), "v"(p) : "memory", "m0");
}
#undef LDS_DMA
#pragma clang diagnostic pop
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t voff, const uint8_t* lds) {
  lds_dma16(base, voff, lds_addr(lds));
}
__device__ __forceinline__ void lds_dma4(const void* base, uint32_t voff, const uint8_t* lds) {
  lds_dma4(base, voff, lds_addr(lds));
}

// A barrier that orders LDS accesses alone: loads and stores to memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace nvfp4moe
