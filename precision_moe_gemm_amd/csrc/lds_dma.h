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
// program, so the block holds them itself.  The load comes one state after the write of M0,
// from which it takes its LDS address.  It comes five states after a vector instruction that
// writes a scalar register of `base`: where the compiler runs out of scalar registers and
// reads bases back from lanes of a vector register (v_readlane), the caller asks for NOP = 3,
// which with s_mov makes five.  Elsewhere NOP is 0; a test of the built code looks for vector
// writes that come too close.  (Five states everywhere: 1158 us for 1104 in the FP8 product
// of 8192^3 with FP32 outputs, 1 to 3 % in the others; nothing in the NVFP4 products.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int NOP = 0>
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop %3\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "s"(lds), "v"(voff), "s"(base), "n"(NOP) : "memory", "m0");
}
template <int NOP = 0>
__device__ __forceinline__ void lds_dma4(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop %3\n\tglobal_load_lds_dword %1, %2"
               :: "s"(lds), "v"(voff), "s"(base), "n"(NOP) : "memory", "m0");
}
__device__ __forceinline__ void lds_dma16(const void* p, uint32_t lds) {   // each lane's own 64-bit address
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" :: "s"(lds), "v"(p) : "memory", "m0");
}
#pragma clang diagnostic pop
template <int NOP = 0>
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t voff, const uint8_t* lds) {
  lds_dma16<NOP>(base, voff, lds_addr(lds));
}
template <int NOP = 0>
__device__ __forceinline__ void lds_dma4(const void* base, uint32_t voff, const uint8_t* lds) {
  lds_dma4<NOP>(base, voff, lds_addr(lds));
}

// A barrier that orders LDS accesses alone: loads and stores to memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace nvfp4moe
