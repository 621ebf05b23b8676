// Direct global -> LDS loads with explicit ordering, shared by the GEMM kernels.
#pragma once

#include "device_common.h"

namespace megamoe {

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// Direct global -> LDS loads.  Issued through inline assembly so that the compiler does not track
// them as LDS writes (it would otherwise wait for every outstanding load before any LDS read it
// cannot prove disjoint, draining the prefetch each stage).  Their ordering is explicit instead:
// wait_vmcnt() for this wave's loads, then s_barrier for everyone's.  The compiler's own vmcnt
// waits stay correct because loads retire in order.  Nothing else in these kernels uses M0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // M0 is written only here (checked in the ISA)
__device__ __forceinline__ uint32_t lds_addr(const uint8_t* p) {
  return (uint32_t)(uintptr_t)(const lds_u8*)p;
}
__device__ __forceinline__ void dma16(const uint8_t* src, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);  // wave-uniform; must live in an SGPR for M0
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
// The same with the non-temporal hint: for bytes read once per call (the 16-row kernels' weight
// scales when they stream the packed codes).
__device__ __forceinline__ void dma16nt(const uint8_t* src, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" ::"s"(lds), "v"(src) : "memory", "m0");
}
// The same from a wave-uniform base and a 32-bit lane offset, without and with the non-temporal hint.
__device__ __forceinline__ uint64_t scalar_addr(const uint8_t* base) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b) |
         (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)) << 32;
}
__device__ __forceinline__ void dma16s(const uint8_t* base, uint32_t off, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off),
               "s"(scalar_addr(base))
               : "memory", "m0");
}
__device__ __forceinline__ void dma16snt(const uint8_t* base, uint32_t off, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(lds), "v"(off),
               "s"(scalar_addr(base))
               : "memory", "m0");
}
__device__ __forceinline__ void dma4(const uint8_t* src, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(src) : "memory", "m0");
}
#pragma clang diagnostic pop

// s_waitcnt vmcnt(n), other counters unconstrained (gfx9 encoding: vmcnt bits 3:0 and 15:14).
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

}  // namespace megamoe
