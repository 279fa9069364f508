// Direct-to-LDS loads of the BF16 and 4-bit products: buffer descriptors, the loads, and their waits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mgs {

typedef int sdesc_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds8;

constexpr uint32_t OUT = 0x80000000u;  // past every record count: reads zeros, without a memory access

// Raw buffer descriptor of `bytes` bytes at `p` (record count capped at 2^31 - 1) in scalar registers.  A descriptor
// that a VALU instruction has just written there needs five wait states before a load reads it, and the compiler
// does not see the loads below: desc_final() stands between.
__device__ __forceinline__ sdesc_t view(const uint8_t* p, int64_t bytes) {
  bytes = bytes < 0 ? 0 : (bytes > 0x7FFFFFFFll ? 0x7FFFFFFFll : bytes);
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  const int n = __builtin_amdgcn_readfirstlane((int)bytes);
  return sdesc_t{(int)lo, (int)(hi & 0xffffu), n, 0x00020000};
}
__device__ __forceinline__ void desc_final(const sdesc_t& d) { asm volatile("s_nop 4" ::"s"(d)); }

// Direct-to-LDS load of 16 (or 4) bytes per lane to LDS byte address `lds` + 16 (or 4) x lane, in inline assembly: the
// compiler would otherwise make later LDS reads wait for it.  It does not count it either; every wait is an
// explicit one.  The whole offset is in the lanes', so that the record count bounds it.
__device__ __forceinline__ void dma16(const sdesc_t& d, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :: "v"(voff), "s"(d), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}
__device__ __forceinline__ void dma4(const sdesc_t& d, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :: "v"(voff), "s"(d), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

}  // namespace mgs
