// lds_dma.cuh -- LDS-direct loads: memory to LDS without a register in between.
// The LDS behind them is dynamic shared memory (an external array): the
// compiler must not conclude that nothing writes it.
#pragma once

#include "common.cuh"

namespace ssmvjp {

typedef __attribute__((address_space(3))) char lds_char;
// raw buffer resource words (the form make_rsrc builds), made wave-uniform so
// that they sit in scalar registers
__device__ __forceinline__ u32x4 rsrc_words_u(const void* base, unsigned bytes) {
  const unsigned long long p = (unsigned long long)base;
  u32x4 r;
  r[0] = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)p);
  r[1] = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)(p >> 32)) & 0xffffu;
  r[2] = (unsigned)__builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000u;
  return r;
}
// LDS-direct loads (each lane's 4 or 16 bytes written to LDS at M0 + the
// lane's slot), issued as assembly: the compiler neither counts them nor, as
// it does for its own LDS-direct loads, waits for every outstanding load
// before the next transposed LDS read.  The caller waits with vmcnt before the
// barrier that publishes the data.  M0 is named as clobbered; the compiler
// uses it for nothing else around them (it keeps no value there across these
// statements), so its warning about clobbering a reserved register is muted.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma_dword(unsigned lds_addr, unsigned off, u32x4 rs) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds_addr), "v"(off), "s"(rs)
               : "memory", "m0");
}
__device__ __forceinline__ void dma_dwordx4(unsigned lds_addr, unsigned off, u32x4 rs) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds_addr), "v"(off), "s"(rs)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// the wave's LDS-direct loads (and its other memory operations) are complete
__device__ __forceinline__ void dma_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ unsigned lds_base(const void* smem) {
  return (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)(unsigned long long)(lds_char*)smem);
}

}  // namespace ssmvjp
