// Device code shared by the 4-bit products and the cache's kernels: loads from memory straight to
// LDS, waits for them, and a rounding to bf16 that keeps NaN.
#pragma once

#include "wq_device.h"

namespace wq {

typedef __attribute__((address_space(3))) uint8_t* lds_ptr_u8;

// One DMA instruction of 64 lanes to LDS byte address `la` on, 16 bytes a lane (dma16), a dword
// (dma4) or a byte widened to a dword (dma1_at), from a wave-uniform base and a lane offset or
// (.._at) from an address a lane.  Written out, with its LDS address in M0: given the builtin, the
// compiler lets LDS reads that it cannot tell from the target wait for every DMA in flight.  The
// kernels order them themselves (vmcnt, then a barrier).  Nothing is loaded into registers.  Six
// wait states stand in front of the load: a base just written by the VALU needs five, M0 one.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t la) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(la) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t la) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(la) : "memory", "m0");
}
__device__ __forceinline__ void dma16_at(const void* at, uint32_t la) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(at), "s"(la) : "memory", "m0");
}
__device__ __forceinline__ void dma4_at(const void* at, uint32_t la) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dword %0, off" ::"v"(at), "s"(la) : "memory", "m0");
}
__device__ __forceinline__ void dma1_at(const void* at, uint32_t la) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_ubyte %0, off" ::"v"(at), "s"(la) : "memory", "m0");
}
#pragma clang diagnostic pop

// at most N of the wave's vector memory operations are still in flight
template <int N>
__device__ __forceinline__ void wait_vm() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// f32 -> bf16 bits, round to nearest even, any input: a NaN stays one (v_cvt_pk_bf16_f32)
__device__ __forceinline__ uint32_t f32_to_bf16_nan(float f) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
}

}  // namespace wq
