// Loads straight into LDS and the barrier that leaves them in flight, for the dense products
// (dense_i8.hip, dense_few.hip).  gemm_tiled.hip holds its own: its counter summaries are tied to its text.
#pragma once

#include "common.hpp"

namespace w4a8 {

// Workgroup barrier that leaves direct-to-LDS loads in flight (__syncthreads'
// release fence would wait for all of them).  The caller waits for what the
// other waves need; the empty asm statements keep the compiler from moving
// memory accesses across.
__device__ __forceinline__ void barrier_loads_in_flight() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// buffer resource of a byte range (gfx9 dword 3: raw, untyped access)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
// LDS byte address of a pointer into a __shared__ variable
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
// Direct loads into LDS: lane l's bytes (at rsrc + voff + soff) go to lds + size * l
// (M0 holds the wave's LDS base).  They are issued from inline assembly, which the
// compiler does not see as writing LDS: given the builtin, its wait insertion cannot
// always tell the ring slot being filled from the one being read, and adds a full
// vmcnt(0) before the group's LDS reads, which drains the prefetch.  The kernel orders
// these loads itself: its own vmcnt waits, then the barrier, before any wave reads
// the slot.  They write no register, so nothing the compiler allocates is in flight.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, void* lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds_addr(lds)), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
}
// the same of bytes that are read once
__device__ __forceinline__ void dma16_nt(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, void* lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
               :: "s"(lds_addr(lds)), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, void* lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :: "s"(lds_addr(lds)), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
}

template <typename T>
__device__ __forceinline__ T lds_load(const void* p) {
  return *reinterpret_cast<const T*>(__builtin_assume_aligned(p, 16));
}

}  // namespace w4a8
