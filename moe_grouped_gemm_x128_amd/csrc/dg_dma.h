// dg_dma.h -- loads from memory straight into LDS through buffer resources,
// and the waits that go with them (device code of the linear layer's and the MoE layer's kernels).
//
// Lane i's 16 bytes land at LDS address lds + 16 i; bytes at or past the
// resource's range read as zero and touch no memory.  Issued through inline
// asm so that the compiler's wait insertion does not make every LDS read wait
// for every load in flight: the waits are the explicit ones below.  The asm
// has no register outputs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {
namespace dma {

typedef int v4i __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// Raw buffer resource over [base, base + bytes), wave-uniform.
__device__ __forceinline__ v4i resource(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)base;
  return v4i{(int)__builtin_amdgcn_readfirstlane((uint32_t)b),
             (int)(__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) & 0xffffu),
             (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load16(uint32_t lds, v4i rsrc, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(voff), "s"(rsrc) : "memory", "m0");
}
// The same for data that is read once (nontemporal cache policy).
__device__ __forceinline__ void load16_nt(uint32_t lds, v4i rsrc, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
               :: "s"(lds), "v"(voff), "s"(rsrc) : "memory", "m0");
}
// 4 bytes per lane, to lds + 4 i.
__device__ __forceinline__ void load4(uint32_t lds, v4i rsrc, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(lds), "v"(voff), "s"(rsrc) : "memory", "m0");
}
#pragma clang diagnostic pop

// This wave's LDS reads have returned (before their place is loaded anew).
__device__ __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// At most N vector-memory operations of this wave in flight.
template <int N>
__device__ __forceinline__ void wait() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

// Workgroup barrier behind this wave's LDS reads and writes.
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

}  // namespace dma
}  // namespace dg
