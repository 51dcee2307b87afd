// Device pieces of the LDS rings that the prefill GEMMs keep: scalar loads of
// read-only tables, direct global -> LDS loads and the per-stage wait.
#pragma once

#include "internal.h"

namespace moe355 {

// A load of memory that no kernel of the launch writes (the tile plan, the
// bucket offsets) through the constant address space: at a wavefront-uniform
// address the compiler makes it a scalar load, whose wait (lgkmcnt) does not
// also wait for the vector-memory stores and direct loads in flight.
template <typename T>
__device__ __forceinline__ T ld_const(const T* q) {
    typedef const __attribute__((address_space(4))) T* ConstPtr;
    return *(ConstPtr)(q);
}

// A wavefront-uniform pointer held in scalar registers.
__device__ __forceinline__ const void* uniform_ptr(const void* q) {
    const uint64_t v = reinterpret_cast<uint64_t>(q);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return reinterpret_cast<const void*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// Direct loads of base + voff (32-bit byte offset, per lane) into LDS at lds;
// base and lds are wavefront-uniform.
__device__ __forceinline__ void dma16(const void* base, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(voff), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                 :: "v"(voff), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}

// Wait until at most N of this wavefront's loads are in flight and its LDS reads
// are done, then meet the other wavefronts.
template <int N>
__device__ __forceinline__ void stage_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void* q) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q));
}

}  // namespace moe355
