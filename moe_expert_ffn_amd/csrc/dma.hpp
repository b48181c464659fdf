// Asynchronous copies from global memory to LDS, and the waits on them.
#pragma once

#include "common.hpp"

namespace megamoe {

// The DMA copies are issued from inline assembly, so the compiler's wait-count
// pass does not see them and cannot serialise the ring (it would otherwise
// wait for every outstanding copy before any LDS read).  The waits on them are
// explicit.  Vector-memory operations complete in issue order, so the
// compiler's own waits for its loads stay correct, but they also wait for
// every copy issued before those loads.  A spill reload placed between a
// tile's copies and its K loop, or inside the loop, therefore drains the
// ring; in the 256-row kernel (all 128 registers in use) the reloads sit
// after each tile's K loop, and edits that moved them cost 3-12%.
template <int n>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(n >= 0 && n < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}

// One 16-byte chunk per lane, global -> LDS; lane i writes LDS bytes
// [lds_base + 16 i, lds_base + 16 i + 16).  lds_base is wave-uniform (M0).
// The source is a wave-uniform base (a scalar register pair) plus a 32-bit
// per-lane byte offset, so each copy stream holds one vector register.
__device__ __forceinline__ void dma16(const void *sbase, uint32_t voff, uint32_t lds_base) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "global_load_lds_dwordx4 %1, %2"
        :
        : "s"(lds_base), "v"(voff), "s"(sbase)
        : "memory", "m0");
}

// The same copy with the non-temporal hint (streamed data: the weights).
__device__ __forceinline__ void dma16_nt(const void *sbase, uint32_t voff, uint32_t lds_base) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "global_load_lds_dwordx4 %1, %2 nt"
        :
        : "s"(lds_base), "v"(voff), "s"(sbase)
        : "memory", "m0");
}

__device__ __forceinline__ uint32_t lds_addr(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// One dword per lane, global -> LDS (lane i writes LDS bytes [lds_base + 4 i,
// lds_base + 4 i + 4)).
__device__ __forceinline__ void dma4(const void *gptr, uint32_t lds_base) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "global_load_lds_dword %1, off"
        :
        : "s"(lds_base), "v"(gptr)
        : "memory", "m0");
}

}  // namespace megamoe
