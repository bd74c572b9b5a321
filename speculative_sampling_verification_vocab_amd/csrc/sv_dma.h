// Stages of operands moved from memory straight into LDS (gfx950): the DMA, the
// wait for it, which the compiler does not keep track of, and the barrier of a
// pipeline whose buffers are refilled behind it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sv {

// At most N of the wave's vector memory operations are still in flight.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A barrier that leaves DMAs in flight.  The wave's own LDS reads are done
// before it, wherever the compiler puts the products that use them: the buffer
// they come from is refilled behind it.
__device__ __forceinline__ void block_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// One 16-byte global_load_lds per lane: lane l's bytes land at lds + 16 * l (lds
// is the wave's uniform base).  The default cache policy: the nontemporal one
// measured 10-35 % slower in the static-shortlist head.
__device__ __forceinline__ void dma16(const void* g, uint8_t* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_global_load_lds(g, lds, 16, 0, 0);
#endif
}

}  // namespace sv
