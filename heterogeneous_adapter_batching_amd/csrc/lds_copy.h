// Direct copies from memory to LDS, and the waits for them.
#pragma once

#include <hip/hip_runtime.h>

#include "device_ops.h"

namespace lora {
namespace {

// A direct copy of 16 bytes a lane from memory to LDS at m0 + 16 * lane, past
// the registers.  Written as one instruction block: the compiler then does not
// wait for every copy before the next LDS read, and the kernel counts them
// itself.  Out-of-range lanes write zeros.  (The wait states cover a resource
// word that a vector instruction wrote just before: 5; m0 needs 1.)
// ONCE: the bytes are read by no other workgroup, and streamed past the L2.
template <bool ONCE = false>
__device__ __forceinline__ void copy_to_lds(u32x4 rsrc, uint32_t voff, uint32_t soff,
                                            uint32_t lds) {
    if constexpr (ONCE)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                     ::"s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     ::"s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
                     : "memory");
}
template <int N> __device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ u32x4 raw_rsrc(const void *base, uint32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return u32x4{uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(p))),
                 uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(p >> 32) & 0xffffu)),
                 uint32_t(__builtin_amdgcn_readfirstlane(bytes)), uint32_t(kRsrcWord3)};
}

}  // namespace
}  // namespace lora
