// Loads from global memory straight to LDS, reads of what they brought, and the waits between.
#pragma once

#include "mx_device.h"

namespace moed {

// 16 bytes per lane from global memory straight to LDS: lane i of the wavefront
// writes base + 16 i (base uniform). No register receives the data; the caller
// waits on vmcnt before a barrier. Written as asm because the compiler makes
// every later LDS read wait for the builtin's load, whatever buffer it fills.
// The address is a uniform base plus a lane's 32-bit offset.
__device__ __forceinline__ void load_to_lds16(const uint8_t* from, uint32_t offset, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(from), "s"(base)
                 : "memory", "m0");
}

// The same from an address of each lane's own.
__device__ __forceinline__ void load_to_lds16(const uint8_t* from, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(base) : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Until all but the N last things that this wavefront asked LDS for have come.
template <int N = 0>
__device__ __forceinline__ void wait_lds()
{
    asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"(N) : "memory");
}

// What this wavefront wrote to LDS is there for its other lanes.
__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A workgroup's barrier and nothing else: what has to have come or gone before it is the caller's to wait for.
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }

__device__ __forceinline__ u32x4 lds16(const uint8_t* p) { return *reinterpret_cast<const u32x4*>(p); }

}  // namespace moed
