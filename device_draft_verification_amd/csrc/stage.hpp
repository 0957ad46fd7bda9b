// Waits and barriers that leave loads from memory on their way.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace specv {

__device__ constexpr int wait_loads(int n) {
    // s_waitcnt operand: vmcnt n (bits 3:0 and 15:14), lgkmcnt 0 (bits 11:8), expcnt not waited
    return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4);
}

// At most n global loads and no LDS access of this wavefront outstanding, then
// the workgroup's barrier. Unlike __syncthreads it leaves the n youngest loads
// in flight; the empty asm keeps the compiler from moving memory accesses across.
template <int N>
__device__ __forceinline__ void stage_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_loads(N));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// What a wavefront's lanes wrote to LDS before it is there for all its lanes behind it. The
// LDS keeps a wavefront's accesses in order, so that this is no instruction; without it
// the compiler may take them for one lane's own.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The workgroup's barrier for exchanges through LDS: unlike __syncthreads it
// does not wait for global loads, so that a row stays on its way while its list
// is reduced. The empty asm keeps the compiler from moving accesses across.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    // s_waitcnt: lgkmcnt 0, vmcnt and expcnt at their largest (not waited)
    __builtin_amdgcn_s_waitcnt((0xF) | (0x3 << 14) | (0x7 << 4));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace specv
