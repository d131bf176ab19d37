// Asynchronous copies into per-thread shared-memory slots, and barriers of a
// group of warps.
//
// A thread copies the 16-byte pieces it will read itself, some rows ahead
// (cp.async), so waiting for them takes no barrier: the copies of a thread are
// visible to it when its own wait returns.  That keeps tens of kilobytes per SM
// in flight, which HBM's latency needs, without holding them in registers.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "mhcpb_check.cuh"

namespace mhcpb {
namespace ops {

__device__ __forceinline__ void copy16(void* shared, const void* global) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(shared))),
                 "l"(global)
                 : "memory");
}
__device__ __forceinline__ void copy4(void* shared, const void* global) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(shared))),
                 "l"(global)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N committed groups of this thread have arrived.
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Barrier of the `threads` (a multiple of 32) of group `group` of the block.
__device__ __forceinline__ void group_sync(int group, int threads) {
    if (threads == 32)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

}  // namespace ops
}  // namespace mhcpb
