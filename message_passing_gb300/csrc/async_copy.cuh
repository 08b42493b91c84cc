// Asynchronous copies of 4, 8 or 16 bytes from global to shared memory, thread by thread. A thread that
// reads only what it copied itself needs no barrier: copies_wait is enough.
#pragma once
#include <cstdint>

namespace e3gb {

__device__ __forceinline__ uint32_t shared_address(const void* p) { return uint32_t(__cvta_generic_to_shared(p)); }

// BYTES bytes, or zeros where `live` is false (nothing is read then). Both addresses are multiples of BYTES either way.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool live = true) {
    const int n = live ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(shared_address(dst)), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(shared_address(dst)), "l"(src), "n"(BYTES), "r"(n)
                     : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most N of this thread's groups are still on their way
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace e3gb
