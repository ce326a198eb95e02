// Bulk copies of contiguous bytes from global to shared memory, counted by an
// mbarrier, and waits on them that give up after a limit.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

// How long a wait goes on, and bytes that every phase expects above its copies' (test-only builds change them).
#ifndef EQC_BULK_WAIT_LIMIT_NS
#define EQC_BULK_WAIT_LIMIT_NS 2000000000ull   // 2 s
#endif
#ifndef EQC_TEST_BULK_DEFICIT
#define EQC_TEST_BULK_DEFICIT 0
#endif

namespace eqc {
namespace bulk {

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// A phase takes `count` arrivals (and the bytes they expect).
__device__ __forceinline__ void init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void fence_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }

__device__ __forceinline__ void expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// dst, src and bytes are multiples of 16.
__device__ __forceinline__ void copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// Orders this thread's writes to shared memory before copies issued behind the next barrier.
__device__ __forceinline__ void fence_writes() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Waits for the phase of `parity`; false when the limit passed without it.
// The limit is each thread's own: threads that go on together agree on the
// outcome first (a vote of the warp, or of the CTA at its next barrier).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    uint64_t t0 = 0;
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(a), "r"(parity), "r"(1000u)
            : "memory");
        if (done) return true;
        uint64_t now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (!t0) t0 = now;
        else if (now - t0 > EQC_BULK_WAIT_LIMIT_NS) return false;
    }
}

}  // namespace bulk
}  // namespace eqc
