// Device helpers of the staged loss kernels: mbarriers with bounded waits and
// 1-D bulk copies between global and shared memory.  (step_tma.cu has its own,
// which its recorded DRAM counters go with.)
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace shardstep {

// Bits of the device status word (shardstep_device_status).
constexpr unsigned kStatusConsumerTimeout = 1u;
constexpr unsigned kStatusProducerTimeout = 2u;
constexpr unsigned kStatusDrainTimeout = 4u;
// How long a block waits for its own copies in flight before it exits.
constexpr unsigned long long kDrainNs = 2000000000ull;

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count)
                 : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(b)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(b)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_addr(b)), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
// Non-blocking test of the phase of `parity`.
__device__ __forceinline__ bool mbar_test_now(uint64_t* b, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_addr(b)), "r"(parity)
        : "memory");
    return done != 0;
}
// Limits below this are a test control: their waits poll without blocking
// and read the clock after every poll, so that they run out even when each
// blocking poll would have lasted until the copy landed.
constexpr unsigned long long kShortWaitNs = 1000000ull;
// Waits for the phase of `parity` to complete; false after limit_ns.  The
// usual limit polls with try_wait, which suspends the thread until the
// phase completes or a hardware time slice ends, and reads the clock every
// 256 polls.
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity,
                                          unsigned long long limit_ns) {
    if (limit_ns < kShortWaitNs) {
        const unsigned long long t0 = now_ns();
        while (!mbar_test_now(b, parity))
            if (now_ns() - t0 > limit_ns) return false;
        return true;
    }
    if (mbar_test(b, parity)) return true;   // the clock is read only by a wait that lasts
    const unsigned long long t0 = now_ns();
    for (uint32_t k = 1;; ++k) {
        if (mbar_test(b, parity)) return true;
        if ((k & 255u) == 0 && now_ns() - t0 > limit_ns) return false;
    }
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}
// The L2 policy of data that will not be touched again soon.
__device__ __forceinline__ uint64_t evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
// bulk_load of data that is not read again.
__device__ __forceinline__ void bulk_load_once(void* dst, const void* src, uint32_t bytes,
                                               uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1], %2, [%3], %4;" ::"r"(smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}
// A bulk store of shared memory, in this thread's current bulk group.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes,
                                           uint64_t policy) {
    asm volatile(
        "cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;" ::"l"(dst),
        "r"(smem_addr(src)), "r"(bytes), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void bulk_commit() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until at most N of this thread's groups still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
// Orders this thread's writes to shared memory before later bulk copies that
// read it (issued after a barrier by another thread).
__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

}  // namespace shardstep
