// The fifth-generation tensor cores: descriptors, and the tcgen05 instructions
// that the matrix kernels issue.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "tma.cuh"

namespace shardstep {

// Shared-memory operand of 16-bit elements in the 128-byte swizzle: rows of 128
// bytes, eight rows to a group of 1024, the 16-byte pieces of row r at their
// place xor r % 8.  K-major: a row holds 64 consecutive k of one m (or n); the
// groups of eight m follow each other.  MN-major: a row holds 64 consecutive m
// (or n) of one k; the groups of eight k follow each other, and `next` bytes on
// come the next 64 m.
// Everything but the address and `next` is the same for all: the high words are, so that
// only low ones are formed and moved.
constexpr uint32_t kDescHigh = (1024 / 16) |       // from group to group
                               (1u << 14) |        // version
                               (2u << 29);         // 128-byte swizzle
__device__ __forceinline__ uint32_t k_major(uint32_t addr) {
    return (1u << 16) | ((addr & 0x3FFFFu) >> 4);
}
__device__ __forceinline__ uint32_t mn_major(uint32_t addr, uint32_t next) {
    return ((next / 16) << 16) | ((addr & 0x3FFFFu) >> 4);
}
// fp16 x fp16 -> fp32, m x n; which operands are MN-major.
__device__ __forceinline__ uint32_t half_product(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n / 8) << 17) | (static_cast<uint32_t>(m / 16) << 24);
}

// Tensor memory: columns of 128 lanes x 32 bits.  A whole warp calls these (in both
// blocks of a pair); the address lands in shared memory.
template <bool PAIR, int COLUMNS>
__device__ __forceinline__ void tmem_alloc(uint32_t* to) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(to)),
                     "n"(COLUMNS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(to)),
                     "n"(COLUMNS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <bool PAIR, int COLUMNS>
__device__ __forceinline__ void tmem_free(uint32_t addr) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr),
                     "n"(COLUMNS)
                     : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr),
                     "n"(COLUMNS)
                     : "memory");
}

// One lane of a warp that is together, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(p));
    return p != 0;
}
// One thread (of a pair's first block): D (+)= A B for 16 k, A and B given by their
// descriptors' low words.  A pair's blocks hold half of A's rows and half of B's columns
// each, at the same shared addresses, and get their rows of D.
template <bool PAIR>
__device__ __forceinline__ void mma_half(uint32_t d, uint32_t a, uint32_t b, uint32_t form,
                                         bool add) {
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %4, 0;\n"
            " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
            "r"(a), "r"(b), "r"(form), "r"(static_cast<uint32_t>(add)), "n"(kDescHigh)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %4, 0;\n"
            " mov.b64 a, {%1, %5};\n mov.b64 b, {%2, %5};\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
            "r"(a), "r"(b), "r"(form), "r"(static_cast<uint32_t>(add)), "n"(kDescHigh)
            : "memory");
}
// Arrives at the barrier (of both blocks of a pair) when this thread's products so
// far are done.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                smem_addr(bar))
            : "memory");
}

// A pair's blocks: this one's rank, arrivals at the first one's barrier, waits for
// arrivals from either (mbar_wait, but ordering what another block did before).
__device__ __forceinline__ uint32_t pair_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void arrive_at_first(uint64_t* bar) {
    asm volatile(
        "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n"
        " mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n}\n" ::"r"(smem_addr(bar))
        : "memory");
}
// The same for tensor memory that has been read: the fences of tcgen05 order it, nothing
// else has to be seen (a release of all memory takes 1000 clocks).
__device__ __forceinline__ void tmem_read_at_first(uint64_t* bar) {
    asm volatile(
        "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n"
        " mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n}\n" ::"r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
__device__ __forceinline__ bool mbar_wait_pair(uint64_t* b, uint32_t parity,
                                               unsigned long long limit_ns) {
    unsigned long long t0 = 0;
    for (uint32_t k = 0;; ++k) {
        uint32_t done;
        if (limit_ns < kShortWaitNs)
            asm volatile(
                "{\n .reg .pred p;\n"
                " mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                " selp.u32 %0, 1, 0, p;\n}\n"
                : "=r"(done)
                : "r"(smem_addr(b)), "r"(parity)
                : "memory");
        else
            asm volatile(
                "{\n .reg .pred p;\n"
                " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                " selp.u32 %0, 1, 0, p;\n}\n"
                : "=r"(done)
                : "r"(smem_addr(b)), "r"(parity)
                : "memory");
        if (done) return true;
        if (k == 0) t0 = now_ns();
        else if ((limit_ns < kShortWaitNs || (k & 255u) == 0) && now_ns() - t0 > limit_ns)
            return false;
    }
}
__device__ __forceinline__ void tmem_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// A warp's 32 lanes (its quarter) of 8 columns.
__device__ __forceinline__ void tmem_load8(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
        " tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(addr)
        : "memory");
}
// Of 32 columns.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];\n"
        " tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

}  // namespace shardstep
