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
constexpr uint64_t kDescBase = (uint64_t{1} << 46) |              // version
                               (uint64_t{2} << 61) |              // 128-byte swizzle
                               (uint64_t{1024 / 16} << 32);       // from group to group
__device__ __forceinline__ uint64_t k_major(uint32_t addr) {
    return kDescBase | (uint64_t{1} << 16) | ((addr & 0x3FFFFu) >> 4);
}
__device__ __forceinline__ uint64_t mn_major(uint32_t addr, uint32_t next) {
    return kDescBase | (static_cast<uint64_t>(next / 16) << 16) | ((addr & 0x3FFFFu) >> 4);
}
// fp16 x fp16 -> fp32, m x n, A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t half_product(int m, int n, bool b_mn_major) {
    return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n / 8) << 17) |
           (static_cast<uint32_t>(m / 16) << 24);
}

// Tensor memory: columns of 128 lanes x 32 bits.  A whole warp calls these; the
// address lands in shared memory.
template <int COLUMNS>
__device__ __forceinline__ void tmem_alloc(uint32_t* to) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(to)),
                 "n"(COLUMNS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLUMNS>
__device__ __forceinline__ void tmem_free(uint32_t addr) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLUMNS)
                 : "memory");
}

// One thread: D (+)= A B for 16 k.
__device__ __forceinline__ void mma_half(uint32_t d, uint64_t a, uint64_t b, uint32_t form,
                                         bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(form), "r"(static_cast<uint32_t>(add))
        : "memory");
}
// Arrives at the barrier when this thread's products so far are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// A warp's 32 lanes (its quarter) of 32 columns.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

}  // namespace shardstep
