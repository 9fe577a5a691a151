// Inline-PTX wrappers of the fifth-generation tensor cores (sm_103a): tensor
// memory, tcgen05.mma on e4m3 operands in shared memory, and its completion.
#pragma once

#include <cstdint>

namespace pa {
namespace tc {

// Shared-memory matrix descriptor of a 128-byte-swizzled operand at `addr`
// (16-byte aligned, its tile 1024-byte aligned): rows of 128 bytes, groups of
// eight rows 1024 bytes apart.  K-major: a row is one M (or N) index and holds
// 128 K values; MN-major: a row is one K index and holds 128 M values.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
  constexpr uint64_t kGroup = 1024 >> 4;
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (kGroup << 16) | (kGroup << 32) | (1ull << 46) |
         (2ull << 61);
}

// The same for a 32-byte-swizzled MN-major operand (its tile 256-byte aligned):
// rows of 32 bytes, a K index with 32 values, groups of eight rows 256 bytes
// apart; the two 16-byte halves of rows 4-7 of a group change places.
__device__ __forceinline__ uint64_t desc_sw32(uint32_t addr) {
  constexpr uint64_t kGroup = 256 >> 4;
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (kGroup << 16) | (kGroup << 32) | (1ull << 46) |
         (6ull << 61);
}

// Instruction descriptor: e4m3 x e4m3 -> fp32, M x N, each operand K-major or
// (a_mn, b_mn) MN-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D[tmem] (+)= A B over 32 values of K; issued by one thread.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

// Arrives at `bar` once every tcgen05.mma this thread issued before is done.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// One warp: allocates `columns` (a power of two >= 32) of tensor memory and
// stores its address at `slot`.
__device__ __forceinline__ void alloc(uint32_t slot, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void dealloc(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

// This warp's 32 lanes (lane field of addr) by N columns: thread i gets lane
// i's values, once wait_ld() has returned.
__device__ __forceinline__ void ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
// Waits for this thread's loads; the values pass through, so that no use of
// them is scheduled ahead of the wait.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

}  // namespace tc
}  // namespace pa
