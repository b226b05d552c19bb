// tc5.cuh -- the fifth-generation tensor cores (tcgen05) and their memory.
//
// One thread issues a 128-row MMA whose operands lie in shared memory (A may
// lie in tensor memory) and whose fp32 accumulators lie in tensor memory, 128
// lanes by 512 columns per SM.  Lane r of an accumulator is row r; a warp reads
// and writes the 32 lanes of its rank modulo four.
#pragma once

#include "common.cuh"

namespace ssa {

// Takes all 512 columns; the address (0) goes to *dst.  One warp.
__device__ __forceinline__ void tmem_alloc_all(uint32_t* dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;"
               ::"r"(smem_u32(dst)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_all(uint32_t addr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(addr));
}

__device__ __forceinline__ void tc5_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc5_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// MMAs and commits are issued by one elected thread of a warp that runs them
// together: in converged code the operands stay in uniform registers (under an
// if for one lane every MMA fetched its six words anew, 80 clocks an MMA of 64).
// The barrier gets one arrival when every MMA issued so far by this warp is done.
__device__ __forceinline__ void tc5_commit(uint64_t* bar) {
  asm volatile("{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
               "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
               ::"r"(smem_u32(bar)) : "memory");
}

// Shared-memory operand with the 128-byte swizzle: the words of its descriptor.
// K-major: rows of 64 16-bit elements, 1024 bytes between groups of 8 rows (kb
// 16).  MN-major: kb bytes between groups of 64 elements, 1024 between 8 k.
// Addresses advance by 16 bytes a unit of the low word.
constexpr uint32_t kTc5DescHigh = 1024u >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t tc5_desc(uint32_t addr, uint32_t kb) { return addr >> 4 | kb >> 4 << 16; }
// kind::f16, fp32 accumulators, 128 x N; b_mn: B is MN-major
__host__ __device__ constexpr uint32_t tc5_idesc(bool bf16, int N, bool b_mn) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_mn ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 |
         (uint32_t)(128 >> 4) << 24;
}
// d (+)= a b^T, a and b in shared memory
__device__ __forceinline__ void tc5_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile("{\n.reg .pred p, e;\n.reg .b64 a, b;\nelect.sync _|e, 0xffffffff;\nsetp.ne.u32 p, %4, 0;\n"
               "mov.b64 a, {%1, %5};\nmov.b64 b, {%2, %5};\n"
               "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}"
               ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kTc5DescHigh) : "memory");
}
// a in tensor memory
__device__ __forceinline__ void tc5_mma_ta(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile("{\n.reg .pred p, e;\n.reg .b64 b;\nelect.sync _|e, 0xffffffff;\nsetp.ne.u32 p, %4, 0;\n"
               "mov.b64 b, {%2, %5};\n"
               "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}"
               ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(kTc5DescHigh) : "memory");
}

// 32 columns of this warp's lanes.
#define SSA_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), \
                     "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define SSA_W8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), \
                     "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
__device__ __forceinline__ void tmem_ld32(uint32_t* x, uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
               "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : SSA_R8(x, 0), SSA_R8(x, 8), SSA_R8(x, 16), SSA_R8(x, 24) : "r"(addr));
}
// Waits for the loads so far; x, loaded by the last of them, has its values only now.
#define SSA_RW8(x, i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3]), "+r"(x[i + 4]), \
                      "+r"(x[i + 5]), "+r"(x[i + 6]), "+r"(x[i + 7])
__device__ __forceinline__ void tmem_wait_ld(uint32_t* x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : SSA_RW8(x, 0), SSA_RW8(x, 8), SSA_RW8(x, 16), SSA_RW8(x, 24) :: "memory");
}
// 16 columns
__device__ __forceinline__ void tmem_ld16(uint32_t* x, uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
               "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : SSA_R8(x, 0), SSA_R8(x, 8) : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t* x) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : SSA_RW8(x, 0), SSA_RW8(x, 8) :: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
               "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
               ::SSA_W8(x, 0), SSA_W8(x, 8), "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

}  // namespace ssa
