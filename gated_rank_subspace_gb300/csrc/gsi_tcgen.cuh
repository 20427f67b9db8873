// Wrappers of the tcgen05 products, TMEM accesses and operand descriptors that the
// attention's row tiles and the gathered weights share (sm_103a inline PTX).
#pragma once

#include "gsi_async.cuh"

namespace gsi {

__device__ __forceinline__ void tl_mma_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(uint32_t(acc))
      : "memory");
}
__device__ __forceinline__ void tl_mma_ts(uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(at), "l"(bd), "r"(idesc), "r"(uint32_t(acc))
      : "memory");
}
// One lane of the warp.  (The compiler knows that a branch on this has one
// thread, and the products' operands then reach their uniform registers
// directly; behind `lane == 0` it loops over the threads there might be, at
// ~190 cycles a product.)
__device__ __forceinline__ bool tl_elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tl_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sa(bar)) : "memory");
}
__device__ __forceinline__ void tl_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tl_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tl_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tl_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define GSI_R8(r, i) "=r"((r)[(i)]), "=r"((r)[(i) + 1]), "=r"((r)[(i) + 2]), "=r"((r)[(i) + 3]), "=r"((r)[(i) + 4]), \
                     "=r"((r)[(i) + 5]), "=r"((r)[(i) + 6]), "=r"((r)[(i) + 7])
#define GSI_W8(r, i) "r"((r)[(i)]), "r"((r)[(i) + 1]), "r"((r)[(i) + 2]), "r"((r)[(i) + 3]), "r"((r)[(i) + 4]), \
                     "r"((r)[(i) + 5]), "r"((r)[(i) + 6]), "r"((r)[(i) + 7])
// 32 columns of this warp's 32 lanes (no wait).
__device__ __forceinline__ void tl_ld32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%32];"
      : GSI_R8(r, 0), GSI_R8(r, 8), GSI_R8(r, 16), GSI_R8(r, 24)
      : "r"(t));
}
__device__ __forceinline__ void tl_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(t), GSI_W8(r, 0), GSI_W8(r, 8), GSI_W8(r, 16), GSI_W8(r, 24)
      : "memory");
}

// After tl_wait_ld(): nothing that uses these registers may move before it.
#define GSI_H8(r, i) "+r"((r)[(i)]), "+r"((r)[(i) + 1]), "+r"((r)[(i) + 2]), "+r"((r)[(i) + 3]), "+r"((r)[(i) + 4]), \
                     "+r"((r)[(i) + 5]), "+r"((r)[(i) + 6]), "+r"((r)[(i) + 7])
__device__ __forceinline__ void tl_arrived32(uint32_t* r) {
  asm volatile("" : GSI_H8(r, 0), GSI_H8(r, 8), GSI_H8(r, 16), GSI_H8(r, 24)::"memory");
}

// Shared-memory operand descriptors, 128-byte swizzle (version 1).  K-major
// (Q, K: rows of 64 columns): 8-row groups 1024 bytes apart.  MN-major (V: a
// row is a key, its 64 columns run along N): 8-key groups 1024 bytes apart,
// the next 64 columns `slab` bytes on.
__device__ __forceinline__ uint64_t tl_desc(uint32_t addr, uint32_t slab) {
  return uint64_t((addr & 0x3ffffu) >> 4) | (uint64_t(slab >> 4) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}
// kind::f16, A and B bf16, D float32; b_mn: B is MN-major.
__host__ __device__ constexpr uint32_t tl_idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(b_mn) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

__device__ __forceinline__ void tl_load_query(uint32_t dst, const CUtensorMap* map, uint32_t bar, int col, int head, int tok) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(col), "r"(head), "r"(tok), "r"(bar)
      : "memory");
}

}  // namespace gsi
