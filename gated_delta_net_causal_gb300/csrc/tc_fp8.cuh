// tcgen05 on 8-bit operands and over pairs of CTAs (a cluster of two).
#pragma once

#include "gdn_common.cuh"
#include "tc_common.cuh"

namespace gdn {

// Arrive on a barrier of another CTA of the cluster (address from mapa).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

namespace tc {

constexpr uint32_t kE4M3 = 0;  // operand format of kind::f8f6f4

// One MMA on 8-bit floating operands (32 of K), both from shared memory, issued
// by one elected lane of a converged warp. The instruction descriptor's operand
// formats are kE4M3.
__device__ __forceinline__ void mma_f8_elect(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id,
                                             bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(id), "r"((uint32_t)accumulate)
      : "memory");
}
// The same over a pair of CTAs (a cluster of two): A and B each half in either
// CTA's shared memory at the same place, D's upper half of the rows in the
// second CTA's TMEM. Issued by the first CTA alone.
__device__ __forceinline__ void mma_f8_pair_elect(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t id,
                                                  bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(id), "r"((uint32_t)accumulate)
      : "memory");
}
// Arrive on the barrier at this place in both CTAs once the pair's MMAs issued
// so far have completed.
__device__ __forceinline__ void mma_commit_pair_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// TMEM of a pair: one warp of each CTA allocates, and frees, its half.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// tma_load_2d completing on a barrier of either CTA of a pair (an address of
// the cluster's shared memory).
__device__ __forceinline__ void tma_load_2d_pair(void* smem_dst, const void* tmap, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(smem_dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

}  // namespace tc
}  // namespace gdn
