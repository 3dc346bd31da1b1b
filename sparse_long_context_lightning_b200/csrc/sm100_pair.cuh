// PTX wrappers for kernels in which the two CTAs of a cluster of two share their matrix instructions
// (tcgen05 with cta_group::2).  An M = 128 instruction of a pair takes rows [0, 64) of A from the even CTA's shared
// memory and [64, 128) from the odd one's, and half of B's N rows from each; both operands are given by one
// descriptor, so they lie at the same offsets in both CTAs.  Each CTA's tensor memory holds its own 64 rows: lane
// r < 64 columns [0, N/2) of row r, lane 64 + r columns [N/2, N).
#pragma once

#include "sm100.cuh"

namespace lsa {
namespace sm100 {

// one lane of a converged warp, with the branch known to be uniform: the matrix instructions that it issues take
// their descriptors from uniform registers without a conversion for each (65 -> 24 clocks an instruction, measured)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// allocation and release by one warp of each CTA of the pair
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// issued by the even CTA only
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrive on the barrier at this offset in both CTAs once the thread's earlier pair instructions are complete
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
      ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3))
      : "memory");
}
// tile load into this CTA's shared memory that signals a barrier of either CTA of the pair (shared::cluster address)
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* m, uint32_t cbar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(m)), "r"(cbar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Arrive on a barrier of either CTA of the pair (shared::cluster address).  The release is at CTA scope: what it publishes
// is this CTA's own tensor memory (loaded to registers before) and its own shared memory (written, then fenced for the
// async proxy), and the matrix instructions that follow read them where they lie.  A release at cluster scope also
// waits for the thread's accesses at the L2's distance: about 1000 clocks an arrival, two in every block.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t caddr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(caddr) : "memory");
}

// the cluster's barrier without the wait for this thread's earlier stores: for an end where nothing is read any more
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

}  // namespace sm100
}  // namespace lsa
