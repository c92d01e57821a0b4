// pair.cuh -- CTA pairs: a cluster of two CTAs on two neighbouring SMs whose
// tcgen05 MMAs (.cta_group::2, issued by rank 0) span the tensor memory of both.
#pragma once

#include "cluster.cuh"
#include "ptx.cuh"

namespace moe {

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// 2-D tiled TMA load into this CTA's shared memory that completes on an
// mbarrier of either CTA of the pair (bar = shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* smem_dst, const CUtensorMap* m, int32_t c0,
                                                 int32_t c1, uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar_cluster)
      : "memory");
}

// TMEM allocation for a CTA pair: one warp of each CTA executes it.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(smem_slot)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// Arrive once on the barrier at `bar`'s offset in both CTAs of the pair (their
// ranks' bits) when the issuing thread's earlier tcgen05 operations have completed.
__device__ __forceinline__ void tc2_commit_both_warp(uint64_t* bar, uint16_t both = 3) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "h"(both)
      : "memory");
}

// ... on this CTA's barrier only.
__device__ __forceinline__ void tc2_commit_local_warp(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}

// mbar_wait_warp for waits that end within a microsecond and for arrivals from
// the other CTA of the pair (acquire at cluster scope): polls without sleeping,
// since a sleeping warp wakes up late; bounded as the others are.
__device__ __forceinline__ bool mbar_poll_warp(uint64_t* bar, uint32_t parity, uint64_t timeout_ns,
                                               int32_t* status, int32_t code,
                                               volatile int32_t* abort) {
  const uint32_t a = smem_u32(bar);
  uint64_t t0 = 0;
  bool ok = false;
  for (uint32_t n = 1;; ++n) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(a), "r"(parity)
        : "memory");
    if (done) {
      ok = true;
      break;
    }
    if ((n & 63) == 0) {
      if (*abort) break;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > timeout_ns) {
        atomicCAS(status, 0, code);
        *abort = 1;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

}  // namespace moe
