// Thread-block clusters: the hardware barrier and reads of another CTA's shared memory.  Written from the
// public PTX ISA description of these instructions.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace dsa {

// All threads of all CTAs of the cluster (converged warps); earlier writes, to shared and to global memory, are
// visible to the cluster afterwards.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// 32-bit word at `addr` (a shared-memory address of this CTA) in CTA `rank` of the cluster.
__device__ __forceinline__ int32_t ld_cluster_s32(uint32_t addr, uint32_t rank) {
  int32_t v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.s32 %0, [a];\n\t}"
               : "=r"(v)
               : "r"(addr), "r"(rank)
               : "memory");
  return v;
}

}  // namespace dsa
