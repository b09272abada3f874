// A cluster's blocks: their barrier and each other's shared memory.
#pragma once

#include "wcomp_impl.cuh"

namespace wc {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float, or a word, of block `rank` at the shared-memory address that `at` is in this one.
__device__ __forceinline__ float cluster_lds(uint32_t at, uint32_t rank) {
  float v;
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.f32 %0, [r];\n\t}"
               : "=f"(v)
               : "r"(at), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_lds_u32(uint32_t at, uint32_t rank) {
  return __float_as_uint(cluster_lds(at, rank));
}

}  // namespace wc
