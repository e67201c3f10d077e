// Inline-PTX wrappers around launch dependencies and clusters, for the kernels
// around the attention call.
#pragma once

#include <cstdint>

#include "sm103_ptx.cuh"

namespace attn {
namespace ptx {

// Barrier over the threads of a cluster; what they wrote before it, to each
// other's shared memory too, is visible behind it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// This block's rank in its cluster.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
// Writes v to the place that `addr` has in the shared memory of the cluster's
// block `rank`.
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, uint32_t rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.f32 [a], %2;\n\t}" ::"r"(addr),
      "r"(rank), "f"(v)
      : "memory");
}

// Reads from the place that `addr` has in the shared memory of the cluster's
// block `rank`.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// Lets a dependent grid be launched when all blocks have come here or ended.
__device__ __forceinline__ void grid_dependency_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// Waits until the grids this one depends on have completed and their writes
// are visible (a launch that may begin before them).
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace ptx
}  // namespace attn
