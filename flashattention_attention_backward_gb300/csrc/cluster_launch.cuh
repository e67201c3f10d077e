// Launches of a kernel whose units are shared by clusters of CTAs (sink_units.cuh).
#pragma once

#include <atomic>

#include "attn_common.cuh"

namespace attn {

// K names the kernel (K::kern), its threads a CTA and its bytes of shared memory
// (K::kBlock, K::kSmem).
template <typename K>
struct Clusters {
  // A launch of `units` clusters of `ctas` CTAs; attr is the caller's.
  static cudaLaunchConfig_t config(long long units, int ctas, cudaLaunchAttribute& attr) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ctas);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(static_cast<unsigned>(units * ctas));
    c.blockDim = dim3(K::kBlock);
    c.dynamicSmemBytes = K::kSmem;
    c.attrs = &attr;
    c.numAttrs = 1;
    return c;
  }

  // Clusters of `ctas` CTAs (2, 4 or 8) that run at once on the current device, asked
  // once per device (15 of 8, 36 of 4, 76 of 2 on 152 SMs); 0 if it cannot say.
  static int at_once(int ctas) {
    static std::atomic<int> known[kMaxTrackedDevices][3];
    static std::atomic<bool> configured[kMaxTrackedDevices];
    if (!set_smem_limit_once(K::kern, K::kSmem, configured)) {
      cudaGetLastError();  // not for the launch that does without clusters to report
      return 0;
    }
    const int s = ctas == 2 ? 0 : ctas == 4 ? 1 : 2;
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const bool tracked = dev >= 0 && dev < kMaxTrackedDevices;
    if (tracked && (n = known[dev][s].load(std::memory_order_relaxed)) > 0) return n;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t c = config(1, ctas, attr);
    if (cudaOccupancyMaxActiveClusters(&n, K::kern, &c) != cudaSuccess) {
      cudaGetLastError();  // a smaller cluster may do
      return 0;
    }
    if (tracked) known[dev][s].store(n, std::memory_order_relaxed);
    return n;
  }

  // `units` units, each by a cluster of `ctas` CTAs that at_once has been asked about.
  template <typename... Args>
  static int launch(long long units, int ctas, cudaStream_t stream, const Args&... args) {
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t c = config(units, ctas, attr);
    c.stream = stream;
    if (cudaLaunchKernelEx(&c, K::kern, args...) != cudaSuccess) {
      cudaGetLastError();  // reported here, not by a later call
      return ATTN_ERR_LAUNCH;
    }
    return ATTN_OK;
  }
};

}  // namespace attn
