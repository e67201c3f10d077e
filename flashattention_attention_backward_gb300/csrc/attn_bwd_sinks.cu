// attn_bwd_sinks at d = 64 and 128: the kernels of attn_bwd_kernel.cuh with sinks, and
// how their units are shared out. A source file of its own: the forms without sinks
// keep their code (sinks as a run-time matter cost the dropout form 2 % in spills).
#include <algorithm>

#include "attn_bwd_kernel.cuh"
#include "element.cuh"

namespace attn {
namespace bwd {

// The units from p.first_unit on; behind the clusters' launch they may begin beside its.
template <int D, bool SOFTCAP>
int launch_units(const Maps& m, const SinkParams& p, int grid, cudaStream_t stream) {
  auto kern = attn_bwd_kernel<D, false, SOFTCAP, false, false, true, false>;
  static std::atomic<bool> configured[kMaxTrackedDevices];
  if (!set_smem_limit_once(kern, Layout<D>::kBytes, configured)) return ATTN_ERR_LAUNCH;
  if (p.split > 1)
    return launch_overlapped(kern, dim3(static_cast<unsigned>(grid)), kThreads, Layout<D>::kBytes,
                             0, stream, m.q, m.k, m.v, m.dO, m.dq, m.dk, m.dv, p);
  kern<<<grid, kThreads, Layout<D>::kBytes, stream>>>(m.q, m.k, m.v, m.dO, m.dq, m.dk, m.dv, p);
  return launch_status();
}

template <int D, bool SOFTCAP>
struct Split {
  static constexpr auto kern = attn_bwd_kernel<D, false, SOFTCAP, false, false, true, true>;

  // A launch of `units` clusters of `split` CTAs; attr is the caller's.
  static cudaLaunchConfig_t config(int units, int split, cudaLaunchAttribute& attr) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(split);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(static_cast<unsigned>(units) * static_cast<unsigned>(split));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = Layout<D>::kBytes;
    c.attrs = &attr;
    c.numAttrs = 1;
    return c;
  }

  static bool prepare() {
    static std::atomic<bool> configured[kMaxTrackedDevices];
    return set_smem_limit_once(kern, Layout<D>::kBytes, configured);
  }

  // Clusters of `split` CTAs (2, 4 or 8) that run at once on the current device, asked
  // once per device (15 of 8, 36 of 4, 76 of 2 on 152 SMs); 0 if it cannot say.
  static int at_once(int split) {
    static std::atomic<int> known[kMaxTrackedDevices][3];
    const int s = split == 2 ? 0 : split == 4 ? 1 : 2;
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const bool tracked = dev >= 0 && dev < kMaxTrackedDevices;
    if (tracked && (n = known[dev][s].load(std::memory_order_relaxed)) > 0) return n;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t c = config(1, split, attr);
    if (cudaOccupancyMaxActiveClusters(&n, kern, &c) != cudaSuccess) {
      cudaGetLastError();  // a smaller cluster may do
      return 0;
    }
    if (tracked) known[dev][s].store(n, std::memory_order_relaxed);
    return n;
  }

  // The units 0 .. p.n_units - 1, each by a cluster of p.split CTAs.
  static int launch(const Maps& m, const SinkParams& p, cudaStream_t stream) {
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t c = config(p.n_units, p.split, attr);
    c.stream = stream;
    if (cudaLaunchKernelEx(&c, kern, m.q, m.k, m.v, m.dO, m.dq, m.dk, m.dv, p) != cudaSuccess) {
      cudaGetLastError();  // reported here, not by a later call
      return ATTN_ERR_LAUNCH;
    }
    return ATTN_OK;
  }
};

template <int D, bool SOFTCAP>
int launch_both(const Maps& m, SinkParams p, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_LAUNCH;
  const int with_sinks = (p.sinks + kBc - 1) / kBc * p.H_kv * p.B;  // units, the first ones
  // query tiles of a unit of a band, of one with sinks (all tiles but those before
  // the unit's block), and of all units
  const long long group = p.H / p.H_kv, most = group * p.m_blocks;
  const long long band_tiles = std::min<long long>(
      p.m_blocks, (static_cast<long long>(p.win_left) + p.win_right + kBc - 1) / kBr + 1);
  const long long all = with_sinks * most + (p.n_units - with_sinks) * group * band_tiles;
  // A unit with sinks that outlasts what an SM has on average is shared by a
  // cluster of CTAs, in a launch of its own that the other units' runs beside (1 x 8
  // heads over 1 x 16384 x 128, window 1024: the step takes 357 us, 528 with one launch
  // behind the other, 2361 without clusters; 1 x 4 x 8192 x 64, window 512: 51, 67, 149).
  // The last such unit has the fewest tiles: one for each CTA at least. How many CTAs:
  // those with the earliest end, in tiles, where a unit's start and epilogue are worth
  // kTurn, clusters that do not run at once go in rounds, and the other units begin
  // with the last round, on the SMs that it leaves or, if they need more, behind it. (1
  // x 32 heads over 8 x 16384, window 1024: 8 CTAs, 870 us; as many as bring the unit
  // down to the average, 2, took 1134. 1 x 16 over 8 x 8192, window 512, 200 sinks: 16
  // clusters of 4, 221 us; of 8, which run 15 at a time, 247.)
  constexpr int kTurn = 4;
  const long long least = group * (p.m_blocks - (p.sinks - 1) / kBc);
  const int others = p.n_units - with_sinks;
  int grid = p.n_units < sms ? p.n_units : sms;
  if (most * sms > all * 5 / 4) {
    if (!Split<D, SOFTCAP>::prepare()) return ATTN_ERR_LAUNCH;
    const int g = others < sms ? others : sms;
    const long long band = g > 0 ? (others + g - 1) / g * (group * band_tiles + kTurn) : 0;
    long long best = 0;
    for (int split = 2; split <= 8 && split <= least; split *= 2) {
      const int at_once = Split<D, SOFTCAP>::at_once(split);
      if (at_once <= 0) break;
      const long long heavy = (most + split - 1) / split + kTurn;
      const int before = (with_sinks - 1) / at_once;  // rounds in front of the last
      const long long last = static_cast<long long>(with_sinks - before * at_once) * split;
      const long long end =
          before * heavy + (last + g <= sms ? std::max(heavy, band) : heavy + band);
      if (p.split > 1 && end > best) continue;
      best = end;
      p.split = split;
    }
    if (p.split > 1) {
      SinkParams shared = p;
      shared.n_units = with_sinks;
      const int rc = Split<D, SOFTCAP>::launch(m, shared, stream);
      if (rc != ATTN_OK || others == 0) return rc;
      p.first_unit = with_sinks;
      p.n_units = others;
      grid = g;
    }
  }
  if (p.split == 1) {
    p.heavy_passes = with_sinks / grid;
    p.heavy = with_sinks % grid;
    p.ahead = p.heavy > 0 ? static_cast<int>((p.m_blocks + band_tiles / 2) / band_tiles) : 0;
  }
  return launch_units<D, SOFTCAP>(m, p, grid, stream);
}

int launch_sinks(const Maps& m, const Params& base, int sinks, void* dk, void* dv, int d,
                 cudaStream_t stream) {
  SinkParams p{};
  static_cast<Params&>(p) = base;
  p.sinks = sinks;
  p.split = 1;
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  const bool cap = p.softcap > 0.f;
  if (d == 128)
    return cap ? launch_both<128, true>(m, p, stream) : launch_both<128, false>(m, p, stream);
  return cap ? launch_both<64, true>(m, p, stream) : launch_both<64, false>(m, p, stream);
}

int sinks_status(int* status, bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_status, sizeof(int)) != cudaSuccess) return ATTN_ERR_LAUNCH;
  *status = v;
  const int zero = 0;
  if (clear && v != 0 && cudaMemcpyToSymbol(g_status, &zero, sizeof(int)) != cudaSuccess)
    return ATTN_ERR_LAUNCH;
  return ATTN_OK;
}

}  // namespace bwd
}  // namespace attn
