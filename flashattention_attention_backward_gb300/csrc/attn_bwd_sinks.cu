// attn_bwd_sinks at d = 64 and 128: the kernels of attn_bwd_kernel.cuh with sinks, and
// how their units are shared out. A source file of its own: the forms without sinks
// keep their code (sinks as a run-time matter cost the dropout form 2 % in spills).
#include <algorithm>

#include "attn_bwd_kernel.cuh"
#include "cluster_launch.cuh"
#include "element.cuh"
#include "sink_units.cuh"

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

// The units 0 .. p.n_units - 1, each by a cluster of p.split CTAs.
template <int D, bool SOFTCAP>
struct Split {
  static constexpr auto kern = attn_bwd_kernel<D, false, SOFTCAP, false, false, true, true>;
  static constexpr int kBlock = kThreads, kSmem = Layout<D>::kBytes;
};

template <int D, bool SOFTCAP>
int launch_both(const Maps& m, SinkParams p, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_LAUNCH;
  const int with_sinks = (p.sinks + kBc - 1) / kBc * p.H_kv * p.B;  // units, the first ones
  const int others = p.n_units - with_sinks;
  // a unit with sinks visits all query tiles but those before its block
  const long long group = p.H / p.H_kv;
  const long long band_tiles = std::min<long long>(
      p.m_blocks, (static_cast<long long>(p.win_left) + p.win_right + kBc - 1) / kBr + 1);
  const SinkUnits units{with_sinks, others, group * p.m_blocks, group * band_tiles,
                        group * (p.m_blocks - (p.sinks - 1) / kBc)};
  using Shared = Clusters<Split<D, SOFTCAP>>;
  p.split = sinks_cluster(units, sms, Shared::at_once);
  int grid = p.n_units < sms ? p.n_units : sms;
  if (p.split > 1) {
    SinkParams shared = p;
    shared.n_units = with_sinks;
    const int rc = Shared::launch(with_sinks, p.split, stream, m.q, m.k, m.v, m.dO, m.dq, m.dk,
                                  m.dv, shared);
    if (rc != ATTN_OK || others == 0) return rc;
    p.first_unit = with_sinks;
    p.n_units = others;
    grid = others < sms ? others : sms;
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
