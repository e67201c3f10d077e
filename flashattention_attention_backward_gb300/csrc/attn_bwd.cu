// attn_bwd and its local, dropout and deterministic forms at d = 64 and 128: host
// code, and the kernels of attn_bwd_kernel.cuh without sinks. The device status
// calls.
#include <cstdint>
#include <cuda_bf16.h>

#include "attn_bwd_kernel.cuh"
#include "cache_common.cuh"

namespace attn {
namespace bwd {

// Exercises the bounded wait of the kernels above on the device: warp 0
// waits on an mbarrier that nothing arrives on, gives up after
// `limit_cycles`, raises the abort flag and records ATTN_ERR_DEVICE_TIMEOUT;
// warp 1, waiting on another such barrier with a far longer limit, returns
// on the abort flag. Nothing faults or traps; the context stays usable.
__global__ void __launch_bounds__(64, 1) wait_timeout_probe(long long limit_cycles) {
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ int abort_flag;
  Ctx c;
  c.bars = smem_u32(bars);
  c.abort = &abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(c.bars, 1);
    mbar_init(c.bars + 8, 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x < 32)
    (void)wait(c, 0, 0, limit_cycles);
  else
    (void)wait(c, 1, 0, 64 * limit_cycles);
  __syncthreads();
}

template <int D, bool CAUSAL, bool SOFTCAP, bool DET, bool DROP>
int launch(const Maps& m, const Params& p, int grid, cudaStream_t stream) {
  auto kern = attn_bwd_kernel<D, CAUSAL, SOFTCAP, DET, DROP, false, false>;
  static std::atomic<bool> configured[kMaxTrackedDevices];
  if (!set_smem_limit_once(kern, Layout<D>::kBytes, configured)) return ATTN_ERR_LAUNCH;
  kern<<<grid, kThreads, Layout<D>::kBytes, stream>>>(m.q, m.k, m.v, m.dO, m.dq, m.dk, m.dv, p);
  return launch_status();
}

}  // namespace bwd
}  // namespace attn

using namespace attn;

namespace attn {
namespace bwd {

template <bool DET, bool DROP>
int dispatch(const Maps& m, const Params& p, int grid, cudaStream_t s, int d, bool cs, bool cap) {
  if (d == 128) {
    if (cs)
      return cap ? launch<128, true, true, DET, DROP>(m, p, grid, s)
                 : launch<128, true, false, DET, DROP>(m, p, grid, s);
    return cap ? launch<128, false, true, DET, DROP>(m, p, grid, s)
               : launch<128, false, false, DET, DROP>(m, p, grid, s);
  }
  if (cs)
    return cap ? launch<64, true, true, DET, DROP>(m, p, grid, s)
               : launch<64, true, false, DET, DROP>(m, p, grid, s);
  return cap ? launch<64, false, true, DET, DROP>(m, p, grid, s)
             : launch<64, false, false, DET, DROP>(m, p, grid, s);
}

// Shared by attn_bwd (dQ added into dq_target) and attn_bwd_deterministic
// (dQ tiles stored into the partials buffer dq_target).
// `before_launch`, when given, runs once every argument check and tensor-map
// encoding has passed, right before the kernel is enqueued (d = 64 and 128
// only); a non-zero return ends the call with that code and nothing more is
// enqueued.
int run(const void* q, const void* k, const void* v, const void* dO, const float* lse,
        float* dq_target, void* dk, void* dv, int B, int H, int H_kv, int N, int d, float scale,
        int causal, float softcap, const float* dpsum, void* stream, bool det, float p_drop = 0.f,
        unsigned long long seed = 0, int window_left = -1, int window_right = -1, int sinks = 0,
        int (*before_launch)(void*) = nullptr, void* before_ctx = nullptr) {
  if (!q || !k || !v || !dO || !lse || !dq_target || !dk || !dv || !dpsum) return ATTN_ERR_NULL;
  int rc = check_shape(B, H, H_kv, N, d);
  if (rc != ATTN_OK) return rc;
  if (d != 64 && d != 128 && d != 256) return ATTN_ERR_UNSUPPORTED;  // d = 256: its own kernel
  if (!std::isfinite(scale) || scale == 0.f || std::isnan(softcap)) return ATTN_ERR_SHAPE;
  if (!(p_drop >= 0.f && p_drop < 1.f) || sinks < 0) return ATTN_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dO) || !aligned16(lse) ||
      !aligned16(dq_target) || !aligned16(dk) || !aligned16(dv) || !aligned16(dpsum))
    return ATTN_ERR_ALIGN;
  if (B == 0 || H == 0 || N == 0) return ATTN_OK;
  if (d == 256 && before_launch != nullptr) return ATTN_ERR_UNSUPPORTED;
  const Band band = band_of(N, causal, window_left, window_right, sinks);
  if (d == 256) {
    // dQ partials: one tile of 128 query rows per (query block, key block)
    // pair, as for d <= 128
    const long long mb = (N + kBr - 1) / kBr, nb = (N + kBc - 1) / kBc;
    const long long pairs256 = causal ? mb * (mb + 1) / 2 : mb * nb;
    if (det && static_cast<long long>(B) * H * pairs256 > 0x7fffffffLL) return ATTN_ERR_TOO_LARGE;
    return bwd256_run(q, k, v, dO, lse, dq_target, dk, dv, B, H, H_kv, N, scale, causal, softcap,
                      dpsum, band, det, static_cast<int>(pairs256), p_drop, seed,
                      as_stream(stream));
  }

  Params p;
  p.lse = lse;
  p.dpsum = dpsum;
  p.dq_accum = dq_target;
  p.B = B;
  p.H = H;
  p.H_kv = H_kv;
  p.N = N;
  p.n_blocks = (N + kBc - 1) / kBc;
  p.m_blocks = (N + kBr - 1) / kBr;
  const long long units = static_cast<long long>(p.n_blocks) * H_kv * B;
  if (units > 0x7fffffffLL) return ATTN_ERR_TOO_LARGE;
  p.n_units = static_cast<int>(units);
  const long long pairs = causal ? static_cast<long long>(p.m_blocks) * (p.m_blocks + 1) / 2
                                 : static_cast<long long>(p.m_blocks) * p.n_blocks;
  if (det && static_cast<long long>(B) * H * pairs > 0x7fffffffLL) return ATTN_ERR_TOO_LARGE;
  p.pairs = static_cast<int>(pairs);
  p.scale = scale;
  const bool cap = softcap > 0.f;
  p.softcap = cap ? softcap : 0.f;
  p.win_left = band.left;
  p.win_right = band.right;
  // persistent: one CTA per SM (or per unit, if there are fewer units)
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_LAUNCH;
  const int grid = p.n_units < sms ? p.n_units : sms;
  const bool drop = p_drop > 0.f;
  p.drop.seed_lo = static_cast<uint32_t>(seed);
  p.drop.seed_hi = static_cast<uint32_t>(seed >> 32);
  p.drop.threshold = dropout_threshold(p_drop);
  p.drop.inv_keep = 1.f / (1.f - p_drop);
  p.drop.keep = 1.f - p_drop;
  p.drop.log2_inv_keep =
      static_cast<float>(-std::log2(1.0 - static_cast<double>(p_drop)));

  Maps m;
  const long long hq = static_cast<long long>(B) * H, hk = static_cast<long long>(B) * H_kv;
  const bool dq_ok =
      det ? encode_f32_3d(&m.dq, dq_target, d, kBr, hq * pairs, 32, d == 128 ? d : 32)
          : encode_f32_3d(&m.dq, dq_target, d, N, hq, 32, d == 128 ? d : 32);
  if (!encode_bf16_3d(&m.q, q, d, N, hq, kBr) || !encode_bf16_3d(&m.k, k, d, N, hk, kBc) ||
      !encode_bf16_3d(&m.v, v, d, N, hk, kBc) || !encode_bf16_3d(&m.dO, dO, d, N, hq, kBr) ||
      !dq_ok || !encode_bf16_3d(&m.dk, dk, d, N, hk, kBc) ||
      !encode_bf16_3d(&m.dv, dv, d, N, hk, kBc))
    return ATTN_ERR_LAUNCH;

  if (before_launch != nullptr) {
    rc = before_launch(before_ctx);
    if (rc != ATTN_OK) return rc;
  }
  cudaStream_t s = as_stream(stream);
  const bool cs = causal != 0;
  if (band.sinks > 0) return launch_sinks(m, p, band.sinks, dk, dv, d, s);  // no drop, no det
  if (drop) return dispatch<false, true>(m, p, grid, s, d, cs, cap);  // not combined with det
  return det ? dispatch<true, false>(m, p, grid, s, d, cs, cap)
             : dispatch<false, false>(m, p, grid, s, d, cs, cap);
}

}  // namespace bwd
}  // namespace attn

extern "C" int attn_bwd(const void* q, const void* k, const void* v, const void* o,
                        const void* dO, const float* lse, float* dq_accum, void* dk, void* dv,
                        int B, int H, int H_kv, int N, int d, float scale, int causal,
                        float softcap, const float* dpsum, void* stream) {
  (void)o;  // D = rowsum(dO o O) arrives precomputed in dpsum
  return bwd::run(q, k, v, dO, lse, dq_accum, dk, dv, B, H, H_kv, N, d, scale, causal, softcap,
                  dpsum, stream, false);
}

extern "C" int attn_bwd_dropout(const void* q, const void* k, const void* v, const void* o,
                                const void* dO, const float* lse, float* dq_accum, void* dk,
                                void* dv, int B, int H, int H_kv, int N, int d, float scale,
                                int causal, float softcap, const float* dpsum, float p_drop,
                                unsigned long long seed, void* stream) {
  (void)o;
  return bwd::run(q, k, v, dO, lse, dq_accum, dk, dv, B, H, H_kv, N, d, scale, causal, softcap,
                  dpsum, stream, false, p_drop, seed);
}

extern "C" int attn_bwd_local(const void* q, const void* k, const void* v, const void* o,
                              const void* dO, const float* lse, float* dq_accum, void* dk,
                              void* dv, int B, int H, int H_kv, int N, int d, float scale,
                              int causal, float softcap, const float* dpsum, int window_left,
                              int window_right, void* stream) {
  (void)o;
  return bwd::run(q, k, v, dO, lse, dq_accum, dk, dv, B, H, H_kv, N, d, scale, causal, softcap,
                  dpsum, stream, false, 0.f, 0, window_left, window_right);
}

extern "C" int attn_bwd_sinks(const void* q, const void* k, const void* v, const void* o,
                              const void* dO, const float* lse, float* dq_accum, void* dk,
                              void* dv, int B, int H, int H_kv, int N, int d, float scale,
                              int causal, float softcap, const float* dpsum, int window_left,
                              int window_right, int sinks, void* stream) {
  (void)o;
  return bwd::run(q, k, v, dO, lse, dq_accum, dk, dv, B, H, H_kv, N, d, scale, causal, softcap,
                  dpsum, stream, false, 0.f, 0, window_left, window_right, sinks);
}

extern "C" int attn_bwd_deterministic(const void* q, const void* k, const void* v,
                                      const void* o, const void* dO, const float* lse,
                                      float* dq_partials, void* dk, void* dv, int B, int H,
                                      int H_kv, int N, int d, float scale, int causal,
                                      float softcap, const float* dpsum, void* stream) {
  (void)o;
  return bwd::run(q, k, v, dO, lse, dq_partials, dk, dv, B, H, H_kv, N, d, scale, causal,
                  softcap, dpsum, stream, true);
}

namespace attn {

int bwd_run_hooked(const void* q, const void* k, const void* v, const void* dO, const float* lse,
                   float* dq_accum, void* dk, void* dv, int B, int H, int H_kv, int N, int d,
                   float scale, int causal, float softcap, const float* dpsum, void* stream,
                   int (*before_launch)(void*), void* ctx) {
  return bwd::run(q, k, v, dO, lse, dq_accum, dk, dv, B, H, H_kv, N, d, scale, causal, softcap,
                  dpsum, stream, false, 0.f, 0, -1, -1, 0, before_launch, ctx);
}

}  // namespace attn

extern "C" int attn_device_status(int* status, int clear, void* stream) {
  if (!status) return ATTN_ERR_NULL;
  cudaStream_t s = as_stream(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return ATTN_ERR_LAUNCH;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, bwd::g_status, sizeof(int)) != cudaSuccess) return ATTN_ERR_LAUNCH;
  if (clear) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(bwd::g_status, &zero, sizeof(int)) != cudaSuccess)
      return ATTN_ERR_LAUNCH;
  }
  int vf = 0, v256 = 0;  // the forward and d = 256 kernels keep their own words
  if (fwd_status(&vf, clear != 0) != ATTN_OK) return ATTN_ERR_LAUNCH;
  if (bwd256_status(&v256, clear != 0) != ATTN_OK) return ATTN_ERR_LAUNCH;
  int vs = 0, va = 0, vc = 0;  // so do those with sinks and over a paged cache
  if (bwd::sinks_status(&vs, clear != 0) != ATTN_OK) return ATTN_ERR_LAUNCH;
  if (cache_append_status(&va, clear != 0) != ATTN_OK) return ATTN_ERR_LAUNCH;
  if (cache_fwd_status(&vc, clear != 0) != ATTN_OK) return ATTN_ERR_LAUNCH;
  *status = 0;
  for (const int word : {v, vf, v256, vs, va, vc})
    if (*status == 0) *status = word;
  return ATTN_OK;
}

extern "C" int attn_selftest_wait_timeout(int* status, void* stream) {
  if (!status) return ATTN_ERR_NULL;
  cudaStream_t s = as_stream(stream);
  const int zero = 0;
  if (cudaMemcpyToSymbolAsync(bwd::g_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) !=
      cudaSuccess)
    return ATTN_ERR_LAUNCH;
  bwd::wait_timeout_probe<<<1, 64, 0, s>>>(1000000LL);  // about half a millisecond
  const int rc = launch_status();
  if (rc != ATTN_OK) return rc;
  return attn_device_status(status, 1, stream);
}

extern "C" const char* attn_strerror(int code) {
  switch (code) {
    case ATTN_OK: return "success";
    case ATTN_ERR_NULL: return "a required pointer is NULL";
    case ATTN_ERR_SHAPE: return "invalid shape or scalar argument";
    case ATTN_ERR_UNSUPPORTED: return "unsupported head dimension";
    case ATTN_ERR_ALIGN: return "a pointer is not 16-byte aligned";
    case ATTN_ERR_LAUNCH: return "CUDA launch or runtime error";
    case ATTN_ERR_DEVICE_TIMEOUT: return "a kernel timed out waiting on a barrier";
    case ATTN_ERR_DEVICE: return "a kernel detected an internal fault";
    case ATTN_ERR_TOO_LARGE: return "a size exceeds the supported range";
    case ATTN_ERR_PAGE: return "a slot lies outside the page table or the cache";
    default: return "unknown error code";
  }
}
