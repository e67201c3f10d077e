// attn_cache_fwd: attention of a ragged batch's new tokens over a paged
// key/value cache.
//
// Row t of the batch, at position p of its sequence, and query head h see the keys
// j <= p (or all of the sequence's) with j >= p - left or j < sinks:
//   x_j = logit of q and key j,  O = sum_j e^(x_j - m) v_j / l,
//   l = sum_j e^(x_j - m),  LSE = m + ln l
// with the running maximum m and sum l of one pass over the keys. One warp per
// row and head; its lanes hold d / 32 columns each.
#include <cmath>
#include <cstdint>

#include "cache_common.cuh"
#include "element.cuh"
#include "grid_ptx.cuh"

namespace attn {
namespace cache {

__device__ int g_fwd_status;

struct Fwd {
  Batch batch;
  const void *q, *k, *v;
  void* o;
  float* lse;
  long long q_in[2], o_to[2];        // (token, head)
  long long k_in[3], v_in[3];        // (page, slot, head)
  int H, H_kv;
  float scale, softcap;
  int causal, left, sinks;
};

template <typename T, int D>
__global__ void __launch_bounds__(256) rows_kernel(Fwd p) {
  ptx::grid_dependency_wait();
  constexpr int E = D / 32;
  const Batch& c = p.batch;
  const int lane = threadIdx.x & 31;
  const long long rows = static_cast<long long>(c.T) * p.H;
  for (long long w = blockIdx.x * 8LL + (threadIdx.x >> 5); w < rows; w += gridDim.x * 8LL) {
    const int t = static_cast<int>(w / p.H), h = static_cast<int>(w % p.H);
    const int b = sequence_of(c, t);
    if (b < 0 || b >= c.B) continue;
    const long long cap = static_cast<long long>(c.max_pages) * c.page_size;
    const long long pos = static_cast<long long>(c.lengths[b]) - (c.starts[b + 1] - t);
    long long len = c.lengths[b];
    if (len > cap) {
      len = cap;
      if (lane == 0) atomicCAS(&g_fwd_status, 0, ATTN_ERR_PAGE);
    }
    const long long last = p.causal ? min(pos, len - 1) : len - 1;
    const long long first = p.left < 0 ? 0 : max(0LL, pos - p.left);
    const long long sinks = min(static_cast<long long>(p.sinks), min(first, last + 1));
    float q[E], o[E];
    const T* qr = static_cast<const T*>(p.q) + t * p.q_in[0] + h * p.q_in[1] + lane * E;
    for (int e = 0; e < E; ++e) {
      q[e] = to_f32(qr[e]) * p.scale;
      o[e] = 0.f;
    }
    const int g = h / (p.H / p.H_kv);
    float m = -INFINITY, l = 0.f;
    for (long long j = sinks > 0 ? 0 : first; j <= last; j = j + 1 == sinks ? first : j + 1) {
      const int page = c.pages[static_cast<long long>(b) * c.max_pages + j / c.page_size];
      const int slot = static_cast<int>(j % c.page_size);
      float k[E], v[E];
      const bool ok = page >= 0 && page < c.n_pages;
      if (!ok && lane == 0) atomicCAS(&g_fwd_status, 0, ATTN_ERR_PAGE);
      const T* kr = static_cast<const T*>(p.k) + page * p.k_in[0] + slot * p.k_in[1] +
                    g * p.k_in[2] + lane * E;
      const T* vr = static_cast<const T*>(p.v) + page * p.v_in[0] + slot * p.v_in[1] +
                    g * p.v_in[2] + lane * E;
      float x = 0.f;
      for (int e = 0; e < E; ++e) {
        k[e] = ok ? to_f32(kr[e]) : 0.f;
        v[e] = ok ? to_f32(vr[e]) : 0.f;
        x = fmaf(q[e], k[e], x);
      }
      for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
      if (p.softcap > 0.f) x = p.softcap * tanhf(x / p.softcap);
      const float m_new = fmaxf(m, x);
      const float f = m_new > -INFINITY ? expf(m - m_new) : 1.f;
      const float w1 = m_new > -INFINITY ? expf(x - m_new) : 0.f;
      l = l * f + w1;
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + w1 * v[e];
      m = m_new;
    }
    T* orow = static_cast<T*>(p.o) + t * p.o_to[0] + h * p.o_to[1] + lane * E;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    for (int e = 0; e < E; ++e) orow[e] = from_f32<T>(o[e] * inv);
    if (lane == 0 && p.lse) p.lse[w] = l > 0.f ? m + logf(l) : -INFINITY;
  }
}

template <typename T>
int launch(const Fwd& p, int d, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_LAUNCH;
  const long long want = (static_cast<long long>(p.batch.T) * p.H + 7) / 8;
  const dim3 grid(static_cast<unsigned>(want < sms * 8LL ? want : sms * 8LL));
  if (d == 64) return launch_overlapped(rows_kernel<T, 64>, grid, 256, 0, 0, s, p);
  if (d == 128) return launch_overlapped(rows_kernel<T, 128>, grid, 256, 0, 0, s, p);
  return launch_overlapped(rows_kernel<T, 256>, grid, 256, 0, 0, s, p);
}

}  // namespace cache

int cache_fwd_status(int* status, bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, cache::g_fwd_status, sizeof(int)) != cudaSuccess)
    return ATTN_ERR_LAUNCH;
  *status = v;
  const int zero = 0;
  if (clear && v != 0 &&
      cudaMemcpyToSymbol(cache::g_fwd_status, &zero, sizeof(int)) != cudaSuccess)
    return ATTN_ERR_LAUNCH;
  return ATTN_OK;
}

}  // namespace attn

using namespace attn;

namespace attn {
namespace cache {

// Sizes that both entry points check.
int check_sizes(int T, int B, int H, int H_kv, int d) {
  if (T < 0 || B < 0 || H < 0 || H_kv < 1 || H % H_kv != 0 || d < 1) return ATTN_ERR_SHAPE;
  if (d != 64 && d != 128 && d != 256) return ATTN_ERR_UNSUPPORTED;
  if (H / H_kv > 128) return ATTN_ERR_UNSUPPORTED;
  if (H > 16384 || static_cast<long long>(T) * H >= (1LL << 40) / d) return ATTN_ERR_TOO_LARGE;
  return ATTN_OK;
}

}  // namespace cache
}  // namespace attn

extern "C" long long attn_cache_fwd_workspace_bytes(int T, int B, int H, int H_kv, int d) {
  const int rc = cache::check_sizes(T, B, H, H_kv, d);
  if (rc != ATTN_OK) return rc;
  return 0;
}

extern "C" int attn_cache_fwd(const void* q, const void* k_cache, const void* v_cache, void* o,
                              float* lse, const int* starts, const int* lengths, const int* pages,
                              void* workspace, int T, int B, int H, int H_kv, int d,
                              int page_size, int max_pages, int n_pages, float scale, int causal,
                              float softcap, int window_left, int sinks, int dtype,
                              const long long* strides, void* stream) {
  cache::Fwd p{};
  p.batch = {starts, lengths, pages, T, B, page_size, max_pages, n_pages};
  int rc = cache::check_batch(p.batch);
  if (rc != ATTN_OK) return rc;
  rc = cache::check_sizes(T, B, H, H_kv, d);
  if (rc != ATTN_OK) return rc;
  if (!std::isfinite(scale) || !(scale > 0.f) || std::isnan(softcap) || sinks < 0)
    return ATTN_ERR_SHAPE;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_SHAPE;
  if (page_size % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  const bool empty = T == 0 || B == 0 || H == 0;
  if (!empty && (!q || !k_cache || !v_cache || !o || !workspace)) return ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
      !aligned16(lse) || !aligned16(workspace))
    return ATTN_ERR_ALIGN;
  auto at = [&](int i) { return strides != nullptr ? strides + i : nullptr; };
  if ((rc = cache::row_strides(p.q_in, at(0), T, H, d, false)) != ATTN_OK ||
      (rc = cache::row_strides(p.o_to, at(2), T, H, d, true)) != ATTN_OK ||
      (rc = cache::cache_strides(p.k_in, at(4), p.batch, H_kv, d, false)) != ATTN_OK ||
      (rc = cache::cache_strides(p.v_in, at(7), p.batch, H_kv, d, false)) != ATTN_OK)
    return rc;
  long long bits = 0;
  for (int i = 0; i < 2; ++i) bits |= p.q_in[i] | p.o_to[i];
  for (int i = 0; i < 3; ++i) bits |= p.k_in[i] | p.v_in[i];
  if (bits % 8 != 0) return ATTN_ERR_ALIGN;
  if (empty) return ATTN_OK;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.o = o;
  p.lse = lse;
  p.H = H;
  p.H_kv = H_kv;
  p.scale = scale;
  p.softcap = softcap > 0.f ? softcap : 0.f;
  p.causal = causal != 0;
  p.left = window_left;
  p.sinks = sinks;
  return dtype == ATTN_BF16 ? cache::launch<__nv_bfloat16>(p, d, as_stream(stream))
                            : cache::launch<__half>(p, d, as_stream(stream));
}
