// attn_cache_append: the new tokens' keys and values into a paged cache, with the
// rotary positions of q and k applied on the way.
//
// Row t of the batch belongs to the sequence b with starts[b] <= t < starts[b + 1]
// and stands at position p = lengths[b] - (starts[b + 1] - t):
//   q_out[t] = R(p) q[t],  k_cache[slot of p] = R(p) k[t],  v_cache[slot of p] = v[t]
// with R of attn_rotary (m times a rotation of each column pair by p w_i, the
// angle exact for any position). Values are copied bit by bit.
#include <cmath>
#include <cstdint>

#include "cache_common.cuh"
#include "element.cuh"
#include "grid_ptx.cuh"
#include "rotary_core.cuh"

namespace attn {
namespace cache {

__device__ int g_append_status;

struct Append {
  Batch batch;
  const void *q, *k, *v;
  void *q_out, *k_cache, *v_cache;
  long long q_in[2], k_in[2], v_in[2], q_to[2];  // (token, head)
  long long k_to[3], v_to[3];                    // (page, slot, head)
  const unsigned long long* turns;
  int H, H_kv, d, half;
  float magnitude;
};

// Where row t goes: its position, and its page and slot. False for a row behind
// the last sequence. A slot outside the page table, or of a page outside the
// cache, is recorded and leaves page = -1: nothing is written there.
struct Place {
  long long pos;
  int page, slot;
};
__device__ __forceinline__ bool place_of(const Batch& c, int b, int t, bool slots, Place& at) {
  while (b < c.B && c.starts[b + 1] <= t) ++b;
  if (b < 0 || b >= c.B) return false;
  at.pos = static_cast<long long>(c.lengths[b]) -
           (static_cast<long long>(c.starts[b + 1]) - t);
  at.page = -1;
  at.slot = 0;
  if (slots) {
    if (at.pos >= 0 && at.pos < static_cast<long long>(c.max_pages) * c.page_size) {
      const uint32_t p = static_cast<uint32_t>(at.pos), n = static_cast<uint32_t>(c.page_size);
      const int page = c.pages[static_cast<long long>(b) * c.max_pages + p / n];
      if (page >= 0 && page < c.n_pages) {
        at.page = page;
        at.slot = static_cast<int>(p % n);
      }
    }
    if (at.page < 0) atomicCAS(&g_append_status, 0, ATTN_ERR_PAGE);
  }
  return true;
}

template <typename T>
__device__ __forceinline__ T* slot_row(void* cache, const long long (&stride)[3],
                                       const Place& at) {
  return static_cast<T*>(cache) + at.page * stride[0] + at.slot * stride[1];
}

constexpr int kThreads = 128;

// Rows of whole 16-byte groups. As in the rotary kernels a thread keeps the
// angles of one row's two groups and takes them through up to `per` heads of q or
// of k (blockIdx.y); more blocks copy v's groups.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads)
    append_kernel(Append p, int items, int per, int q_groups, int k_groups) {
  ptx::grid_dependency_wait();
  constexpr int E = Vec<T>::kElems, U = 4;
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long row = i / items;
  const int item = static_cast<int>(i - row * items);
  const int t = static_cast<int>(row < p.batch.T ? row : p.batch.T - 1);
  const int b = sequence_of(p.batch, __shfl_sync(0xffffffffu, t, 0));
  if (row >= p.batch.T) return;
  int g = blockIdx.y;
  const bool is_q = g < q_groups;
  Place at;
  if (!place_of(p.batch, b, t, !is_q, at)) return;
  const rotary::Turn turn{p.turns, p.d, p.half, p.magnitude, 1.f, 1.f};
  if (is_q) {
    const int h0 = g * per;
    rotary::rotate_row_heads<T, T, U, INTERLEAVED>(
        turn, static_cast<const T*>(p.q) + t * p.q_in[0] + h0 * p.q_in[1], p.q_in[1],
        static_cast<T*>(p.q_out) + t * p.q_to[0] + h0 * p.q_to[1], p.q_to[1],
        min(per, p.H - h0), item, [&] { return at.pos; });
    return;
  }
  if (at.page < 0) return;
  g -= q_groups;
  if (g < k_groups) {
    const int h0 = g * per;
    rotary::rotate_row_heads<T, T, U, INTERLEAVED>(
        turn, static_cast<const T*>(p.k) + t * p.k_in[0] + h0 * p.k_in[1], p.k_in[1],
        slot_row<T>(p.k_cache, p.k_to, at) + h0 * p.k_to[2], p.k_to[2], min(per, p.H_kv - h0),
        item, [&] { return at.pos; });
    return;
  }
  const int h0 = (g - k_groups) * per, heads = min(per, p.H_kv - h0);
  const T* in = static_cast<const T*>(p.v) + t * p.v_in[0] + h0 * p.v_in[1];
  T* out = slot_row<T>(p.v_cache, p.v_to, at) + h0 * p.v_to[2];
  const int ca = item * E, cb = ca + items * E;
  for (int h = 0; h < heads; h += U) {
    Vec<T> a[U], w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u >= heads) continue;
      a[u] = load_vec(in + (h + u) * p.v_in[1] + ca);
      if (cb < p.d) w[u] = load_vec(in + (h + u) * p.v_in[1] + cb);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u >= heads) continue;
      store_vec(out + (h + u) * p.v_to[2] + ca, a[u]);
      if (cb < p.d) store_vec(out + (h + u) * p.v_to[2] + cb, w[u]);
    }
  }
}

// Any d, strides and rot: one thread per column pair (or copied column) of a row.
template <typename T>
__global__ void __launch_bounds__(256) append_any_kernel(Append p, bool interleaved) {
  ptx::grid_dependency_wait();
  const int items = p.d - p.half, heads = p.H + 2 * p.H_kv;
  const long long total = static_cast<long long>(p.batch.T) * heads * items;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  // whole warps stay together: sequence_of is a warp's
  for (long long first = static_cast<long long>(blockIdx.x) * blockDim.x + (threadIdx.x & ~31u);
       first < total; first += stride) {
    const long long i = first + (threadIdx.x & 31u);
    const int b = sequence_of(p.batch, static_cast<int>(first / items / heads));
    if (i >= total) continue;
    const int j = static_cast<int>(i % items);
    const long long rest = i / items;
    int h = static_cast<int>(rest % heads);
    const int t = static_cast<int>(rest / heads);
    const int which = h < p.H ? 0 : h < p.H + p.H_kv ? 1 : 2;
    Place at;
    if (!place_of(p.batch, b, t, which != 0, at) || (which != 0 && at.page < 0)) continue;
    const T* in;
    T* out;
    if (which == 0) {
      in = static_cast<const T*>(p.q) + t * p.q_in[0] + h * p.q_in[1];
      out = static_cast<T*>(p.q_out) + t * p.q_to[0] + h * p.q_to[1];
    } else if (which == 1) {
      h -= p.H;
      in = static_cast<const T*>(p.k) + t * p.k_in[0] + h * p.k_in[1];
      out = slot_row<T>(p.k_cache, p.k_to, at) + h * p.k_to[2];
    } else {
      h -= p.H + p.H_kv;
      in = static_cast<const T*>(p.v) + t * p.v_in[0] + h * p.v_in[1];
      out = slot_row<T>(p.v_cache, p.v_to, at) + h * p.v_to[2];
    }
    if (j >= p.half) {
      out[j + p.half] = in[j + p.half];
      continue;
    }
    const int ca = interleaved ? 2 * j : j, cb = interleaved ? 2 * j + 1 : j + p.half;
    if (which == 2) {
      out[ca] = in[ca];
      out[cb] = in[cb];
      continue;
    }
    float cs, sn;
    rotary::angle(at.pos, p.turns[j], cs, sn);
    cs *= p.magnitude;
    sn *= p.magnitude;
    const float x = to_f32(in[ca]), y = to_f32(in[cb]);
    out[ca] = from_f32<T>(x * cs - y * sn);
    out[cb] = from_f32<T>(x * sn + y * cs);
  }
}

// Whether rows and strides are whole 16-byte groups (of 2-byte elements).
bool whole_groups(const Append& a, bool interleaved) {
  constexpr int E = 8;
  long long bits = a.d | (interleaved ? 2 * a.half : a.half);
  for (int i = 0; i < 2; ++i) bits |= a.q_in[i] | a.k_in[i] | a.v_in[i] | a.q_to[i];
  for (int i = 0; i < 3; ++i) bits |= a.k_to[i] | a.v_to[i];
  return bits % E == 0;
}

template <typename T>
int launch(const Append& a, bool interleaved, cudaStream_t stream) {
  const int sms = sm_count() > 0 ? sm_count() : 1;
  if (!whole_groups(a, interleaved)) {
    const long long total =
        static_cast<long long>(a.batch.T) * (a.H + 2LL * a.H_kv) * (a.d - a.half);
    const long long want = (total + 255) / 256, cap = sms * 8LL;
    return launch_overlapped(append_any_kernel<T>,
                             dim3(static_cast<unsigned>(want < cap ? want : cap)), 256, 0, 0,
                             stream, a, interleaved);
  }
  constexpr int E = Vec<T>::kElems;
  const int items = (a.d + 2 * E - 1) / (2 * E);
  const long long blocks = (static_cast<long long>(a.batch.T) * items + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return ATTN_ERR_TOO_LARGE;
  // heads per thread: as many as leave every SM a block. Each thread looks its row's
  // sequence, page and angles up, so fewer and longer threads are faster than ones
  // enough for several blocks an SM (device times with one block, and with eight:
  // 23 ragged chunks 3.5 and 6.4 us, 8 of 500 tokens 5.4 and 9.0, 256 of one 3.3 and 5.1).
  int per = 8;
  auto groups = [&](int heads) { return (heads + per - 1) / per; };
  while (per > 1 && blocks * (groups(a.H) + 2 * groups(a.H_kv)) < sms) per /= 2;
  const int qg = groups(a.H), kg = groups(a.H_kv);
  return launch_overlapped(
      interleaved ? append_kernel<T, true> : append_kernel<T, false>,
      dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(qg + 2 * kg)), kThreads, 0, 0,
      stream, a, items, per, qg, kg);
}

}  // namespace cache

int cache_append_status(int* status, bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, cache::g_append_status, sizeof(int)) != cudaSuccess)
    return ATTN_ERR_LAUNCH;
  *status = v;
  const int zero = 0;
  if (clear && v != 0 &&
      cudaMemcpyToSymbol(cache::g_append_status, &zero, sizeof(int)) != cudaSuccess)
    return ATTN_ERR_LAUNCH;
  return ATTN_OK;
}

}  // namespace attn

using namespace attn;

extern "C" int attn_cache_append(const void* q, const void* k, const void* v, void* q_out,
                                 void* k_cache, void* v_cache, const unsigned long long* turns,
                                 const int* starts, const int* lengths, const int* pages, int T,
                                 int B, int H, int H_kv, int d, int rot, float magnitude,
                                 int interleaved, int page_size, int max_pages, int n_pages,
                                 int dtype, const long long* strides, void* stream) {
  cache::Append a{};
  a.batch = {starts, lengths, pages, T, B, page_size, max_pages, n_pages};
  int rc = cache::check_batch(a.batch);
  if (rc != ATTN_OK) return rc;
  if (H < 0 || H_kv < 1 || d < 1 || rot < 0 || rot > d || rot % 2 != 0 ||
      !std::isfinite(magnitude))
    return ATTN_ERR_SHAPE;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_SHAPE;
  const bool empty = T == 0 || B == 0;
  if (!empty && ((H > 0 && (!q || !q_out)) || !k || !v || !k_cache || !v_cache ||
                 (rot > 0 && !turns)))
    return ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(turns))
    return ATTN_ERR_ALIGN;
  if (H > 16384 || H_kv > 16384 || B > (1 << 29) ||
      static_cast<long long>(T) * (H + 2LL * H_kv) >= (1LL << 40) / d)
    return ATTN_ERR_TOO_LARGE;
  auto at = [&](int i) { return strides != nullptr ? strides + i : nullptr; };
  if ((rc = cache::row_strides(a.q_in, at(0), T, H, d, false)) != ATTN_OK ||
      (rc = cache::row_strides(a.k_in, at(2), T, H_kv, d, false)) != ATTN_OK ||
      (rc = cache::row_strides(a.v_in, at(4), T, H_kv, d, false)) != ATTN_OK ||
      (rc = cache::row_strides(a.q_to, at(6), T, H, d, true)) != ATTN_OK ||
      (rc = cache::cache_strides(a.k_to, at(8), a.batch, H_kv, d, true)) != ATTN_OK ||
      (rc = cache::cache_strides(a.v_to, at(11), a.batch, H_kv, d, true)) != ATTN_OK)
    return rc;
  if (empty) return ATTN_OK;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.turns = turns;
  a.H = H;
  a.H_kv = H_kv;
  a.d = d;
  a.half = rot / 2;
  a.magnitude = magnitude;
  return dtype == ATTN_BF16
             ? cache::launch<__nv_bfloat16>(a, interleaved != 0, as_stream(stream))
             : cache::launch<__half>(a, interleaved != 0, as_stream(stream));
}
