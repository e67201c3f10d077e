// A ragged batch of new tokens over a paged key/value cache: what the append and
// the attention over the cache share.
//
// Sequence b's new tokens are rows starts[b] .. starts[b + 1] - 1 of the batch's
// T rows, and the last of its lengths[b] positions; position p of it lives in
// slot p mod page_size of page pages[b][p / page_size].
#pragma once

#include <cstdint>

#include "attn_common.cuh"

namespace attn {
namespace cache {

struct Batch {
  const int* starts;   // [B + 1]
  const int* lengths;  // [B]
  const int* pages;    // [B, max_pages]
  int T, B;
  int page_size, max_pages, n_pages;
};

// The sequence that row t belongs to: the largest i in [0, B] with starts[i] <=
// t, or -1 (B: the row lies behind the last sequence). All lanes of a warp come
// with the same t and look at 32 places a step, one load's latency each. Ends for
// any contents of starts (the range shrinks every step).
__device__ __forceinline__ int sequence_of(const Batch& c, int t) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  int lo = 0, hi = c.B + 1;  // starts[lo - 1] <= t, starts[hi] > t
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + lane * step;
    const int n = __popc(__ballot_sync(0xffffffffu, i < hi && c.starts[i] <= t));
    if (n == 0) break;
    hi = min(hi, lo + n * step);
    lo += (n - 1) * step + 1;
  }
  return lo - 1;
}

// Host checks of a batch's description. Returns ATTN_OK or an error code.
inline int check_batch(const Batch& c) {
  if (c.T < 0 || c.B < 0 || c.page_size < 1 || c.max_pages < 0 || c.n_pages < 0)
    return ATTN_ERR_SHAPE;
  if (c.B == 0 || c.T == 0) return ATTN_OK;
  if (!c.starts || !c.lengths || (c.max_pages > 0 && !c.pages)) return ATTN_ERR_NULL;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(c.starts) |
                         reinterpret_cast<uintptr_t>(c.lengths) |
                         reinterpret_cast<uintptr_t>(c.pages);
  return (bits & 3u) != 0 ? ATTN_ERR_ALIGN : ATTN_OK;
}

// `count` element strides of a tensor from a host array (or its dense ones):
// each at least 0, an output's not 0 where elements would share a place, the last
// element's offset below 2^40. A dimension of one element has stride 0.
inline int take_strides(long long* to, const long long* from, const long long* dense,
                        const long long* extent, int count, int d, bool output) {
  bool empty = false;
  for (int i = 0; i < count; ++i) empty = empty || extent[i] == 0;
  long long last = d;
  for (int i = 0; i < count; ++i) {
    const long long s = from != nullptr ? from[i] : dense[i];
    if (s < 0 || (output && s == 0 && extent[i] > 1 && !empty)) return ATTN_ERR_SHAPE;
    to[i] = 0;
    if (extent[i] > 1) {
      if (s >= (1LL << 40) / (extent[i] - 1)) return ATTN_ERR_TOO_LARGE;
      last += s * (extent[i] - 1);
      to[i] = s;
    }
  }
  return last >= (1LL << 40) ? ATTN_ERR_TOO_LARGE : ATTN_OK;
}
// Rows of a ragged batch: (token, head) of [T, heads, d].
inline int row_strides(long long (&to)[2], const long long* from, int T, int heads, int d,
                       bool output) {
  const long long dense[2] = {static_cast<long long>(heads) * d, d};
  const long long extent[2] = {T, heads};
  return take_strides(to, from, dense, extent, 2, d, output);
}
// A cache: (page, slot, head) of [n_pages, page_size, heads, d].
inline int cache_strides(long long (&to)[3], const long long* from, const Batch& c, int heads,
                         int d, bool output) {
  const long long row = static_cast<long long>(heads) * d;
  if (row >= (1LL << 40) / (c.page_size + 1LL)) return ATTN_ERR_TOO_LARGE;
  const long long dense[3] = {row * c.page_size, row, d};
  const long long extent[3] = {c.n_pages, c.page_size, heads};
  return take_strides(to, from, dense, extent, 3, d, output);
}

}  // namespace cache

// Device status words of the append (attn_cache_append.cu) and of the attention
// over the cache (attn_cache_fwd.cu): *status := its value, cleared when `clear`.
int cache_append_status(int* status, bool clear);
int cache_fwd_status(int* status, bool clear);

}  // namespace attn
