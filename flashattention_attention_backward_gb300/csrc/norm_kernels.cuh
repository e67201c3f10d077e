// The layer-norm kernels for one element type: rows of up to kMaxRow columns
// stay on chip, wider ones are read again.
//
// A row is split over TPR threads in 16-byte vectors: vector j of thread t is
// vector t + j TPR of the row. Where the row length is no multiple of a
// vector (RAGGED), vectors are aligned ones of the whole tensor: a row then
// starts inside its first vector, `shift` elements in, and ends inside its
// last; elements outside the row are left out of the sums and not written.
// Loads and stores stay 16 bytes wide for odd row lengths this way, and the
// generator's groups of four elements stay whole.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "grid_ptx.cuh"
#include "norm_common.cuh"

namespace attn {
namespace norm {

template <int TPR_, int VECS_, int LEAST, int CTAS_ = 1>
struct Shape {
  static constexpr int TPR = TPR_;    // threads of a block per row
  static constexpr int VECS = VECS_;  // 16-byte vectors per thread
  static constexpr int CTAS = CTAS_;  // blocks (of a cluster) per row
  static constexpr int BLOCK = TPR_ < LEAST ? LEAST : TPR_;
  static constexpr int ROWS = BLOCK / TPR_;  // rows of a block at a time
  static constexpr int WARPS = (TPR_ > 32 ? TPR_ / 32 : 1) * CTAS_;  // warps per row
  static constexpr int LANES = TPR_ > 32 ? 32 : TPR_;  // lanes of a warp per row
  // the backward of few rows may be one cluster that needs no second launch
  static constexpr bool FINISH = TPR_ < 32 && BLOCK <= 256;
  static_assert(CTAS_ == 1 || BLOCK / TPR_ == 1, "a cluster has one row");
};

// Barrier over a row's threads (rows of several warps; the block's other rows
// go on by themselves).
template <typename S>
__device__ __forceinline__ void row_barrier() {
  if (S::CTAS > 1)
    ptx::cluster_barrier();
  else if (S::ROWS == 1)
    __syncthreads();
  else
    ptx::named_bar_sync(1 + threadIdx.x / S::TPR, S::TPR);
}
// This block's place among those of a row.
template <typename S>
__device__ __forceinline__ int row_rank() {
  return S::CTAS > 1 ? static_cast<int>(ptx::cluster_rank()) : 0;
}
// This thread's warp among those of its row.
template <typename S>
__device__ __forceinline__ int row_warp() {
  constexpr int kHere = S::WARPS / S::CTAS;
  return row_rank<S>() * kHere + threadIdx.x / 32 % kHere;
}
// Writes a float of the row's, in the shared memory of each of its blocks.
template <typename S>
__device__ __forceinline__ void row_share(float* p, float v) {
  if (S::CTAS == 1) {
    *p = v;
  } else {
#pragma unroll
    for (int i = 0; i < S::CTAS; ++i) ptx::st_cluster_f32(ptx::smem_u32(p), i, v);
  }
}

// The weights (or biases) of a thread's N vectors of E columns, from column
// c(j) on, in fp32 pairs: `fill` where there is no array, 0 outside the row.
// All loads go out before any is used. RAGGED: the columns lie at no vector's
// place, and a thread's own one by one would take as many requests as elements
// with a few bytes of each line; the lanes of a row (LANES of them) read them
// side by side and pass them on through `stage` (32 E floats of the warp's).
template <int N, int E, bool RAGGED, int LANES, typename F>
__device__ __forceinline__ void load_weights(const void* p, int C, int wdtype, float fill, F c,
                                             float* stage, uint64_t (&g)[N][E / 2]) {
  float f[N][E];
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i)
      f[j][i] = static_cast<unsigned>(c(j) + i) < static_cast<unsigned>(C) ? fill : 0.f;
  if (p != nullptr && RAGGED) {
    const int lane = threadIdx.x & 31, t = lane % LANES;
    auto load = [&](auto w) {
      using W = decltype(w);
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int col = c(j) - t * E + i * LANES + t;
          f[j][i] = static_cast<unsigned>(col) < static_cast<unsigned>(C)
                        ? to_f32(static_cast<const W*>(p)[col])
                        : 0.f;
        }
    };
    if (wdtype == ATTN_FP32)
      load(float{});
    else if (wdtype == ATTN_BF16)
      load(__nv_bfloat16{});
    else
      load(__half{});
    float* const at = stage + lane / LANES * LANES * E;
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma unroll
      for (int i = 0; i < E; ++i) at[i * LANES + t] = f[j][i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(at + t * E + i);
        f[j][i] = v.x;
        f[j][i + 1] = v.y;
        f[j][i + 2] = v.z;
        f[j][i + 3] = v.w;
      }
      __syncwarp();
    }
  } else if (p != nullptr && wdtype == ATTN_FP32) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (c(j) >= C) continue;
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c(j) + i);
        f[j][i] = v.x;
        f[j][i + 1] = v.y;
        f[j][i + 2] = v.z;
        f[j][i + 3] = v.w;
      }
    }
  } else if (p != nullptr) {
    uint2 v[N][E / 4];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (c(j) >= C) continue;
#pragma unroll
      for (int i = 0; i < E / 4; ++i)
        v[j][i] = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c(j) + 4 * i);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (c(j) >= C) continue;
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const uint32_t w = i % 2 == 0 ? v[j][i / 2].x : v[j][i / 2].y;
        const float2 h = wdtype == ATTN_BF16
                             ? make_float2(__uint_as_float(w << 16),
                                           __uint_as_float(w & 0xffff0000u))
                             : __half22float2(*reinterpret_cast<const __half2*>(&w));
        f[j][2 * i] = h.x;
        f[j][2 * i + 1] = h.y;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < E / 2; ++i) g[j][i] = ptx::f2_make(f[j][2 * i], f[j][2 * i + 1]);
}

// Writes the elements of a vector that reach over the row's ends: the last
// ones (start of a row) or the first ones (end of a row) in pieces of four,
// two and one element of 16 bits, or two and one of 32 bits.
template <typename T>
__device__ __forceinline__ void store_edge(T* p, const Vec<T>& v, int c, int C) {
  constexpr int E = Vec<T>::kElems;
  const uint32_t w[4] = {v.w.x, v.w.y, v.w.z, v.w.w};
  if (c < 0 && c + E > C) {  // a row inside one vector
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (static_cast<unsigned>(c + i) < static_cast<unsigned>(C)) p[i] = e[i];
    return;
  }
  const bool start = c < 0;
  const int n = start ? E + c : C - c;  // elements in the row
  uint32_t* const q = reinterpret_cast<uint32_t*>(p);
  if (E == 4) {
    if (n & 2)
      *reinterpret_cast<uint2*>(q + (start ? 2 : 0)) =
          start ? make_uint2(w[2], w[3]) : make_uint2(w[0], w[1]);
    if (n & 1) {
      const int i = start ? 4 - n : n - 1;
      q[i] = i < 2 ? (i == 0 ? w[0] : w[1]) : (i == 2 ? w[2] : w[3]);
    }
  } else {
    if (n & 4)
      *reinterpret_cast<uint2*>(q + (start ? 2 : 0)) =
          start ? make_uint2(w[2], w[3]) : make_uint2(w[0], w[1]);
    if (n & 2) {
      const int i = start ? (n & 4 ? 1 : 3) : (n & 4 ? 2 : 0);
      q[i] = i < 2 ? (i == 0 ? w[0] : w[1]) : (i == 2 ? w[2] : w[3]);
    }
    if (n & 1) {
      const int i = start ? 8 - n : n - 1;  // odd at the start of a row, even at its end
      const uint32_t x = i < 4 ? (i < 2 ? w[0] : w[1]) : (i < 6 ? w[2] : w[3]);
      reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(start ? x >> 16 : x);
    }
  }
}

// Writes the vector's elements that lie in the row; edge: it reaches over the
// row's ends.
template <typename T, int E>
__device__ __forceinline__ void store_row_vec(T* p, const float (&f)[E], bool edge, int c, int C) {
  Vec<T> v;
  pack(f, v);
  if (!edge)
    store_vec(p, v);
  else
    store_edge(p, v, c, C);
}

__device__ __forceinline__ void copy_async16(uint32_t smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(global) : "memory");
}
// The first `bytes` of them, zeros behind.
__device__ __forceinline__ void copy_async16(uint32_t smem, const void* global, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(global), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// How the rows fall to the grid's places for one (blocks times rows of threads
// a block): `whole` to each, one more to the first `rest`.
struct Split {
  int whole;
  long long rest;
};

// A block's walk over rows, shared by the two kernels: blocks stay and take
// rows a grid apart, so that a thread's columns are the same in all of its
// rows (RAGGED: the grid is a multiple of 8 blocks, so all of a thread's rows
// start at the same offset within a vector), and its weights, or its sums of
// the weights' gradients, stay in registers. Rows of NT tensors come through
// a ring of STAGES in shared memory, filled by asynchronous copies: a thread
// reads back only what it copied itself, so the ring needs no barrier, and
// the next rows' loads run while these are reduced. A turn takes R rows, whose
// chains of dependent steps (sums over lanes, the barrier) then overlap.
// Vectors outside the row read as zeros, rows behind the last too.
template <typename T, typename S, int STAGES, int R, int NT, bool RAGGED>
struct Walk {
  static constexpr int E = Vec<T>::kElems;
  static constexpr int kAhead = STAGES - R;               // rows being copied
  static constexpr int kStage = NT * S::VECS * S::BLOCK;  // slots of a stage
  static_assert(STAGES % R == 0 && kAhead >= 0, "a turn's rows lie side by side in the ring");
  uint4* ring;        // this thread's slots: [STAGES][NT][VECS], BLOCK apart
  const T* from[NT];  // vector 0 of the next row to copy
  int edges;          // bits: vectors that reach over the row's ends (RAGGED)
  long long stride;   // elements between this thread's rows
  long long e;        // element of the turn's first row's vector 0
  long long row, step;
  int left, to_copy;  // this thread's rows still to come, and to be copied
  int t, shift, C;
  int fill, take;     // where the stages begin

  __device__ __forceinline__ Walk(uint4* smem, const void* const (&src)[NT], int C_,
                                  const Split& split)
      : ring(smem + threadIdx.x), C(C_), fill(0), take(0) {
    row = static_cast<long long>(blockIdx.x) / S::CTAS * S::ROWS + threadIdx.x / S::TPR;
    step = static_cast<long long>(gridDim.x) / S::CTAS * S::ROWS;
    shift = RAGGED ? static_cast<int>((row * C) & (E - 1)) : 0;
    t = threadIdx.x % S::TPR + row_rank<S>() * (S::TPR * S::VECS);
    e = row * C - shift + t * E;
    stride = step * C;
    left = split.whole + (row < split.rest);
    to_copy = left;
    edges = 0;
#pragma unroll
    for (int j = 0; j < S::VECS; ++j)
      if (RAGGED && inside(j) && (column(j) < 0 || column(j) + E > C)) edges |= 1 << j;
#pragma unroll
    for (int q = 0; q < NT; ++q) from[q] = static_cast<const T*>(src[q]) + e;
#pragma unroll
    for (int j = 0; j < S::VECS; ++j)
      if (!inside(j))
        for (int k = 0; k < STAGES * NT; ++k)
          ring[(k * S::VECS + j) * S::BLOCK] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) copy_next();
  }
  // the first column of this thread's vector j; below 0, or less than a
  // vector from the row's end, it reaches over the row's ends (RAGGED)
  __device__ __forceinline__ int column(int j) const { return (t + j * S::TPR) * E - shift; }
  __device__ __forceinline__ bool inside(int j) const { return column(j) < C; }
  __device__ __forceinline__ bool edge(int j) const { return RAGGED && (edges >> j & 1) != 0; }
  // element of vector j, less that of vector 0
  __device__ __forceinline__ static constexpr int offset(int j) { return j * S::TPR * E; }
  // rows to take: this thread's; where several rows share a warp, the most
  // that one of the block's threads has
  __device__ __forceinline__ int count(const Split& split) const {
    if (S::TPR >= 32) return left;
    return split.whole + (static_cast<long long>(blockIdx.x) * S::ROWS < split.rest);
  }
  // whether the turn's k-th row is one
  __device__ __forceinline__ bool active(int k) const {
    return (k == 0 && S::TPR >= 32) || left > k;
  }

  __device__ __forceinline__ void copy_next() {
    uint4* to = ring + fill;
    if (to_copy > 0) {
#pragma unroll
      for (int j = 0; j < S::VECS; ++j) {
        if (inside(j)) {
#pragma unroll
          for (int q = 0; q < NT; ++q) {
            uint4* slot = to + (q * S::VECS + j) * S::BLOCK;
            const T* p = from[q] + offset(j);
            if (RAGGED)  // not behind the row, which may be the tensor's last
              copy_async16(ptx::smem_u32(slot), p,
                           min(C - column(j), E) * static_cast<int>(sizeof(T)));
            else
              copy_async16(ptx::smem_u32(slot), p);
          }
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < NT * S::VECS; ++k) to[k * S::BLOCK] = make_uint4(0u, 0u, 0u, 0u);
    }
    copy_commit();
    --to_copy;
#pragma unroll
    for (int q = 0; q < NT; ++q) from[q] += stride;
    fill = fill == (STAGES - 1) * kStage ? 0 : fill + kStage;
  }
  // starts the next copies and waits for the turn's N rows (R of them, fewer
  // in the last turn); of the first `trimmed` tensors, what the first vector
  // has of the row before becomes zero
  template <int N>
  __device__ __forceinline__ void arrive(int trimmed) {
#pragma unroll
    for (int k = 0; k < N; ++k) copy_next();
    copy_wait<kAhead>();
    if (RAGGED && column(0) < 0) {
      uint32_t m[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (column(0) + i >= 0)
          m[i * 4 / E] |= sizeof(T) == 4 ? 0xffffffffu : (i % 2 == 0 ? 0xffffu : 0xffff0000u);
#pragma unroll
      for (int k = 0; k < N; ++k)
        for (int q = 0; q < trimmed; ++q) {
          uint4& v = ring[take + k * kStage + q * S::VECS * S::BLOCK];
          v = make_uint4(v.x & m[0], v.y & m[1], v.z & m[2], v.w & m[3]);
        }
    }
  }
  // vector j of tensor q of the turn's k-th row
  __device__ __forceinline__ void get(int k, int q, int j, float (&f)[E]) const {
    Vec<T> v;
    v.w = ring[take + k * kStage + (q * S::VECS + j) * S::BLOCK];
    unpack(v, f);
  }
  __device__ __forceinline__ void next() {
    row += R * step;
    e += R * stride;
    left -= R;
    take = take == (STAGES - R) * kStage ? 0 : take + R * kStage;
  }
};

// Sum over groups of W lanes, the same value in each.
template <int W>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int off = W / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// R values to sum over a warp's lanes, R = 1, 2 or 4. While more than one is
// left a lane hands half of them to its partner and keeps the others, so that
// R values take few more exchanges than one: 5, 5 or 6 instead of 5, 10 or 20.
// A lane ends with the sum of value lane / (32 / R).
template <int R>
__device__ __forceinline__ float warp_sums(float (&v)[R]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = R; n > 1; n /= 2) {
    const int off = 16 * n / R;
    const bool low = (lane & off) == 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = low ? v[n / 2 + i] : v[i];
      v[i] = (low ? v[i] : v[n / 2 + i]) + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
#pragma unroll
  for (int off = 16 / R; off >= 1; off /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
  return v[0];
}

// Sum of R values over a row's threads, the same in each; all R at a time.
// `part` has R * WARPS floats of the row's own. One barrier.
template <typename S, int R>
__device__ __forceinline__ void row_sums(float (&v)[R], float* part) {
  if (S::WARPS == 1) {
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = lane_sum<S::LANES>(v[i]);
    return;
  }
  const int lane = threadIdx.x & 31;
  const float mine = warp_sums<R>(v);
  if (lane % (32 / R) == 0)
    row_share<S>(part + lane / (32 / R) * S::WARPS + row_warp<S>(), mine);
  row_barrier<S>();
  // a group of lanes adds up each value's parts
  constexpr int kGroup = S::WARPS < 32 / R ? S::WARPS : 32 / R;
  const float* p = part + lane / kGroup % R * S::WARPS + lane % kGroup;
  float sum = p[0];
#pragma unroll
  for (int i = kGroup; i < S::WARPS; i += kGroup) sum += p[i];
  sum = lane_sum<kGroup>(sum);
#pragma unroll
  for (int i = 0; i < R; ++i) v[i] = R == 1 ? sum : __shfl_sync(0xffffffffu, sum, i * kGroup);
}

// s / n, rounded to nearest (Markstein, 1990: a product with the rounded
// reciprocal, corrected by its exact remainder); infinities and NaN stay.
__device__ __forceinline__ float quotient(float s, float n, float inv_n) {
  const float q = s * inv_n;
  const float nearest = fmaf(fmaf(-q, n, s), inv_n, q);
  return fabsf(q) < __int_as_float(0x7f800000) ? nearest : q;
}

// Forward: a row (its sum with the residual, behind the dropout) is held in
// fp32 registers, in pairs (one instruction for two columns). A warp takes the
// mean of its part and the squares about that; parts of n_w elements are
// joined by
//   mu = sum n_w mu_w / C,  sum of squares = sum (q_w + n_w (mu_w - mu)^2),
// which loses nothing to cancellation and costs one barrier a turn of R rows.
// Means are quotients, not products with 1 / C: a row of equal values whose sums
// are exact has that value as its mean, and y = beta. The root's reciprocal is the
// hardware's, 2 steps of 2^-24 to 2^-23: rounded to nearest (__frsqrt_rn) the
// forward takes 1 to 5 % longer (60000 x 333 31.6 us, 30.0).
// ADD: with a residual, and z written.
// Bound by HBM: 8192 x 4096 bf16 takes 22.7 us for 134 MB (5.9 TB/s), with
// residual and dropout 49.1 us for 269 MB (5.5 TB/s; half of the cycles issue,
// and dropping costs 1 us of it). One row a turn took 3 us more, and three
// blocks of 256 threads at 80 registers, not two at 128, 66 us with dropout and
// the same without.
template <typename T, typename S, int STAGES, int R, bool ADD, bool DROP, bool RAGGED>
__global__ void __launch_bounds__(S::BLOCK, S::BLOCK <= 256 ? 2 : 1)
    fwd_kernel(FwdArgs a, Split split) {
  ptx::grid_dependency_wait();
  constexpr int E = Vec<T>::kElems, VECS = S::VECS, P = E / 2, NT = ADD ? 2 : 1;
  constexpr int kLanes = S::LANES, kWarps = S::WARPS;
  // a block behind the last row (the grid comes in eights)
  if (split.whole == 0 && blockIdx.x / S::CTAS * S::ROWS >= split.rest) return;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float2 parts[S::ROWS][2][R * kWarps];
  __shared__ float all_counts[S::ROWS][kWarps];
  auto& part = parts[kWarps > 1 ? threadIdx.x / S::TPR : 0];
  auto& counts = all_counts[kWarps > 1 ? threadIdx.x / S::TPR : 0];
  const int lane = threadIdx.x & 31, warp = row_warp<S>();
  const void* src[NT];
  src[0] = a.x;
  if (ADD) src[NT - 1] = a.residual;
  Walk<T, S, STAGES, R, NT, RAGGED> w(ring, src, a.C, split);
  const float C = static_cast<float>(a.C), inv_C = 1.0f / C;
  uint64_t gamma[VECS][P], beta[VECS][P];
  __shared__ __align__(16) float stages[RAGGED ? S::BLOCK / 32 : 1][32 * E];
  float* const stage = stages[RAGGED ? threadIdx.x / 32 : 0];
  auto column = [&](int j) { return w.column(j); };
  load_weights<VECS, E, RAGGED, kLanes>(a.gamma, a.C, a.wdtype, 1.f, column, stage, gamma);
  load_weights<VECS, E, RAGGED, kLanes>(a.beta, a.C, a.wdtype, 0.f, column, stage, beta);
  int mine = 0;  // this thread's columns inside the row
#pragma unroll
  for (int j = 0; j < VECS; ++j)
    if (w.inside(j)) mine += RAGGED ? min(w.column(j) + E, a.C) - max(w.column(j), 0) : E;
  const float count = lane_sum<kLanes>(static_cast<float>(mine));  // n_w
  const float inv_count = count > 0.f ? 1.0f / count : 0.f;
  if (kWarps > 1) {
    if (S::CTAS > 1) ptx::cluster_barrier();  // all of the cluster's blocks have begun
    if (lane == 0) row_share<S>(&counts[warp], count);
    row_barrier<S>();
  }
  const uint64_t inv_keep = ptx::f2_make(a.drop.inv_keep, a.drop.inv_keep);
  int parity = 0;
  auto turn = [&](auto rows_of_turn) {
    constexpr int N = decltype(rows_of_turn)::value;
    // the parts that a lane joins: of the turn's row lane / kGroup
    constexpr int kGroup = kWarps < 32 / N ? kWarps : 32 / N;
    w.template arrive<N>(NT);
    uint64_t v[N][VECS][P];
    float mu[N], q[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      uint64_t s2 = 0;
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        const long long e = w.e + k * w.stride + w.offset(j);
        float f[E];
        w.get(k, 0, j, f);
        if (DROP) drop_vec<E>(f, e, a.drop);
#pragma unroll
        for (int i = 0; i < P; ++i) v[k][j][i] = ptx::f2_make(f[2 * i], f[2 * i + 1]);
        if (ADD) {
          float r[E];
          w.get(k, NT - 1, j, r);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const uint64_t r2 = ptx::f2_make(r[2 * i], r[2 * i + 1]);
            v[k][j][i] = DROP ? ptx::f2_fma(v[k][j][i], inv_keep, r2) : ptx::f2_add(v[k][j][i], r2);
            f[2 * i] = ptx::f2_lo(v[k][j][i]);
            f[2 * i + 1] = ptx::f2_hi(v[k][j][i]);
          }
          if (w.active(k) && w.inside(j))
            store_row_vec(static_cast<T*>(a.z) + e, f, w.edge(j), w.column(j), a.C);
        }
#pragma unroll
        for (int i = 0; i < P; ++i) s2 = ptx::f2_add(s2, v[k][j][i]);
      }
      mu[k] = ptx::f2_lo(s2) + ptx::f2_hi(s2);
    }
    if (kWarps > 1 && N > 1) {
      const float mean = quotient(warp_sums<N>(mu), count, inv_count);
#pragma unroll
      for (int k = 0; k < N; ++k) mu[k] = __shfl_sync(0xffffffffu, mean, k * (32 / N));
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) mu[k] = quotient(lane_sum<kLanes>(mu[k]), count, inv_count);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      uint64_t q2 = 0;
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        if (w.edge(j)) {  // partly outside: mu in place of its zeros there
          const int c = w.column(j);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const bool lo = static_cast<unsigned>(c + 2 * i) < static_cast<unsigned>(a.C);
            const bool hi = static_cast<unsigned>(c + 2 * i + 1) < static_cast<unsigned>(a.C);
            v[k][j][i] = ptx::f2_make(lo ? ptx::f2_lo(v[k][j][i]) : mu[k],
                                      hi ? ptx::f2_hi(v[k][j][i]) : mu[k]);
          }
        }
        const float m = w.inside(j) ? -mu[k] : 0.f;  // outside the row v is 0
        const uint64_t minus = ptx::f2_make(m, m);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const uint64_t d = ptx::f2_add(v[k][j][i], minus);
          q2 = ptx::f2_fma(d, d, q2);
        }
      }
      q[k] = ptx::f2_lo(q2) + ptx::f2_hi(q2);
    }
    float rstd[N];
    if (kWarps > 1) {
      const float sum = warp_sums<N>(q);
      float mean = mu[0];  // of the row that this lane's sum belongs to
#pragma unroll
      for (int k = 1; k < N; ++k) mean = lane / (32 / N) == k ? mu[k] : mean;
      if (lane % (32 / N) == 0) {
        float2* to = &part[parity][lane / (32 / N) * kWarps + warp];
        row_share<S>(&to->x, mean);
        row_share<S>(&to->y, sum);
      }
      row_barrier<S>();
      // a group of lanes joins each row's parts
      const int first = lane / kGroup % N * kWarps + lane % kGroup;
      const float* n = &counts[lane % kGroup];
      float2 p[kWarps / kGroup];
      float total = 0.f, squares = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps / kGroup; ++i) {
        p[i] = part[parity][first + i * kGroup];
        total = fmaf(n[i * kGroup], p[i].x, total);
      }
      total = quotient(lane_sum<kGroup>(total), C, inv_C);
#pragma unroll
      for (int i = 0; i < kWarps / kGroup; ++i) {
        const float d = p[i].x - total, c = n[i * kGroup];
        squares += c > 0.f ? fmaf(c * d, d, p[i].y) : 0.f;
      }
      squares = lane_sum<kGroup>(squares);
      const float r = rsqrtf(fmaf(squares, inv_C, a.eps));
#pragma unroll
      for (int k = 0; k < N; ++k) {
        mu[k] = N == 1 ? total : __shfl_sync(0xffffffffu, total, k * kGroup);
        rstd[k] = N == 1 ? r : __shfl_sync(0xffffffffu, r, k * kGroup);
      }
      parity ^= 1;
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) rstd[k] = rsqrtf(fmaf(lane_sum<kLanes>(q[k]), inv_C, a.eps));
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint64_t minus_mu = ptx::f2_make(-mu[k], -mu[k]), r2 = ptx::f2_make(rstd[k], rstd[k]);
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        float f[E];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const uint64_t h = ptx::f2_mul(ptx::f2_add(v[k][j][i], minus_mu), r2);
          const uint64_t o = ptx::f2_fma(h, gamma[j][i], beta[j][i]);
          f[2 * i] = ptx::f2_lo(o);
          f[2 * i + 1] = ptx::f2_hi(o);
        }
        if (w.active(k) && w.inside(j))
          store_row_vec(static_cast<T*>(a.y) + w.e + k * w.stride + w.offset(j), f, w.edge(j),
                        w.column(j), a.C);
      }
      if (w.active(k) && w.t == 0) {
        if (a.mean != nullptr) a.mean[w.row + k * w.step] = mu[k];
        if (a.rstd != nullptr) a.rstd[w.row + k * w.step] = rstd[k];
      }
    }
  };
  int count_down = w.count(split);
  for (; count_down >= R; count_down -= R, w.next()) turn(std::integral_constant<int, R>{});
  if (R > 1 && count_down > 0) turn(std::integral_constant<int, 1>{});
  copy_wait<0>();
}

// Backward: first the turn's rows' two sums each and their part of the
// weights' gradients, whose column sums stay in registers over all of the
// thread's rows; then, with the sums joined over the rows' threads, the rows'
// gradients, from the ring again. DZ: with a dz to add.
// 8192 x 4096 bf16: 36.8 us for 201 MB, of which 31.6 the rows' gradients (6.4
// TB/s) and the rest the weights' (their second stage, and the partial sums);
// with dz and dropout 58.5 us for 336 MB (5.8 TB/s), bound by issue and the
// multiply pipe (59 % of the cycles issue) about as much as by HBM. A row at a
// time took 45 and 69 us; 64 registers for twice the threads 44 and 82.
template <typename T, typename S, int STAGES, int R, bool DZ, bool DROP, bool RAGGED>
__global__ void __launch_bounds__(S::BLOCK, S::BLOCK <= 256 ? 3 : 1)
    bwd_kernel(BwdArgs a, Split split) {
  constexpr int E = Vec<T>::kElems, VECS = S::VECS, BLOCK = S::BLOCK, P = E / 2;
  constexpr int NT = DZ ? 3 : 2;
  ptx::grid_dependency_wait();
  ptx::grid_dependency_launch();  // the second stage's launch, which waits for this grid's end
  // a block behind the last row (the grid comes in eights)
  if (split.whole == 0 && blockIdx.x / S::CTAS * S::ROWS >= split.rest &&
      !(S::FINISH && a.finish != 0))
    return;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float parts[S::ROWS][2][2 * R * S::WARPS];
  auto& part = parts[S::WARPS > 1 ? threadIdx.x / S::TPR : 0];
  const void* src[NT];
  src[0] = a.dy;
  src[1] = a.z;
  if (DZ) src[NT - 1] = a.dz;
  Walk<T, S, STAGES, R, NT, RAGGED> w(ring, src, a.C, split);
  const float inv_C = 1.0f / static_cast<float>(a.C);
  // the statistics of the rows to come, one turn ahead
  float mu_next[R], r_next[R];
  auto statistics = [&](int ahead) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mu_next[k] = r_next[k] = 0.f;
      if (w.left > ahead + k) {
        mu_next[k] = a.mean[w.row + (ahead + k) * w.step];
        r_next[k] = a.rstd[w.row + (ahead + k) * w.step];
      }
    }
  };
  statistics(0);
  uint64_t dgamma[VECS][P], dbeta[VECS][P], gamma[VECS][P];
#pragma unroll
  for (int j = 0; j < VECS; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) dgamma[j][i] = dbeta[j][i] = 0;
  __shared__ __align__(16) float stages[RAGGED ? S::BLOCK / 32 : 1][32 * E];
  load_weights<VECS, E, RAGGED, S::LANES>(
      a.gamma, a.C, a.wdtype, 1.f, [&](int j) { return w.column(j); },
      stages[RAGGED ? threadIdx.x / 32 : 0], gamma);
  const uint64_t inv_keep = ptx::f2_make(a.drop.inv_keep, a.drop.inv_keep);
  // dy and z - mean of vector j of the turn's k-th row (dy = 0 outside the row)
  auto gather = [&](int k, int j, float mu, uint64_t (&dy)[P], uint64_t (&d)[P]) {
    float fd[E], fz[E];
    w.get(k, 0, j, fd);
    w.get(k, 1, j, fz);
    const uint64_t minus_mu = ptx::f2_make(-mu, -mu);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      dy[i] = ptx::f2_make(fd[2 * i], fd[2 * i + 1]);
      d[i] = ptx::f2_add(ptx::f2_make(fz[2 * i], fz[2 * i + 1]), minus_mu);
    }
  };
  if (S::CTAS > 1) ptx::cluster_barrier();  // all of the cluster's blocks have begun
  int parity = 0;
  auto turn = [&](auto rows_of_turn) {
    constexpr int N = decltype(rows_of_turn)::value;
    float mu[N], r[N], sums[2 * N];  // of row k: sum dy gamma, sum dy (z - mean) gamma
#pragma unroll
    for (int k = 0; k < N; ++k) {
      mu[k] = mu_next[k];
      r[k] = r_next[k];
    }
    statistics(R);
    w.template arrive<N>(2);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint64_t r2 = ptx::f2_make(r[k], r[k]);
      uint64_t s2 = 0, u2 = 0;
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        uint64_t dy[P], d[P];
        gather(k, j, mu[k], dy, d);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const uint64_t t = ptx::f2_mul(dy[i], d[i]);
          dgamma[j][i] = ptx::f2_fma(t, r2, dgamma[j][i]);
          dbeta[j][i] = ptx::f2_add(dbeta[j][i], dy[i]);
          s2 = ptx::f2_fma(dy[i], gamma[j][i], s2);
          u2 = ptx::f2_fma(t, gamma[j][i], u2);
        }
      }
      sums[2 * k] = ptx::f2_lo(s2) + ptx::f2_hi(s2);
      sums[2 * k + 1] = ptx::f2_lo(u2) + ptx::f2_hi(u2);
    }
    row_sums<S, 2 * N>(sums, part[parity]);
    parity ^= 1;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      // dz = r g - r (r u / C) h - r s / C + dz_in, h = (z - mean) r
      const float rs = -r[k] * (sums[2 * k] * inv_C);
      const float ru = -r[k] * (r[k] * sums[2 * k + 1] * inv_C);
      const uint64_t r2 = ptx::f2_make(r[k], r[k]);
      const uint64_t rs2 = ptx::f2_make(rs, rs), ru2 = ptx::f2_make(ru, ru);
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        const int c = w.column(j);
        const long long e = w.e + k * w.stride + w.offset(j);
        uint64_t dy[P], d[P];
        gather(k, j, mu[k], dy, d);
        float f[E];
        if (DZ) w.get(k, NT - 1, j, f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const uint64_t g = ptx::f2_mul(dy[i], gamma[j][i]);
          dy[i] = ptx::f2_fma(g, r2, ptx::f2_fma(ptx::f2_mul(d[i], r2), ru2, rs2));
          if (DZ) dy[i] = ptx::f2_add(dy[i], ptx::f2_make(f[2 * i], f[2 * i + 1]));
          f[2 * i] = ptx::f2_lo(dy[i]);
          f[2 * i + 1] = ptx::f2_hi(dy[i]);
        }
        const bool write = w.active(k) && w.inside(j);
        if (write) store_row_vec(static_cast<T*>(a.dres) + e, f, w.edge(j), c, a.C);
        if (DROP) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            dy[i] = ptx::f2_mul(dy[i], inv_keep);
            f[2 * i] = ptx::f2_lo(dy[i]);
            f[2 * i + 1] = ptx::f2_hi(dy[i]);
          }
          drop_vec<E>(f, e, a.drop);
        }
        if ((DROP || a.dx != nullptr) && write)
          store_row_vec(static_cast<T*>(a.dx) + e, f, w.edge(j), c, a.C);
      }
    }
  };
  int count_down = w.count(split);
  for (; count_down >= R; count_down -= R, w.next()) turn(std::integral_constant<int, R>{});
  if (R > 1 && count_down > 0) turn(std::integral_constant<int, 1>{});
  copy_wait<0>();
  if (a.workspace == nullptr) return;
  // This thread's sums go side by side with those of the block's other rows of
  // threads to the ring's memory, where each column is added up over them in
  // order; straight to the workspace where there is one row of threads. RAGGED:
  // a thread's columns are at no vector's place and go one by one, a word of
  // distance behind every eight so that the lanes' banks differ. Where the grid
  // is one cluster, its blocks then add theirs up, each a part of the columns:
  // few rows need no second launch.
  float* const out = a.workspace + 2LL * (blockIdx.x / S::CTAS) * a.C;
  float* const sums = reinterpret_cast<float*>(ring);
  constexpr bool kGather = S::ROWS > 1 || (RAGGED && S::CTAS == 1);
  auto place = [](int i) { return RAGGED && kGather ? i + (i >> 3) : i; };
  const int size = place(2 * a.C);
  float* const own = kGather ? sums + threadIdx.x / S::TPR * size : out;
  if (kGather) __syncthreads();
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int c = w.column(j);
    if (c >= a.C) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint64_t(&v)[P] = half == 0 ? dgamma[j] : dbeta[j];
      const int first = half * a.C + c;
      if (!RAGGED) {  // columns and C are multiples of four
#pragma unroll
        for (int i = 0; i < P; i += 2)
          *reinterpret_cast<float4*>(own + first + 2 * i) =
              make_float4(ptx::f2_lo(v[i]), ptx::f2_hi(v[i]), ptx::f2_lo(v[i + 1]),
                          ptx::f2_hi(v[i + 1]));
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (static_cast<unsigned>(c + i) < static_cast<unsigned>(a.C))
            own[place(first + i)] = i % 2 == 0 ? ptx::f2_lo(v[i / 2]) : ptx::f2_hi(v[i / 2]);
      }
    }
  }
  if (kGather) {
    // rows of threads that had rows
    const long long first = static_cast<long long>(blockIdx.x) * S::ROWS;
    const int n = split.whole > 0 || split.rest - first > S::ROWS
                      ? S::ROWS
                      : static_cast<int>(split.rest - first);
    __syncthreads();
    if (S::FINISH && a.finish != 0) {
      for (int i = threadIdx.x; i < 2 * a.C; i += BLOCK) {
        float v = 0.f;
#pragma unroll 4
        for (int k = 0; k < n; ++k) v += sums[k * size + place(i)];
        sums[place(i)] = v;  // column i is this thread's alone
      }
      ptx::cluster_barrier();
      for (int i = blockIdx.x * BLOCK + threadIdx.x; i < 2 * a.C; i += gridDim.x * BLOCK) {
        float part[8], v = 0.f;  // (a cluster has eight blocks at most)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          part[k] = k < static_cast<int>(gridDim.x)
                        ? ptx::ld_cluster_f32(ptx::smem_u32(sums + place(i)), k)
                        : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) v += part[k];
        void* const to = i < a.C ? a.dgamma : a.dbeta;
        if (to != nullptr) store_as(to, i < a.C ? i : i - a.C, a.wdtype, v);
      }
      ptx::cluster_barrier();  // no block leaves while another reads its sums
    } else if (!RAGGED) {
      for (int i = threadIdx.x; i < a.C / 2; i += BLOCK) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
          const float4 x = *reinterpret_cast<const float4*>(sums + k * size + 4 * i);
          v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
        }
        *reinterpret_cast<float4*>(out + 4 * i) = v;
      }
    } else {
      for (int i = threadIdx.x; i < 2 * a.C; i += BLOCK) {
        float v = 0.f;
#pragma unroll 4
        for (int k = 0; k < n; ++k) v += sums[k * size + place(i)];
        out[i] = v;
      }
    }
  }
}

// Sum over the block, the same value in every thread.
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += part[i];
  return s;
}

// Sums of N values f(c, values) over a row's columns c, the same in every
// thread of the block. A thread takes eight columns at a time, if TOGETHER their
// loads in flight together, and its sums go up two levels of 16 to one, so that
// a term takes part in at most 40 + C / 2^19 additions of the thread's and 13 of
// the block's, not in C / 256 in a row.
template <bool TOGETHER, int N, typename F>
__device__ __forceinline__ void wide_sums(int C, F f, float (&sum)[N]) {
  constexpr int kStep = 8 * kThreads, kLow = 16 * kStep, kMid = 16 * kLow;
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = 0.f;
  for (int c2 = threadIdx.x; c2 < C; c2 += kMid) {
    float mid[N] = {};
    const int end2 = min(C, c2 + kMid);
    for (int c1 = c2; c1 < end2; c1 += kLow) {
      float low[N] = {};
      const int end1 = min(C, c1 + kLow);
      for (int c = c1; c < end1; c += kStep) {
        float v[8][N];
        if (TOGETHER && c + 7 * kThreads < C) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f(c + j * kThreads, v[j]);
#pragma unroll
          for (int i = 0; i < N; ++i)
            low[i] += ((v[0][i] + v[1][i]) + (v[2][i] + v[3][i])) +
                      ((v[4][i] + v[5][i]) + (v[6][i] + v[7][i]));
        } else {
          float eight[N] = {};
#pragma unroll 1
          for (int k = c; k < min(C, c + kStep); k += kThreads) {
            f(k, v[0]);
#pragma unroll
            for (int i = 0; i < N; ++i) eight[i] += v[0][i];
          }
#pragma unroll
          for (int i = 0; i < N; ++i) low[i] += eight[i];
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) mid[i] += low[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] += mid[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = block_sum(sum[i]);
}

// Rows wider than the ones above: one block per row, which reads the row three
// times (twice from L2). The second reading sums d = v - m, m being the first
// one's mean, and d^2: m + mean(d) is the mean but for a rounding, however far
// it is above the spread, and mean(d^2) - mean(d)^2 the variance (the corrected
// two-pass sums of Chan, Golub and LeVeque, 1983). 1024 x 32768 bf16: 151 us, with
// residual and dropout 500 us (floors 20 and 40): two bytes a load, and the
// generator drawn three times. 32 registers keep eight blocks an SM, so that
// these rows are one wave (60 registers: 238 us).
template <typename T, bool DROP>
__global__ void __launch_bounds__(kThreads, 8) fwd_wide_kernel(FwdArgs a) {
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const long long base = row * a.C;
    const T* const x = static_cast<const T*>(a.x) + base;
    const T* const res = a.residual != nullptr ? static_cast<const T*>(a.residual) + base : nullptr;
    auto value = [&](int c) {
      float v = to_f32(x[c]);
      if (DROP) v = kept(base + c, a.drop) ? v * a.drop.inv_keep : 0.f;
      return res != nullptr ? v + to_f32(res[c]) : v;
    };
    float s[1], q[2];
    wide_sums<!DROP>(a.C, [&](int c, float (&v)[1]) { v[0] = value(c); }, s);
    const float m = s[0] / a.C;
    wide_sums<!DROP>(
        a.C,
        [&](int c, float (&v)[2]) {
          v[0] = value(c) - m;
          v[1] = v[0] * v[0];
        },
        q);
    const float rest = q[0] / a.C;  // no number where the row has an infinity
    const float mu = isfinite(rest) ? m + rest : m;
    const float var = fmaf(-rest, rest, q[1] / a.C);
    const float r = 1.0f / sqrtf((var < 0.f ? 0.f : var) + a.eps);
    for (int c = threadIdx.x; c < a.C; c += kThreads) {
      const float v = value(c);
      float o = ((v - m) - rest) * r;
      if (a.gamma != nullptr) o *= load_as(a.gamma, c, a.wdtype);
      if (a.beta != nullptr) o += load_as(a.beta, c, a.wdtype);
      if (a.z != nullptr) static_cast<T*>(a.z)[base + c] = from_f32<T>(v);
      static_cast<T*>(a.y)[base + c] = from_f32<T>(o);
    }
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = mu;
      if (a.rstd != nullptr) a.rstd[row] = r;
    }
  }
}

// The same of the backward, with the statistics given; its roundings are written
// out, so that they do not depend on which of the outputs are wanted. 1024 x
// 32768 bf16 with the weights' gradients: 204 us (floor 30).
template <typename T>
__global__ void __launch_bounds__(kThreads, 8) bwd_wide_kernel(BwdArgs a) {
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const long long base = row * a.C;
    const T* const dy = static_cast<const T*>(a.dy) + base;
    const T* const z = static_cast<const T*>(a.z) + base;
    const T* const dz = a.dz != nullptr ? static_cast<const T*>(a.dz) + base : nullptr;
    const float mu = a.mean[row], r = a.rstd[row];
    auto grad = [&](int c) {
      const float g = to_f32(dy[c]);
      return a.gamma != nullptr ? __fmul_rn(g, load_as(a.gamma, c, a.wdtype)) : g;
    };
    auto normed = [&](int c) { return __fmul_rn(to_f32(z[c]) - mu, r); };
    float sums[2];
    wide_sums<true>(
        a.C,
        [&](int c, float (&v)[2]) {
          v[0] = grad(c);
          v[1] = __fmul_rn(v[0], normed(c));
        },
        sums);
    const float s = sums[0] / a.C, t = sums[1] / a.C;
    for (int c = threadIdx.x; c < a.C; c += kThreads) {
      float v = __fmul_rn(r, fmaf(-normed(c), t, grad(c) - s));
      if (dz != nullptr) v = __fadd_rn(v, to_f32(dz[c]));
      if (a.dres != nullptr) static_cast<T*>(a.dres)[base + c] = from_f32<T>(v);
      if (a.dx != nullptr) {
        if (a.drop.on) v = kept(base + c, a.drop) ? v * a.drop.inv_keep : 0.f;
        static_cast<T*>(a.dx)[base + c] = from_f32<T>(v);
      }
    }
  }
}

// Weight gradients of wide rows: 32 columns by a chunk of rows.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    weights_wide_kernel(BwdArgs a, long long rows_per_chunk) {
  __shared__ float part[2][8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  const long long first = blockIdx.y * rows_per_chunk;
  const long long last = first + rows_per_chunk < a.rows ? first + rows_per_chunk : a.rows;
  float s = 0.f, t = 0.f;
  if (c < a.C) {
    for (long long row = first + ty; row < last; row += 8) {
      const float g = to_f32(static_cast<const T*>(a.dy)[row * a.C + c]);
      const float z = to_f32(static_cast<const T*>(a.z)[row * a.C + c]);
      const float h = (z - a.mean[row]) * a.rstd[row];
      s += g;
      t = fmaf(g, h, t);
    }
  }
  part[0][ty][tx] = t;
  part[1][ty][tx] = s;
  __syncthreads();
  if (ty < 2 && c < a.C) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[ty][i][tx];
    a.workspace[(static_cast<long long>(blockIdx.y) * 2 + ty) * a.C + c] = v;
  }
}

inline unsigned grid_for(long long want) {
  const long long cap = static_cast<long long>(sm_count() > 0 ? sm_count() : 1) * 8;
  return static_cast<unsigned>(want < cap ? want : cap);
}

// f(Shape) for the row length: up to 16 elements a thread, so that weights and
// the backward's sums stay in registers. The widest rows take a cluster of two
// blocks for it (2048 x 16384 bf16: forward 40 us, backward 58 us; with one
// block and 32 elements a thread 45 and 72 us, with the weights read again for
// each row 44 and 97 us). Blocks have at least LEAST threads.
template <typename T, int LEAST, bool BACKWARD, typename F>
int with_shape(int C, F f) {
  constexpr int E = Vec<T>::kElems;
  // a ragged row takes up to one vector more than its length needs
  const int n = C % E == 0 ? C : C + 2 * E - 2;
  // short rows of the backward: small blocks, three an SM (524288 x 64 bf16 36
  // us against 47 with 512 threads, 262144 x 128 36 against 38; from 256 columns
  // on the same or slower)
  if (n <= 64) return f(Shape<8, 8 / E, 256>{});
  if (n <= 128) return f(Shape<BACKWARD ? 16 : 8, (BACKWARD ? 8 : 16) / E, 256>{});
  if (n <= 256) return f(Shape<16, 16 / E, LEAST>{});
  if (n <= 512) return f(Shape<32, 16 / E, LEAST>{});
  if (n <= 1024) return f(Shape<64, 16 / E, LEAST>{});
  if (n <= 2048) return f(Shape<128, 16 / E, LEAST>{});
  if (n <= 4096) return f(Shape<256, 16 / E, LEAST>{});
  if (n <= 8192) return f(Shape<512, 16 / E, LEAST>{});
  return f(Shape<512, 16 / E, LEAST, 2>{});
}

template <typename T>
bool fits(int C) {
  constexpr int E = Vec<T>::kElems;
  return (C % E == 0 ? C : C + 2 * E - 2) <= kMaxRow;
}

// Launches a walking kernel: as many rows' blocks as are resident at a time, in
// eights, no more than there are rows for or `most`; returns the number of
// blocks (clusters, for rows of several blocks) that get rows, or a negative
// error. The ring takes `smem` bytes. `resident` is the caller's record per device.
template <typename S, typename Kernel, typename Args>
int launch_walk(Kernel kern, const Args& a, int smem, long long most,
                std::atomic<bool> (&limit_set)[kMaxTrackedDevices],
                std::atomic<int> (&resident)[kMaxTrackedDevices], cudaStream_t stream) {
  if (!set_smem_limit_once(kern, smem, limit_set)) return ATTN_ERR_LAUNCH;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_LAUNCH;
  const bool tracked = dev >= 0 && dev < kMaxTrackedDevices;
  int at_once = tracked ? resident[dev].load(std::memory_order_relaxed) : 0;
  if (at_once <= 0) {
    if (S::CTAS > 1) {
      cudaLaunchAttribute cluster;
      cluster.id = cudaLaunchAttributeClusterDimension;
      cluster.val.clusterDim.x = S::CTAS;
      cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
      cudaLaunchConfig_t config{};
      config.gridDim = dim3(S::CTAS);
      config.blockDim = dim3(S::BLOCK);
      config.dynamicSmemBytes = static_cast<size_t>(smem);
      config.attrs = &cluster;
      config.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&at_once, kern, &config) != cudaSuccess)
        return (void)cudaGetLastError(), ATTN_ERR_LAUNCH;
    } else {
      if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&at_once, kern, S::BLOCK, smem) !=
          cudaSuccess)
        return (void)cudaGetLastError(), ATTN_ERR_LAUNCH;
      at_once *= sm_count();
    }
    if (at_once <= 0) return ATTN_ERR_LAUNCH;
    if (tracked) resident[dev].store(at_once, std::memory_order_relaxed);
  }
  long long n = std::max(8LL, std::min<long long>(at_once, most) / 8 * 8);
  n = std::min(n, ((a.rows + S::ROWS - 1) / S::ROWS + 7) / 8 * 8);
  const Split split{static_cast<int>(a.rows / (n * S::ROWS)), a.rows % (n * S::ROWS)};
  const int rc = launch_overlapped(kern, dim3(static_cast<unsigned>(n * S::CTAS)), S::BLOCK, smem,
                                   S::CTAS > 1 ? S::CTAS : 0, stream, a, split);
  if (rc != ATTN_OK) return rc;
  return static_cast<int>(std::min(n, (a.rows + S::ROWS - 1) / S::ROWS));
}

// Launches a walking kernel as one cluster of `blocks` blocks; 0, or a negative
// error.
template <typename S, typename Kernel, typename Args>
int launch_cluster(Kernel kern, const Args& a, int smem, int blocks,
                   std::atomic<bool> (&limit_set)[kMaxTrackedDevices], cudaStream_t stream) {
  if (!set_smem_limit_once(kern, smem, limit_set)) return ATTN_ERR_LAUNCH;
  const long long places = static_cast<long long>(blocks) * S::ROWS;
  const Split split{static_cast<int>(a.rows / places), a.rows % places};
  return launch_overlapped(kern, dim3(static_cast<unsigned>(blocks)), S::BLOCK, smem, blocks,
                           stream, a, split);
}

// Stages of a ring whose stage has `bytes`: what `room` has place for, in
// pairs, up to eight.
constexpr int stages_for(int bytes, int room) {
  const int n = room / bytes;
  return n >= 8 ? 8 : n >= 6 ? 6 : n >= 4 ? 4 : n >= 2 ? 2 : 1;
}

template <typename T, bool ADD, bool DROP, bool RAGGED>
int fwd_rows(const FwdArgs& a, cudaStream_t stream) {
  return with_shape<T, 256, false>(a.C, [&](auto shape) {
    using S = decltype(shape);
    static std::atomic<bool> limit_set[kMaxTrackedDevices];
    static std::atomic<int> resident[kMaxTrackedDevices];
    constexpr int kBytes = (ADD ? 2 : 1) * S::VECS * S::BLOCK * 16;
    constexpr int kStages = stages_for(kBytes, (S::BLOCK <= 256 ? 104 : 208) * 1024);
    constexpr int kRows = kStages > 2 ? 2 : 1;
    const int n = launch_walk<S>(fwd_kernel<T, S, kStages, kRows, ADD, DROP, RAGGED>, a,
                                 kStages * kBytes, 1LL << 20, limit_set, resident, stream);
    return n < 0 ? n : static_cast<int>(ATTN_OK);
  });
}

template <typename T, bool RAGGED>
int fwd_kinds(const FwdArgs& a, cudaStream_t stream) {
  if (a.residual == nullptr) return fwd_rows<T, false, false, RAGGED>(a, stream);
  return a.drop.on ? fwd_rows<T, true, true, RAGGED>(a, stream)
                   : fwd_rows<T, true, false, RAGGED>(a, stream);
}

template <typename T>
int run_fwd(const FwdArgs& a, cudaStream_t stream) {
  if (!fits<T>(a.C)) {
    const auto kern = a.drop.on ? fwd_wide_kernel<T, true> : fwd_wide_kernel<T, false>;
    kern<<<grid_for(a.rows), kThreads, 0, stream>>>(a);
    return launch_status();
  }
  return a.C % Vec<T>::kElems != 0 ? fwd_kinds<T, true>(a, stream) : fwd_kinds<T, false>(a, stream);
}

template <typename T, bool DZ, bool DROP, bool RAGGED>
int bwd_rows(const BwdArgs& a, cudaStream_t stream) {
  // rows of more than 128 columns: one block of 512 threads an SM, so one
  // partial sum a column each
  return with_shape<T, 512, true>(a.C, [&](auto shape) {
    using S = decltype(shape);
    static std::atomic<bool> limit_set[kMaxTrackedDevices];
    static std::atomic<int> resident[kMaxTrackedDevices];
    constexpr int kBytes = (DZ ? 3 : 2) * S::VECS * S::BLOCK * 16;
    constexpr int kStages = stages_for(kBytes, (S::BLOCK <= 256 ? 72 : 208) * 1024);
    // the ring's memory also takes the sums of the block's rows of threads
    static_assert(kStages * kBytes >= S::BLOCK * S::VECS * Vec<T>::kElems * 9,
                  "ring too small for the sums");
    // (with 16 elements a thread, two rows of a warp's own a turn spill)
    constexpr int kRows = kStages > 2 && (S::WARPS > 1 || S::BLOCK <= 256) ? 2 : 1;
    const auto kern = bwd_kernel<T, S, kStages, kRows, DZ, DROP, RAGGED>;
    // Weight gradients of up to eight blocks' rows of one turn: one cluster
    // finishes them itself (500 rows of 64 columns 3.2 us, 4.1 with the second
    // launch; 100 of 100 3.9 and 4.7). From 512 columns on reading the other
    // blocks' sums costs as much as that launch, or more (32 of 4096 9.0 and
    // 6.6).
    if (S::FINISH && a.workspace != nullptr && a.rows <= 8LL * S::ROWS * kRows) {
      BwdArgs b = a;
      b.finish = 1;
      int blocks = 1;  // RAGGED: where threads take two rows, a multiple of 8 rows apart
      while (blocks < 8 && blocks * S::ROWS < a.rows) blocks *= 2;
      return launch_cluster<S>(kern, b, kStages * kBytes, blocks, limit_set, stream);
    }
    return launch_walk<S>(kern, a, kStages * kBytes, kMaxChunks, limit_set, resident, stream);
  });
}

template <typename T, bool RAGGED>
int bwd_kinds(const BwdArgs& a, cudaStream_t stream) {
  if (a.dz != nullptr)
    return a.drop.on ? bwd_rows<T, true, true, RAGGED>(a, stream)
                     : bwd_rows<T, true, false, RAGGED>(a, stream);
  return a.drop.on ? bwd_rows<T, false, true, RAGGED>(a, stream)
                   : bwd_rows<T, false, false, RAGGED>(a, stream);
}

template <typename T>
int run_bwd(const BwdArgs& a, cudaStream_t stream) {
  if (!fits<T>(a.C)) {
    int chunks = 0;
    if (a.workspace != nullptr) {
      chunks = static_cast<int>(std::min<long long>((a.rows + 63) / 64, kMaxChunks));
      const dim3 grid(static_cast<unsigned>((a.C + 31) / 32), static_cast<unsigned>(chunks));
      weights_wide_kernel<T><<<grid, kThreads, 0, stream>>>(a, (a.rows + chunks - 1) / chunks);
    }
    bwd_wide_kernel<T><<<grid_for(a.rows), kThreads, 0, stream>>>(a);
    const int rc = launch_status();
    return rc != ATTN_OK ? rc : chunks;
  }
  return a.C % Vec<T>::kElems != 0 ? bwd_kinds<T, true>(a, stream) : bwd_kinds<T, false>(a, stream);
}

}  // namespace norm
}  // namespace attn
