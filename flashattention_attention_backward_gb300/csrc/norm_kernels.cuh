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

#include "norm_common.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace norm {

template <int TPR_, int VECS_, int LEAST>
struct Shape {
  static constexpr int TPR = TPR_;    // threads per row
  static constexpr int VECS = VECS_;  // 16-byte vectors per thread
  static constexpr int BLOCK = TPR_ < LEAST ? LEAST : TPR_;
  static constexpr int ROWS = BLOCK / TPR_;  // rows of a block at a time
  static constexpr int WARPS = TPR_ > 32 ? TPR_ / 32 : 1;  // warps per row
  static constexpr int LANES = TPR_ > 32 ? 32 : TPR_;      // lanes of a warp per row
};

// Barrier over a row's threads (rows of several warps; the block's other rows
// go on by themselves).
template <typename S>
__device__ __forceinline__ void row_barrier() {
  if (S::ROWS == 1)
    __syncthreads();
  else
    ptx::named_bar_sync(1 + threadIdx.x / S::TPR, S::TPR);
}

// The E weights (or biases) of columns c .. c + E - 1 (a multiple of four) as
// they lie in memory, widened by get(); `fill` where there is no array.
template <int E>
struct Weights {
  uint32_t w[E];  // 16-bit types fill the first half
  __device__ __forceinline__ void load(const void* p, int c, int wdtype) {
    if (p == nullptr) return;
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      if (wdtype == ATTN_FP32) {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + c + i);
        w[i] = v.x;
        w[i + 1] = v.y;
        w[i + 2] = v.z;
        w[i + 3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c + i);
        w[i / 2] = v.x;
        w[i / 2 + 1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void get(const void* p, int wdtype, float fill, float (&f)[E]) const {
    if (p == nullptr) {
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = fill;
    } else if (wdtype == ATTN_FP32) {
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = __uint_as_float(w[i]);
    } else if (wdtype == ATTN_BF16) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = h.x;
        f[2 * i + 1] = h.y;
      }
    }
  }
};

// The same for any c, one element at a time; `fill` outside the row too.
template <int E>
__device__ __forceinline__ void load_weights_ragged(const void* p, int c, int C, int wdtype,
                                                    float fill, float (&f)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i)
    f[i] = p != nullptr && static_cast<unsigned>(c + i) < static_cast<unsigned>(C)
               ? load_as(p, c + i, wdtype)
               : fill;
}

// Sets the elements of columns outside the row to `fill`.
template <int E>
__device__ __forceinline__ void keep_inside(float (&f)[E], int c, int C, float fill) {
  if (c >= 0 && c + E <= C) return;
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (static_cast<unsigned>(c + i) >= static_cast<unsigned>(C)) f[i] = fill;
}

// Writes the vector's elements that lie in the row.
template <typename T, bool RAGGED, int E>
__device__ __forceinline__ void store_row_vec(T* p, const float (&f)[E], int c, int C) {
  if (!RAGGED || (c >= 0 && c + E <= C)) {
    Vec<T> v;
    pack(f, v);
    store_vec(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (static_cast<unsigned>(c + i) < static_cast<unsigned>(C)) p[i] = from_f32<T>(f[i]);
  }
}

__device__ __forceinline__ void copy_async16(uint32_t smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(global) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A block's walk over rows, shared by the two kernels: blocks stay and take
// rows a grid apart, so that a thread's columns are the same in all of its
// rows (RAGGED: the grid is a multiple of 8 blocks, so all of a thread's rows
// start at the same offset within a vector), and its weights, or its sums of
// the weights' gradients, stay in registers. Rows of NT tensors come through
// a ring of STAGES in shared memory, filled by asynchronous copies: a thread
// reads back only what it copied itself, so the ring needs no barrier, and
// the next rows' loads run while this one is reduced. A row's slots stay for
// LAG turns more. Vectors outside the row read as zeros.
template <typename T, typename S, int STAGES, int LAG, int NT, bool RAGGED>
struct Walk {
  static constexpr int E = Vec<T>::kElems;
  static constexpr int kAhead = STAGES - 1 - LAG;  // rows being copied
  static constexpr int kStage = NT * S::VECS * S::BLOCK;  // slots of a stage
  uint4* ring;        // this thread's slots: [STAGES][NT][VECS], BLOCK apart
  const T* from[NT];  // vector 0 of the next row to copy
  const T* end[NT];   // behind the tensors (RAGGED)
  long long stride;   // elements between this thread's rows
  long long e;        // element of the current row's vector 0
  long long row, step;
  int left, to_copy;  // this thread's rows still to come, and to be copied
  int t, shift, C;
  int fill, take;     // where the stages begin

  __device__ __forceinline__ Walk(uint4* smem, const void* const (&src)[NT], long long rows, int C_)
      : ring(smem + threadIdx.x), C(C_), fill(0), take(0) {
    t = threadIdx.x % S::TPR;
    row = static_cast<long long>(blockIdx.x) * S::ROWS + threadIdx.x / S::TPR;
    step = static_cast<long long>(gridDim.x) * S::ROWS;
    shift = RAGGED ? static_cast<int>((row * C) % E) : 0;
    e = row * C - shift + t * E;
    stride = step * C;
    left = row < rows ? static_cast<int>((rows - row + step - 1) / step) : 0;
    to_copy = left;
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      from[q] = static_cast<const T*>(src[q]) + e;
      end[q] = static_cast<const T*>(src[q]) + rows * C;
    }
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
  // element of vector j, less that of vector 0
  __device__ __forceinline__ static constexpr int offset(int j) { return j * S::TPR * E; }
  // turns to take: this thread's rows; where several rows share a warp, the
  // most that one of the block's has (active() tells whether a row is there)
  __device__ __forceinline__ int turns(long long rows) const {
    if (S::TPR >= 32) return left;
    const long long first = static_cast<long long>(blockIdx.x) * S::ROWS;
    return first < rows ? static_cast<int>((rows - first + step - 1) / step) : 0;
  }
  __device__ __forceinline__ bool active() const { return S::TPR >= 32 || left > 0; }

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
            if (!RAGGED || p + E <= end[q]) {
              copy_async16(ptx::smem_u32(slot), p);
            } else {  // the tensor's last vector is no whole one
              T* v = reinterpret_cast<T*>(slot);
              for (int i = 0; i < E; ++i) v[i] = p + i < end[q] ? p[i] : from_f32<T>(0.f);
            }
          }
        }
      }
    } else if (S::TPR < 32) {  // the warp's other rows go on: no stale values
#pragma unroll
      for (int k = 0; k < NT * S::VECS; ++k) to[k * S::BLOCK] = make_uint4(0u, 0u, 0u, 0u);
    }
    copy_commit();
    --to_copy;
#pragma unroll
    for (int q = 0; q < NT; ++q) from[q] += stride;
    fill = fill == (STAGES - 1) * kStage ? 0 : fill + kStage;
  }
  // starts the next copies and waits for the current row's
  __device__ __forceinline__ void arrive() {
    copy_next();
    copy_wait<kAhead>();
  }
  // vector j of tensor q in the stage that begins at `at`
  __device__ __forceinline__ void get(int at, int q, int j, float (&f)[E]) const {
    Vec<T> v;
    v.w = ring[at + (q * S::VECS + j) * S::BLOCK];
    unpack(v, f);
  }
  __device__ __forceinline__ void next() {
    row += step;
    e += stride;
    --left;
    take = take == (STAGES - 1) * kStage ? 0 : take + kStage;
  }
};

// Sum over groups of W lanes, the same value in each.
template <int W>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int off = W / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Weights of columns c .. c + E - 1 in fp32 pairs (a null array: `fill`).
template <int E, bool RAGGED>
__device__ __forceinline__ void weight_pairs(const void* p, int c, int C, int wdtype, float fill,
                                             uint64_t (&g)[E / 2]) {
  float f[E];
  if (c >= C) {
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = 0.f;
  } else if (RAGGED) {
    load_weights_ragged<E>(p, c, C, wdtype, fill, f);
  } else {
    Weights<E> w;
    w.load(p, c, wdtype);
    w.get(p, wdtype, fill, f);
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) g[i] = ptx::f2_make(f[2 * i], f[2 * i + 1]);
}

// What a row leaves for the second half of its turn.
struct Mark {
  long long e, row;
  int stage;
  bool active;
};

// Forward, a row in two halves.
// First half: its sum with the residual, behind the dropout, goes to fp32
// registers, in pairs (one instruction for two columns); a warp takes the mean
// of its part and the squares about that. Second half: parts of n_w elements
// are joined by
//   mu = sum n_w mu_w / C,  sum of squares = sum (q_w + n_w (mu_w - mu)^2),
// which loses nothing to cancellation and costs one barrier a row, and the
// output is written. LAG = 1: a row's second half runs in one turn with the
// next row's first, so that the reductions of one are covered by the
// arithmetic of the other. ADD: with a residual, and z written.
template <typename T, typename S, int STAGES, int LAG, bool ADD, bool DROP, bool RAGGED>
__global__ void __launch_bounds__(S::BLOCK, S::BLOCK <= 256 ? 2 : 1) fwd_kernel(FwdArgs a) {
  constexpr int E = Vec<T>::kElems, VECS = S::VECS, P = E / 2, NT = ADD ? 2 : 1;
  constexpr bool kKeep = VECS * E <= 16 && S::TPR <= 512;  // weights stay in registers
  constexpr int kLanes = S::LANES, kWarps = S::WARPS;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float2 parts[S::ROWS][2][kWarps];
  __shared__ float counts[S::BLOCK / 32];
  auto& part = parts[kWarps > 1 ? threadIdx.x / S::TPR : 0];
  const int warp = threadIdx.x / 32 % kWarps;  // of the row
  const void* src[NT];
  src[0] = a.x;
  if (ADD) src[NT - 1] = a.residual;
  Walk<T, S, STAGES, 0, NT, RAGGED> w(ring, src, a.rows, a.C);
  const float inv_C = 1.0f / static_cast<float>(a.C);
  uint64_t gamma[kKeep ? VECS : 1][P], beta[kKeep ? VECS : 1][P];
  int mine = 0;  // this thread's columns inside the row
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int c = w.column(j);
    if (kKeep) {
      weight_pairs<E, RAGGED>(a.gamma, c, a.C, a.wdtype, 1.f, gamma[j]);
      weight_pairs<E, RAGGED>(a.beta, c, a.C, a.wdtype, 0.f, beta[j]);
    }
    if (w.inside(j)) mine += RAGGED ? min(c + E, a.C) - max(c, 0) : E;
  }
  const float count = lane_sum<kLanes>(static_cast<float>(mine));  // n_w
  const float inv_count = count > 0.f ? 1.0f / count : 0.f;
  float other = count;  // n_w of the warp whose part this lane joins
  if (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = count;
    __syncthreads();
    other = counts[threadIdx.x / 32 - warp + threadIdx.x % kWarps];
  }
  int parity = 0;

  // first half of the current row: v, and the mean and squares of the warp's part
  auto first_half = [&](uint64_t (&v)[VECS][P], float& mu, float& q) {
    w.arrive();
    const bool active = w.active();
    const uint64_t inv_keep = ptx::f2_make(a.drop.inv_keep, a.drop.inv_keep);
    uint64_t s2 = 0, q2 = 0;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      float f[E];
      w.get(w.take, 0, j, f);
      if (DROP) drop_vec<E>(f, w.e + w.offset(j), a.drop);
#pragma unroll
      for (int i = 0; i < P; ++i) v[j][i] = ptx::f2_make(f[2 * i], f[2 * i + 1]);
      if (ADD) {
        float r[E];
        w.get(w.take, NT - 1, j, r);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const uint64_t r2 = ptx::f2_make(r[2 * i], r[2 * i + 1]);
          v[j][i] = DROP ? ptx::f2_fma(v[j][i], inv_keep, r2) : ptx::f2_add(v[j][i], r2);
          f[2 * i] = ptx::f2_lo(v[j][i]);
          f[2 * i + 1] = ptx::f2_hi(v[j][i]);
        }
        if (active && w.inside(j))
          store_row_vec<T, RAGGED>(static_cast<T*>(a.z) + w.e + w.offset(j), f, w.column(j), a.C);
      }
      if (RAGGED) {
        keep_inside<E>(f, w.column(j), a.C, 0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) v[j][i] = ptx::f2_make(f[2 * i], f[2 * i + 1]);
      }
#pragma unroll
      for (int i = 0; i < P; ++i) s2 = ptx::f2_add(s2, v[j][i]);
    }
    mu = lane_sum<kLanes>(ptx::f2_lo(s2) + ptx::f2_hi(s2)) * inv_count;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = w.column(j);
      if (RAGGED && (c < 0 || c + E > a.C)) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float d = (i % 2 == 0 ? ptx::f2_lo(v[j][i / 2]) : ptx::f2_hi(v[j][i / 2])) - mu;
          if (static_cast<unsigned>(c + i) < static_cast<unsigned>(a.C))
            q2 = ptx::f2_fma(ptx::f2_make(d, 0.f), ptx::f2_make(d, 0.f), q2);
        }
      } else {
        const float m = w.inside(j) ? -mu : 0.f;  // outside the row v is 0
        const uint64_t minus = ptx::f2_make(m, m);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const uint64_t d = ptx::f2_add(v[j][i], minus);
          q2 = ptx::f2_fma(d, d, q2);
        }
      }
    }
    q = lane_sum<kLanes>(ptx::f2_lo(q2) + ptx::f2_hi(q2));
  };
  auto mark = [&]() { return Mark{w.e, w.row, w.take, w.active()}; };
  // second half of row m, from the parts' means and squares
  auto second_half = [&](const Mark& m, const uint64_t (&v)[VECS][P], float mu, float q) {
    if (kWarps > 1) {
      const float mean = lane_sum<kWarps>(other * mu) * inv_C, d = mu - mean;
      mu = mean;
      q = lane_sum<kWarps>(other > 0.f ? fmaf(other * d, d, q) : 0.f);
    }
    const float r = rsqrtf(fmaf(q, inv_C, a.eps));
    const uint64_t minus_mu = ptx::f2_make(-mu, -mu), r2 = ptx::f2_make(r, r);
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = w.column(j), k = kKeep ? j : 0;
      if (!kKeep) {
        weight_pairs<E, RAGGED>(a.gamma, c, a.C, a.wdtype, 1.f, gamma[0]);
        weight_pairs<E, RAGGED>(a.beta, c, a.C, a.wdtype, 0.f, beta[0]);
      }
      float f[E];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint64_t h = ptx::f2_mul(ptx::f2_add(v[j][i], minus_mu), r2);
        const uint64_t o = ptx::f2_fma(h, gamma[k][i], beta[k][i]);
        f[2 * i] = ptx::f2_lo(o);
        f[2 * i + 1] = ptx::f2_hi(o);
      }
      if (m.active && w.inside(j))
        store_row_vec<T, RAGGED>(static_cast<T*>(a.y) + m.e + w.offset(j), f, c, a.C);
    }
    if (m.active && w.t == 0) {
      if (a.mean != nullptr) a.mean[m.row] = mu;
      if (a.rstd != nullptr) a.rstd[m.row] = r;
    }
  };
  // hands the warp's part to the block, and takes the parts back
  auto give = [&](float mu, float q) {
    if (kWarps > 1) {
      if ((threadIdx.x & 31) == 0) part[parity][warp] = make_float2(mu, q);
      row_barrier<S>();
    }
  };
  auto take = [&](float& mu, float& q) {
    if (kWarps > 1) {
      const float2 p = part[parity][threadIdx.x % kWarps];
      mu = p.x;
      q = p.y;
      parity ^= 1;
    }
  };

  int turns = w.turns(a.rows);
  if (turns == 0) return;
  uint64_t v[VECS][P];
  float mu, q;
  if (LAG == 0) {
    for (; turns > 0; --turns, w.next()) {
      first_half(v, mu, q);
      give(mu, q);
      take(mu, q);
      second_half(mark(), v, mu, q);
    }
  } else {
    first_half(v, mu, q);
    Mark m = mark();
    give(mu, q);
    for (w.next(); turns > 1; --turns, w.next()) {
      uint64_t v_next[VECS][P];
      float mu_next, q_next;
      take(mu, q);
      first_half(v_next, mu_next, q_next);
      second_half(m, v, mu, q);
      m = mark();
#pragma unroll
      for (int j = 0; j < VECS; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) v[j][i] = v_next[j][i];
      mu = mu_next;
      q = q_next;
      give(mu, q);
    }
    take(mu, q);
    second_half(m, v, mu, q);
  }
  copy_wait<0>();
}

// Sums of two values over groups of W lanes, the same values in each.
template <int W>
__device__ __forceinline__ void lane_sums(float& s, float& u) {
  s = lane_sum<W>(s);
  u = lane_sum<W>(u);
}
// Over a whole warp: the first exchange leaves half of the lanes with one
// value and half with the other, so that one value a lane is left to sum.
// Lane 0 has the first value's sum, lane 16 the second's.
__device__ __forceinline__ float warp_sums(float s, float u) {
  const bool low = (threadIdx.x & 16) == 0;
  float v = (low ? s : u) + __shfl_xor_sync(0xffffffffu, low ? u : s, 16);
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Backward, a row in two halves like the forward: first the row's two sums
// and its part of the weights' gradients, whose column sums stay in registers
// over all of the thread's rows; then, with the sums joined over the row's
// threads, its gradient, from the ring again. DZ: with a dz to add.
template <typename T, typename S, int STAGES, int LAG, bool DZ, bool DROP, bool RAGGED>
__global__ void __launch_bounds__(S::BLOCK) bwd_kernel(BwdArgs a) {
  constexpr int E = Vec<T>::kElems, VECS = S::VECS, BLOCK = S::BLOCK, P = E / 2;
  constexpr int NT = DZ ? 3 : 2;
  constexpr bool kKeep = VECS * E <= 16;  // weights stay in registers
  constexpr int kLanes = S::LANES, kWarps = S::WARPS;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ __align__(16) float2 parts[S::ROWS][2][kWarps];
  auto& part = parts[kWarps > 1 ? threadIdx.x / S::TPR : 0];
  const void* src[NT];
  src[0] = a.dy;
  src[1] = a.z;
  if (DZ) src[NT - 1] = a.dz;
  Walk<T, S, STAGES, LAG, NT, RAGGED> w(ring, src, a.rows, a.C);
  const float inv_C = 1.0f / static_cast<float>(a.C);
  // the statistics of the row to come, one row ahead
  float mu_next = 0.f, r_next = 0.f;
  if (w.left > 0) {
    mu_next = a.mean[w.row];
    r_next = a.rstd[w.row];
  }
  uint64_t dgamma[VECS][P], dbeta[VECS][P], gamma[kKeep ? VECS : 1][P];
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
#pragma unroll
    for (int i = 0; i < P; ++i) dgamma[j][i] = dbeta[j][i] = 0;
    if (kKeep) weight_pairs<E, RAGGED>(a.gamma, w.column(j), a.C, a.wdtype, 1.f, gamma[j]);
  }
  // dy and z - mean of vector j (columns outside the row: dy = 0)
  auto gather = [&](int at, int j, float mu, uint64_t (&dy)[P], uint64_t (&d)[P]) {
    float fd[E], fz[E];
    w.get(at, 0, j, fd);
    w.get(at, 1, j, fz);
    if (RAGGED) {
      keep_inside<E>(fd, w.column(j), a.C, 0.f);
      keep_inside<E>(fz, w.column(j), a.C, 0.f);
    }
    if (!kKeep) weight_pairs<E, RAGGED>(a.gamma, w.column(j), a.C, a.wdtype, 1.f, gamma[0]);
    const uint64_t minus_mu = ptx::f2_make(-mu, -mu);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      dy[i] = ptx::f2_make(fd[2 * i], fd[2 * i + 1]);
      d[i] = ptx::f2_add(ptx::f2_make(fz[2 * i], fz[2 * i + 1]), minus_mu);
    }
  };
  int parity = 0;
  // first half of the current row: this thread's s = sum dy gamma and
  // u = sum dy (z - mean) gamma; rstd comes in behind the sums
  auto first_half = [&](float& mu, float& r, float& s, float& u) {
    mu = mu_next;
    r = r_next;
    mu_next = r_next = 0.f;
    if (w.left > 1) {
      mu_next = a.mean[w.row + w.step];
      r_next = a.rstd[w.row + w.step];
    }
    w.arrive();
    const uint64_t r2 = ptx::f2_make(r, r);
    uint64_t s2 = 0, u2 = 0;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      uint64_t dy[P], d[P];
      gather(w.take, j, mu, dy, d);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint64_t t = ptx::f2_mul(dy[i], d[i]);
        dgamma[j][i] = ptx::f2_fma(t, r2, dgamma[j][i]);
        dbeta[j][i] = ptx::f2_add(dbeta[j][i], dy[i]);
        s2 = ptx::f2_fma(dy[i], gamma[kKeep ? j : 0][i], s2);
        u2 = ptx::f2_fma(t, gamma[kKeep ? j : 0][i], u2);
      }
    }
    s = ptx::f2_lo(s2) + ptx::f2_hi(s2);
    u = ptx::f2_lo(u2) + ptx::f2_hi(u2);
    if (kWarps > 1)
      s = warp_sums(s, u);
    else
      lane_sums<kLanes>(s, u);
  };
  auto mark = [&]() { return Mark{w.e, w.row, w.take, w.active()}; };
  auto second_half = [&](const Mark& m, float mu, float r, float s, float u) {
    // dz = r g - r (r u / C) h - r s / C + dz_in, h = (z - mean) r
    const float rs = -r * (s * inv_C), ru = -r * (r * u * inv_C);
    const uint64_t r2 = ptx::f2_make(r, r), rs2 = ptx::f2_make(rs, rs), ru2 = ptx::f2_make(ru, ru);
    const uint64_t inv_keep = ptx::f2_make(a.drop.inv_keep, a.drop.inv_keep);
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = w.column(j);
      uint64_t dy[P], d[P];
      gather(m.stage, j, mu, dy, d);
      float f[E];
      if (DZ) w.get(m.stage, NT - 1, j, f);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint64_t g = ptx::f2_mul(dy[i], gamma[kKeep ? j : 0][i]);
        dy[i] = ptx::f2_fma(g, r2, ptx::f2_fma(ptx::f2_mul(d[i], r2), ru2, rs2));
        if (DZ) dy[i] = ptx::f2_add(dy[i], ptx::f2_make(f[2 * i], f[2 * i + 1]));
        f[2 * i] = ptx::f2_lo(dy[i]);
        f[2 * i + 1] = ptx::f2_hi(dy[i]);
      }
      const bool write = m.active && w.inside(j);
      if (write) store_row_vec<T, RAGGED>(static_cast<T*>(a.dres) + m.e + w.offset(j), f, c, a.C);
      if (DROP) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          dy[i] = ptx::f2_mul(dy[i], inv_keep);
          f[2 * i] = ptx::f2_lo(dy[i]);
          f[2 * i + 1] = ptx::f2_hi(dy[i]);
        }
        drop_vec<E>(f, m.e + w.offset(j), a.drop);
      }
      if ((DROP || a.dx != nullptr) && write)
        store_row_vec<T, RAGGED>(static_cast<T*>(a.dx) + m.e + w.offset(j), f, c, a.C);
    }
  };
  // hands the warp's sums to the block, and takes all of them back
  auto give = [&](float s) {
    if (kWarps > 1) {
      if ((threadIdx.x & 15) == 0) {
        float2* p = &part[parity][threadIdx.x / 32 % kWarps];
        ((threadIdx.x & 16) == 0 ? p->x : p->y) = s;
      }
      row_barrier<S>();
    }
  };
  auto take = [&](float& s, float& u) {
    if (kWarps > 1) {
      uint64_t v = 0;
#pragma unroll
      for (int i = 0; i < kWarps; i += 2) {
        const float4 p = *reinterpret_cast<const float4*>(&part[parity][i]);
        v = ptx::f2_add(v, ptx::f2_add(ptx::f2_make(p.x, p.y), ptx::f2_make(p.z, p.w)));
      }
      s = ptx::f2_lo(v);
      u = ptx::f2_hi(v);
      parity ^= 1;
    }
  };

  int turns = w.turns(a.rows);
  float mu = 0.f, r = 0.f, s = 0.f, u = 0.f;
  if (LAG == 0) {
    for (; turns > 0; --turns, w.next()) {
      first_half(mu, r, s, u);
      give(s);
      take(s, u);
      second_half(mark(), mu, r, s, u);
    }
  } else if (turns > 0) {
    first_half(mu, r, s, u);
    Mark m = mark();
    give(s);
    for (w.next(); turns > 1; --turns, w.next()) {
      float mu1, r1, s1, u1;
      take(s, u);
      first_half(mu1, r1, s1, u1);
      second_half(m, mu, r, s, u);
      m = mark();
      mu = mu1;
      r = r1;
      s = s1;
      u = u1;
      give(s);
    }
    take(s, u);
    second_half(m, mu, r, s, u);
  }
  copy_wait<0>();
  if (a.workspace == nullptr) return;
  float* out = a.workspace + 2LL * blockIdx.x * a.C;
  // f(column, dgamma, dbeta) for each of this thread's columns
  auto columns = [&](auto f) {
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = w.column(j);
      if (c >= a.C) continue;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (RAGGED && static_cast<unsigned>(c + i) >= static_cast<unsigned>(a.C)) continue;
        f(c + i, i % 2 == 0 ? ptx::f2_lo(dgamma[j][i / 2]) : ptx::f2_hi(dgamma[j][i / 2]),
          i % 2 == 0 ? ptx::f2_lo(dbeta[j][i / 2]) : ptx::f2_hi(dbeta[j][i / 2]));
      }
    }
  };
  if (S::ROWS == 1) {
    columns([&](int c, float x, float y) {
      out[c] = x;
      out[a.C + c] = y;
    });
  } else {
    // the block's rows of threads leave theirs side by side in the ring's
    // memory, and each column is added up over them in order
    float* sums = reinterpret_cast<float*>(ring);
    float* own = sums + threadIdx.x / S::TPR * 2 * a.C;
    __syncthreads();
    columns([&](int c, float x, float y) {
      own[c] = x;
      own[a.C + c] = y;
    });
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.C; i += BLOCK) {
      float v = 0.f;
#pragma unroll 8
      for (int k = 0; k < S::ROWS; ++k) v += sums[k * 2 * a.C + i];
      out[i] = v;
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

// Rows wider than the ones above: one block per row, which reads the row three
// times (twice from L2).
template <typename T>
__global__ void __launch_bounds__(kThreads) fwd_wide_kernel(FwdArgs a) {
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const long long base = row * a.C;
    auto value = [&](int c) {
      float v = to_f32(x[base + c]);
      if (a.drop.on) v = kept(base + c, a.drop) ? v * a.drop.inv_keep : 0.f;
      return res != nullptr ? v + to_f32(res[base + c]) : v;
    };
    float s = 0.f;
    for (int c = threadIdx.x; c < a.C; c += kThreads) s += value(c);
    const float mu = block_sum(s) / a.C;
    float q = 0.f;
    for (int c = threadIdx.x; c < a.C; c += kThreads) {
      const float d = value(c) - mu;
      q = fmaf(d, d, q);
    }
    const float r = 1.0f / sqrtf(block_sum(q) / a.C + a.eps);
    for (int c = threadIdx.x; c < a.C; c += kThreads) {
      const float v = value(c);
      float o = (v - mu) * r;
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

template <typename T>
__global__ void __launch_bounds__(kThreads) bwd_wide_kernel(BwdArgs a) {
  const T* dy = static_cast<const T*>(a.dy);
  const T* dz = static_cast<const T*>(a.dz);
  const T* z = static_cast<const T*>(a.z);
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const long long base = row * a.C;
    const float mu = a.mean[row], r = a.rstd[row];
    auto grad = [&](int c) {
      const float g = to_f32(dy[base + c]);
      return a.gamma != nullptr ? g * load_as(a.gamma, c, a.wdtype) : g;
    };
    float s = 0.f, t = 0.f;
    for (int c = threadIdx.x; c < a.C; c += kThreads) {
      const float g = grad(c), h = (to_f32(z[base + c]) - mu) * r;
      s += g;
      t = fmaf(g, h, t);
    }
    s = block_sum(s) / a.C;
    t = block_sum(t) / a.C;
    for (int c = threadIdx.x; c < a.C; c += kThreads) {
      const float g = grad(c), h = (to_f32(z[base + c]) - mu) * r;
      float v = r * (g - s - h * t);
      if (dz != nullptr) v += to_f32(dz[base + c]);
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
__global__ void __launch_bounds__(kThreads) weights_wide_kernel(BwdArgs a, long long rows_per_chunk) {
  __shared__ float part[2][8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  const long long first = blockIdx.y * rows_per_chunk;
  const long long last = first + rows_per_chunk < a.rows ? first + rows_per_chunk : a.rows;
  float s = 0.f, t = 0.f;
  if (c < a.C) {
    for (long long row = first + ty; row < last; row += 8) {
      const float g = to_f32(static_cast<const T*>(a.dy)[row * a.C + c]);
      const float h = (to_f32(static_cast<const T*>(a.z)[row * a.C + c]) - a.mean[row]) * a.rstd[row];
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

// f(Shape) for the row length: up to 16 elements a thread (32 for the widest),
// so that the backward's sums stay in registers; blocks of at least LEAST
// threads.
template <typename T, int LEAST, typename F>
int with_shape(int C, F f) {
  constexpr int E = Vec<T>::kElems;
  // a ragged row takes up to one vector more than its length needs
  const int n = C % E == 0 ? C : C + 2 * E - 2;
  if (n <= 64) return f(Shape<8, 8 / E, LEAST>{});
  if (n <= 128) return f(Shape<8, 16 / E, LEAST>{});
  if (n <= 256) return f(Shape<16, 16 / E, LEAST>{});
  if (n <= 512) return f(Shape<32, 16 / E, LEAST>{});
  if (n <= 1024) return f(Shape<64, 16 / E, LEAST>{});
  if (n <= 2048) return f(Shape<128, 16 / E, LEAST>{});
  if (n <= 4096) return f(Shape<256, 16 / E, LEAST>{});
  if (n <= 8192) return f(Shape<512, 16 / E, LEAST>{});
  return f(Shape<512, 32 / E, LEAST>{});
}

template <typename T>
bool fits(int C) {
  constexpr int E = Vec<T>::kElems;
  return (C % E == 0 ? C : C + 2 * E - 2) <= kMaxRow;
}

// Blocks of a kernel that fit an SM at a time (cached per device by the
// caller's record); 0 on error.
template <typename Kernel>
int blocks_per_sm(Kernel kern, int block, int smem, std::atomic<int> (&cache)[kMaxTrackedDevices]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool tracked = dev >= 0 && dev < kMaxTrackedDevices;
  if (tracked) {
    const int n = cache[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, block, smem) != cudaSuccess) return 0;
  if (tracked) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Launches a walking kernel: as many blocks as are resident at a time, in
// eights, no more than there are rows for or `most`; returns their number or a
// negative error. The ring takes `smem` bytes.
template <typename S, typename Kernel, typename Args>
int launch_walk(Kernel kern, const Args& a, int smem, long long most,
                std::atomic<bool> (&limit_set)[kMaxTrackedDevices],
                std::atomic<int> (&resident)[kMaxTrackedDevices], cudaStream_t stream) {
  if (!set_smem_limit_once(kern, smem, limit_set)) return ATTN_ERR_LAUNCH;
  const int per_sm = blocks_per_sm(kern, S::BLOCK, smem, resident);
  if (per_sm <= 0) return ATTN_ERR_LAUNCH;
  long long grid = static_cast<long long>(sm_count() > 0 ? sm_count() : 1) * per_sm;
  grid = std::max(8LL, std::min(grid, most) / 8 * 8);
  grid = std::min(grid, ((a.rows + S::ROWS - 1) / S::ROWS + 7) / 8 * 8);
  kern<<<static_cast<unsigned>(grid), S::BLOCK, smem, stream>>>(a);
  const int rc = launch_status();
  return rc != ATTN_OK ? rc : static_cast<int>(grid);
}

// Stages of a ring whose stage has `bytes`: four, or what `room` has place for.
constexpr int stages_for(int bytes, int room) {
  return bytes * 4 <= room ? 4 : (bytes * 3 <= room ? 3 : (bytes * 2 <= room ? 2 : 1));
}

template <typename T, bool ADD, bool DROP, bool RAGGED>
int fwd_rows(const FwdArgs& a, cudaStream_t stream) {
  return with_shape<T, 256>(a.C, [&](auto shape) {
    using S = decltype(shape);
    static std::atomic<bool> limit_set[kMaxTrackedDevices];
    static std::atomic<int> resident[kMaxTrackedDevices];
    constexpr int kBytes = (ADD ? 2 : 1) * S::VECS * S::BLOCK * 16, 
                  kStages = stages_for(kBytes, S::BLOCK <= 256 ? 98304 : 196608);
    const int n = launch_walk<S>(fwd_kernel<T, S, kStages, 1, ADD, DROP, RAGGED>, a, kStages * kBytes,
                                 1LL << 20, limit_set, resident, stream);
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
    fwd_wide_kernel<T><<<grid_for(a.rows), kThreads, 0, stream>>>(a);
    return launch_status();
  }
  return a.C % Vec<T>::kElems != 0 ? fwd_kinds<T, true>(a, stream) : fwd_kinds<T, false>(a, stream);
}

template <typename T, bool DZ, bool DROP, bool RAGGED>
int bwd_rows(const BwdArgs& a, cudaStream_t stream) {
  // one block of 512 threads an SM: one partial sum a column each
  return with_shape<T, 512>(a.C, [&](auto shape) {
    using S = decltype(shape);
    static std::atomic<bool> limit_set[kMaxTrackedDevices];
    static std::atomic<int> resident[kMaxTrackedDevices];
    constexpr int kBytes = (DZ ? 3 : 2) * S::VECS * S::BLOCK * 16;
    constexpr int kStages = stages_for(kBytes, 196608);
    // the ring's memory also takes the sums of the block's rows of threads
    static_assert(S::ROWS == 1 || kStages * kBytes >= S::BLOCK * S::VECS * Vec<T>::kElems * 8,
                  "ring too small for the sums");
    return launch_walk<S>(bwd_kernel<T, S, kStages, (kStages > 2 ? 1 : 0), DZ, DROP, RAGGED>, a, kStages * kBytes,
                          kMaxChunks, limit_set, resident, stream);
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
