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

template <int TPR_, int VECS_>
struct Shape {
  static constexpr int TPR = TPR_;    // threads per row
  static constexpr int VECS = VECS_;  // 16-byte vectors per thread
  static constexpr int BLOCK = TPR_ <= 32 ? 256 : TPR_;
  static constexpr int ROWS = BLOCK / TPR_;  // rows of a block at a time
};

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

// Drops and scales the E elements from e (a multiple of four) on.
template <int E>
__device__ __forceinline__ void drop_vec(float (&f)[E], long long e, const Drop& d) {
  uint32_t w[E / 4][4];
  keep_words<E / 4>(e, d, w);
#pragma unroll
  for (int i = 0; i < E; ++i) f[i] = w[i / 4][i % 4] >= d.threshold ? f[i] * d.inv_keep : 0.f;
}

// The vector of columns c .. c + E - 1 at p (16-byte aligned). RAGGED: it may
// reach over the row's ends, and past `end`, the tensor's; then only its
// elements inside the tensor are read.
template <typename T, bool RAGGED>
__device__ __forceinline__ Vec<T> load_row_vec(const T* p, const T* end) {
  constexpr int E = Vec<T>::kElems;
  if (!RAGGED || p + E <= end) return load_vec(p);
  Vec<T> v;
  T* e = reinterpret_cast<T*>(&v);
#pragma unroll
  for (int i = 0; i < E; ++i) e[i] = p + i < end ? p[i] : from_f32<T>(0.f);
  return v;
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

__device__ __forceinline__ void copy_async16(void* smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(smem))),
               "l"(global)
               : "memory");
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
// the weights' gradients, stay in registers. Rows come through a ring of
// STAGES in shared memory, filled by asynchronous copies: a thread reads back
// only what it copied itself, so the ring needs no barrier, and the next
// rows' loads run while this one is reduced.
template <typename T, typename S, int STAGES, int TENSORS, bool RAGGED>
struct Walk {
  static constexpr int E = Vec<T>::kElems;
  uint4* ring;               // [STAGES][tensors][VECS][BLOCK], this thread's slots
  const T* src[TENSORS];     // absent tensors come last and are not counted
  int tensors, C;
  long long rows, total, step, row, e;  // e: element of the row's first vector
  int t, shift;
  int stage;

  __device__ __forceinline__ Walk(uint4* smem, const T* const (&from)[TENSORS], int n,
                                  long long rows_, int C_)
      : ring(smem + threadIdx.x), tensors(n), C(C_), rows(rows_), total(rows_ * C_), stage(0) {
#pragma unroll
    for (int q = 0; q < TENSORS; ++q) src[q] = from[q];
    t = threadIdx.x % S::TPR;
    row = static_cast<long long>(blockIdx.x) * S::ROWS + threadIdx.x / S::TPR;
    step = static_cast<long long>(gridDim.x) * S::ROWS;
    shift = RAGGED ? static_cast<int>((row * C) % E) : 0;
    e = row * C - shift;
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) fetch(k, k);
  }
  // the first column of this thread's vector j; below 0 and up to the row's
  // end it reaches over the row's ends (RAGGED)
  __device__ __forceinline__ int column(int j) const { return (t + j * S::TPR) * E - shift; }
  __device__ __forceinline__ bool active() const { return row < rows; }
  __device__ __forceinline__ long long element(int j) const { return e + (t + j * S::TPR) * E; }
  __device__ __forceinline__ uint4* slot(int at, int q, int j) const {
    return ring + ((at * tensors + q) * S::VECS + j) * S::BLOCK;
  }
  // starts the copies of the row `ahead` steps on
  __device__ __forceinline__ void fetch(int ahead, int at) {
    if (row + ahead * step < rows) {
      const long long first = e + ahead * step * C;
#pragma unroll
      for (int j = 0; j < S::VECS; ++j) {
        if (column(j) < C) {
          const long long i = first + (t + j * S::TPR) * E;
#pragma unroll
          for (int q = 0; q < TENSORS; ++q) {
            if (q < tensors) {
              if (!RAGGED || i + E <= total)
                copy_async16(slot(at, q, j), src[q] + i);
              else
                *reinterpret_cast<Vec<T>*>(slot(at, q, j)) =
                    load_row_vec<T, RAGGED>(src[q] + i, src[q] + total);
            }
          }
        }
      }
    }
    copy_commit();
  }
  // starts the next copies and waits for the current row's
  __device__ __forceinline__ void arrive() {
    fetch(STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1);
    copy_wait<STAGES - 1>();
  }
  __device__ __forceinline__ void get(int q, int j, float (&f)[E]) const {
    unpack(*reinterpret_cast<const Vec<T>*>(slot(stage, q, j)), f);
  }
  __device__ __forceinline__ void next() {
    row += step;
    e += step * C;
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  // the block's first row is still one: the same for all of its threads
  __device__ __forceinline__ bool more() const {
    return row - threadIdx.x / S::TPR < rows;
  }
};

// Sum over groups of W lanes, the same value in each.
template <int W>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int off = W / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Weights of all of a thread's columns in fp32 pairs (a null array: `fill`).
template <int E, bool RAGGED>
__device__ __forceinline__ void weight_pairs(const void* p, int c, int C, int wdtype, float fill,
                                             uint64_t (&g)[E / 2]) {
  float f[E];
  if (RAGGED) {
    load_weights_ragged<E>(p, c, C, wdtype, fill, f);
  } else {
    Weights<E> w;
    w.load(p, c, wdtype);
    w.get(p, wdtype, fill, f);
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) g[i] = ptx::f2_make(f[2 * i], f[2 * i + 1]);
}

// Forward: the row (its sum with the residual, behind the dropout) is held in
// fp32 registers, in pairs (one instruction for two columns). A warp takes
// the mean of its part and the squares about that; parts of n_w elements are
// joined by
//   mu = sum n_w mu_w / C,  sum of squares = sum (q_w + n_w (mu_w - mu)^2),
// which loses nothing to cancellation and costs one barrier a row.
template <typename T, typename S, int STAGES, bool DROP, bool RAGGED>
__global__ void __launch_bounds__(S::BLOCK, S::BLOCK <= 256 ? 768 / S::BLOCK : 1)
    fwd_kernel(FwdArgs a) {
  constexpr int E = Vec<T>::kElems, TPR = S::TPR, VECS = S::VECS, P = E / 2;
  constexpr bool kKeep = VECS * E <= 16;  // weights stay in registers
  constexpr int kLanes = TPR < 32 ? TPR : 32, kWarps = TPR / kLanes;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float2 part[2][kWarps];
  __shared__ float counts[kWarps];
  const T* const src[2] = {static_cast<const T*>(a.x), static_cast<const T*>(a.residual)};
  const bool add = a.residual != nullptr;
  Walk<T, S, STAGES, 2, RAGGED> w(ring, src, add ? 2 : 1, a.rows, a.C);
  const float inv_C = 1.0f / static_cast<float>(a.C);
  uint64_t gamma[kKeep ? VECS : 1][P], beta[kKeep ? VECS : 1][P];
  int mine = 0;  // this thread's columns inside the row
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int c = w.column(j);
    if (c < a.C) {
      if (kKeep) {
        weight_pairs<E, RAGGED>(a.gamma, c, a.C, a.wdtype, 1.f, gamma[j]);
        weight_pairs<E, RAGGED>(a.beta, c, a.C, a.wdtype, 0.f, beta[j]);
      }
      mine += RAGGED ? min(c + E, a.C) - max(c, 0) : E;
    }
  }
  const float count = lane_sum<kLanes>(static_cast<float>(mine));  // n_w
  const float inv_count = count > 0.f ? 1.0f / count : 0.f;
  if (kWarps > 1 && (threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = count;
  int parity = 0;
  for (; w.more(); w.next()) {
    w.arrive();
    const bool active = w.active();
    uint64_t v[VECS][P], s2 = 0, q2 = 0;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = w.column(j);
      if (active && c < a.C) {
        float f[E];
        w.get(0, j, f);
        if (DROP) drop_vec<E>(f, w.element(j), a.drop);
        if (add) {
          float r[E];
          w.get(1, j, r);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const uint64_t o = ptx::f2_add(ptx::f2_make(f[2 * i], f[2 * i + 1]),
                                           ptx::f2_make(r[2 * i], r[2 * i + 1]));
            f[2 * i] = ptx::f2_lo(o);
            f[2 * i + 1] = ptx::f2_hi(o);
          }
        }
        if (a.z != nullptr)
          store_row_vec<T, RAGGED>(static_cast<T*>(a.z) + w.element(j), f, c, a.C);
        if (RAGGED) keep_inside<E>(f, c, a.C, 0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          v[j][i] = ptx::f2_make(f[2 * i], f[2 * i + 1]);
          s2 = ptx::f2_add(s2, v[j][i]);
        }
      }
    }
    float mu = lane_sum<kLanes>(ptx::f2_lo(s2) + ptx::f2_hi(s2)) *
               (kWarps > 1 ? inv_count : inv_C);
    const uint64_t minus = ptx::f2_make(-mu, -mu);
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = w.column(j);
      if (active && c < a.C) {
        if (RAGGED && (c < 0 || c + E > a.C)) {
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const float d = (i % 2 == 0 ? ptx::f2_lo(v[j][i / 2]) : ptx::f2_hi(v[j][i / 2])) - mu;
            if (static_cast<unsigned>(c + i) < static_cast<unsigned>(a.C))
              q2 = ptx::f2_fma(ptx::f2_make(d, 0.f), ptx::f2_make(d, 0.f), q2);
          }
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const uint64_t d = ptx::f2_add(v[j][i], minus);
            q2 = ptx::f2_fma(d, d, q2);
          }
        }
      }
    }
    float q = lane_sum<kLanes>(ptx::f2_lo(q2) + ptx::f2_hi(q2));
    if (kWarps > 1) {
      if ((threadIdx.x & 31) == 0) part[parity][threadIdx.x >> 5] = make_float2(mu, q);
      __syncthreads();
      const int k = threadIdx.x % kWarps;
      const float2 p = part[parity][k];
      const float n = counts[k];
      mu = lane_sum<kWarps>(n * p.x) * inv_C;
      const float d = p.x - mu;
      q = lane_sum<kWarps>(n > 0.f ? fmaf(n * d, d, p.y) : 0.f);
      parity ^= 1;
    }
    const float r = rsqrtf(fmaf(q, inv_C, a.eps));
    const uint64_t minus_mu = ptx::f2_make(-mu, -mu), r2 = ptx::f2_make(r, r);
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = w.column(j);
      if (active && c < a.C) {
        const int k = kKeep ? j : 0;
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
        store_row_vec<T, RAGGED>(static_cast<T*>(a.y) + w.element(j), f, c, a.C);
      }
    }
    if (active && w.t == 0) {
      if (a.mean != nullptr) a.mean[w.row] = mu;
      if (a.rstd != nullptr) a.rstd[w.row] = r;
    }
  }
  copy_wait<0>();
}

// Backward: a thread's column sums of the weights' gradients stay in
// registers over all of its rows; the two sums of a row are joined over its
// threads with one barrier.
template <typename T, typename S, int STAGES, bool DROP, bool RAGGED>
__global__ void __launch_bounds__(S::BLOCK, 512 / S::BLOCK) bwd_kernel(BwdArgs a) {
  constexpr int E = Vec<T>::kElems, TPR = S::TPR, VECS = S::VECS, BLOCK = S::BLOCK, P = E / 2;
  // up to 16 elements a thread, weights and row stay in registers over the
  // reduction; above, they are read again from L1 and the ring
  constexpr bool kKeep = VECS * E <= 16;
  constexpr int kLanes = TPR < 32 ? TPR : 32, kWarps = TPR / kLanes;
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float2 part[2][kWarps];
  const T* const src[3] = {static_cast<const T*>(a.dy), static_cast<const T*>(a.z),
                           static_cast<const T*>(a.dz)};
  Walk<T, S, STAGES, 3, RAGGED> w(ring, src, a.dz != nullptr ? 3 : 2, a.rows, a.C);
  const float inv_C = 1.0f / static_cast<float>(a.C);
  // the statistics of the row to come, one row ahead
  float mu = 0.f, r = 0.f;
  if (w.active()) {
    mu = a.mean[w.row];
    r = a.rstd[w.row];
  }
  uint64_t dgamma[VECS][P], dbeta[VECS][P], gamma[kKeep ? VECS : 1][P];
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
#pragma unroll
    for (int i = 0; i < P; ++i) dgamma[j][i] = dbeta[j][i] = 0;
    if (kKeep && w.column(j) < a.C)
      weight_pairs<E, RAGGED>(a.gamma, w.column(j), a.C, a.wdtype, 1.f, gamma[j]);
  }
  // dy, (z - mean) rstd and dy gamma of vector j (columns outside the row: 0)
  auto gather = [&](int j, uint64_t (&dy)[P], uint64_t (&h)[P], uint64_t (&g)[P]) {
    float fd[E], fz[E];
    w.get(0, j, fd);
    w.get(1, j, fz);
    if (RAGGED) {
      keep_inside<E>(fd, w.column(j), a.C, 0.f);
      keep_inside<E>(fz, w.column(j), a.C, mu);
    }
    if (!kKeep) weight_pairs<E, RAGGED>(a.gamma, w.column(j), a.C, a.wdtype, 1.f, gamma[0]);
    const uint64_t minus_mu = ptx::f2_make(-mu, -mu), r2 = ptx::f2_make(r, r);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      dy[i] = ptx::f2_make(fd[2 * i], fd[2 * i + 1]);
      h[i] = ptx::f2_mul(ptx::f2_add(ptx::f2_make(fz[2 * i], fz[2 * i + 1]), minus_mu), r2);
      g[i] = ptx::f2_mul(dy[i], gamma[kKeep ? j : 0][i]);
    }
  };
  int parity = 0;
  for (; w.more(); w.next()) {
    const bool active = w.active();
    float mu_next = 0.f, r_next = 0.f;
    if (w.row + w.step < a.rows) {
      mu_next = a.mean[w.row + w.step];
      r_next = a.rstd[w.row + w.step];
    }
    w.arrive();
    uint64_t s2 = 0, u2 = 0;
    uint64_t h[kKeep ? VECS : 1][P], g[kKeep ? VECS : 1][P];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      if (active && w.column(j) < a.C) {
        const int k = kKeep ? j : 0;
        uint64_t dy[P];
        gather(j, dy, h[k], g[k]);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          dgamma[j][i] = ptx::f2_fma(dy[i], h[k][i], dgamma[j][i]);
          dbeta[j][i] = ptx::f2_add(dbeta[j][i], dy[i]);
          s2 = ptx::f2_add(s2, g[k][i]);
          u2 = ptx::f2_fma(g[k][i], h[k][i], u2);
        }
      }
    }
    float s = lane_sum<kLanes>(ptx::f2_lo(s2) + ptx::f2_hi(s2));
    float u = lane_sum<kLanes>(ptx::f2_lo(u2) + ptx::f2_hi(u2));
    if (kWarps > 1) {
      if ((threadIdx.x & 31) == 0) part[parity][threadIdx.x >> 5] = make_float2(s, u);
      __syncthreads();
      const float2 p = part[parity][threadIdx.x % kWarps];
      s = lane_sum<kWarps>(p.x);
      u = lane_sum<kWarps>(p.y);
      parity ^= 1;
    }
    // dz = r g + (-r mean(g h)) h + (-r mean(g)) + dz_in
    const float rs = -r * (s * inv_C), ru = -r * (u * inv_C);
    const uint64_t r2 = ptx::f2_make(r, r), rs2 = ptx::f2_make(rs, rs), ru2 = ptx::f2_make(ru, ru);
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = w.column(j);
      if (active && c < a.C) {
        const int k = kKeep ? j : 0;
        if (!kKeep) {
          uint64_t dy[P];
          gather(j, dy, h[0], g[0]);
        }
        float f[E];
        if (a.dz != nullptr) {
          w.get(2, j, f);
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) f[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const uint64_t v = ptx::f2_fma(g[k][i], r2, ptx::f2_fma(h[k][i], ru2, rs2));
          const uint64_t o = ptx::f2_add(v, ptx::f2_make(f[2 * i], f[2 * i + 1]));
          f[2 * i] = ptx::f2_lo(o);
          f[2 * i + 1] = ptx::f2_hi(o);
        }
        store_row_vec<T, RAGGED>(static_cast<T*>(a.dres) + w.element(j), f, c, a.C);
        if (a.dx != nullptr) {
          if (DROP) drop_vec<E>(f, w.element(j), a.drop);
          store_row_vec<T, RAGGED>(static_cast<T*>(a.dx) + w.element(j), f, c, a.C);
        }
      }
    }
    mu = mu_next;
    r = r_next;
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
    // the row groups of the block add up in shared memory, one after another
    float* sum = reinterpret_cast<float*>(ring);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.C; i += BLOCK) sum[i] = 0.f;
    for (int k = 0; k < S::ROWS; ++k) {
      __syncthreads();
      if (k == threadIdx.x / TPR)
        columns([&](int c, float x, float y) {
          sum[c] += x;
          sum[a.C + c] += y;
        });
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.C; i += BLOCK) out[i] = sum[i];
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
// so that the backward's sums stay in registers.
template <typename T, typename F>
int with_shape(int C, F f) {
  constexpr int E = Vec<T>::kElems;
  // a ragged row takes up to one vector more than its length needs
  const int n = C % E == 0 ? C : C + 2 * E - 2;
  if (n <= 64) return f(Shape<8, 8 / E>{});
  if (n <= 128) return f(Shape<8, 16 / E>{});
  if (n <= 256) return f(Shape<16, 16 / E>{});
  if (n <= 512) return f(Shape<32, 16 / E>{});
  if (n <= 1024) return f(Shape<128, 8 / E>{});
  if (n <= 2048) return f(Shape<128, 16 / E>{});
  if (n <= 4096) return f(Shape<256, 16 / E>{});
  if (n <= 8192) return f(Shape<512, 16 / E>{});
  return f(Shape<512, 32 / E>{});
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
// negative error. ring(tensors): its shared memory.
template <typename S, int TENSORS, typename Kernel, typename Args>
int launch_walk(Kernel kern, const Args& a, int tensors, int stages, int least_smem,
                long long most, std::atomic<bool> (&limit_set)[kMaxTrackedDevices],
                std::atomic<int> (&resident)[2][kMaxTrackedDevices], cudaStream_t stream) {
  const int stage_bytes = S::VECS * S::BLOCK * 16;
  const int smem = std::max(stages * tensors * stage_bytes, least_smem);
  if (!set_smem_limit_once(kern, stages * TENSORS * stage_bytes, limit_set))
    return ATTN_ERR_LAUNCH;
  const int per_sm = blocks_per_sm(kern, S::BLOCK, smem, resident[TENSORS - tensors]);
  if (per_sm <= 0) return ATTN_ERR_LAUNCH;
  long long grid = static_cast<long long>(sm_count() > 0 ? sm_count() : 1) * per_sm;
  grid = std::max(8LL, std::min(grid, most) / 8 * 8);
  grid = std::min(grid, ((a.rows + S::ROWS - 1) / S::ROWS + 7) / 8 * 8);
  kern<<<static_cast<unsigned>(grid), S::BLOCK, smem, stream>>>(a);
  const int rc = launch_status();
  return rc != ATTN_OK ? rc : static_cast<int>(grid);
}

// Stages of a ring of rows of `bytes`: four within 48 KB a tensor, so that
// several blocks share an SM, and what fits beyond.
constexpr int stages_for(int tensors, int bytes) {
  return tensors * bytes <= 32768 ? 4 : (tensors * bytes * 2 <= 196608 ? 2 : 1);
}

template <typename T, bool DROP, bool RAGGED>
int fwd_rows(const FwdArgs& a, cudaStream_t stream) {
  return with_shape<T>(a.C, [&](auto shape) {
    using S = decltype(shape);
    static std::atomic<bool> limit_set[kMaxTrackedDevices];
    static std::atomic<int> resident[2][kMaxTrackedDevices];
    constexpr int kStages = stages_for(2, S::VECS * S::BLOCK * 16);
    const int n = launch_walk<S, 2>(fwd_kernel<T, S, kStages, DROP, RAGGED>, a,
                                    a.residual != nullptr ? 2 : 1, kStages, 0, 1LL << 20,
                                    limit_set, resident, stream);
    return n < 0 ? n : static_cast<int>(ATTN_OK);
  });
}

template <typename T>
int run_fwd(const FwdArgs& a, cudaStream_t stream) {
  if (!fits<T>(a.C)) {
    fwd_wide_kernel<T><<<grid_for(a.rows), kThreads, 0, stream>>>(a);
    return launch_status();
  }
  const bool ragged = a.C % Vec<T>::kElems != 0;
  if (a.drop.on)
    return ragged ? fwd_rows<T, true, true>(a, stream) : fwd_rows<T, true, false>(a, stream);
  return ragged ? fwd_rows<T, false, true>(a, stream) : fwd_rows<T, false, false>(a, stream);
}

template <typename T, bool DROP, bool RAGGED>
int bwd_rows(const BwdArgs& a, cudaStream_t stream) {
  return with_shape<T>(a.C, [&](auto shape) {
    using S = decltype(shape);
    static std::atomic<bool> limit_set[kMaxTrackedDevices];
    static std::atomic<int> resident[2][kMaxTrackedDevices];
    constexpr int kStages = stages_for(3, S::VECS * S::BLOCK * 16);
    // the block's sums of short rows go through the ring's memory
    return launch_walk<S, 3>(bwd_kernel<T, S, kStages, DROP, RAGGED>, a,
                             a.dz != nullptr ? 3 : 2, kStages, S::ROWS > 1 ? 2 * a.C * 4 : 0,
                             kMaxChunks, limit_set, resident, stream);
  });
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
  const bool ragged = a.C % Vec<T>::kElems != 0;
  if (a.drop.on)
    return ragged ? bwd_rows<T, true, true>(a, stream) : bwd_rows<T, true, false>(a, stream);
  return ragged ? bwd_rows<T, false, true>(a, stream) : bwd_rows<T, false, false>(a, stream);
}

}  // namespace norm
}  // namespace attn
