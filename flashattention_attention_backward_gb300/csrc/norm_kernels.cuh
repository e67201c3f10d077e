// The layer-norm kernels for one element type: rows of up to kMaxRow columns
// stay on chip (registers forward, a shared-memory ring backward), wider ones
// are read again.
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

namespace attn {
namespace norm {

template <int TPR_, int VECS_>
struct Shape {
  static constexpr int TPR = TPR_;    // threads per row
  static constexpr int VECS = VECS_;  // 16-byte vectors per thread
  static constexpr int BLOCK = TPR_ <= 32 ? 256 : TPR_;
  static constexpr int ROWS = BLOCK / TPR_;  // rows of a block at a time
};

// The E weights (or biases) of columns c .. c + E - 1, `fill` where there are
// none: outside the row, or no array.
template <int E, bool RAGGED>
__device__ __forceinline__ void load_weights(const void* p, int c, int C, int wdtype, float fill,
                                             float (&f)[E]) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = fill;
  } else if (RAGGED) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      f[i] = static_cast<unsigned>(c + i) < static_cast<unsigned>(C) ? load_as(p, c + i, wdtype)
                                                                     : fill;
  } else if (wdtype == ATTN_FP32) {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + i);
      f[i] = v.x;
      f[i + 1] = v.y;
      f[i + 2] = v.z;
      f[i + 3] = v.w;
    }
  } else {  // c is a multiple of four: 8 bytes
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c + i);
      const uint32_t w[2] = {v.x, v.y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (wdtype == ATTN_BF16) {
          f[i + 2 * j] = __uint_as_float(w[j] << 16);
          f[i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
          const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
          f[i + 2 * j] = h.x;
          f[i + 2 * j + 1] = h.y;
        }
      }
    }
  }
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

// Sum over a row's threads, the same value in each. `part` is this
// reduction's own: TPR / 32 floats (unused for TPR <= 32).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int off = (TPR < 32 ? TPR : 32) / 2; off >= 1; off >>= 1)
    v += __shfl_xor_sync(0xffffffffu, v, off);
  if (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += part[i];
  }
  return v;
}

// Forward: the row (its sum with the residual, behind the dropout) stays in
// fp32 registers; mean first, then the squares about it, then the output.
template <typename T, typename S, bool DROP, bool RAGGED>
__global__ void __launch_bounds__(S::BLOCK) fwd_kernel(FwdArgs a) {
  constexpr int E = Vec<T>::kElems, TPR = S::TPR, VECS = S::VECS;
  __shared__ float part[2][TPR > 32 ? TPR / 32 : 1];
  const int t = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * S::ROWS + threadIdx.x / TPR;
  const bool active = row < a.rows;
  const long long base = row * a.C;
  const int shift = RAGGED ? static_cast<int>(base % E) : 0;
  auto column = [&](int j) { return (t + j * TPR) * E - shift; };
  auto inside = [&](int j) { return active && column(j) < a.C; };
  auto valid = [&](int c) {
    return !RAGGED || static_cast<unsigned>(c) < static_cast<unsigned>(a.C);
  };

  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  const T* x_end = x + a.rows * a.C;
  const T* res_end = res != nullptr ? res + a.rows * a.C : nullptr;
  float v[VECS][E];
  {
    Vec<T> vx[VECS], vr[VECS];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      if (inside(j)) {
        vx[j] = load_row_vec<T, RAGGED>(x + base + column(j), x_end);
        if (res != nullptr) vr[j] = load_row_vec<T, RAGGED>(res + base + column(j), res_end);
      }
    }
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
#pragma unroll
      for (int i = 0; i < E; ++i) v[j][i] = 0.f;
      if (inside(j)) {
        unpack(vx[j], v[j]);
        if (DROP) {
          uint32_t w[E / 4][4];
          keep_words<E / 4>(base + column(j), a.drop, w);
#pragma unroll
          for (int i = 0; i < E; ++i)
            v[j][i] = w[i / 4][i % 4] >= a.drop.threshold ? v[j][i] * a.drop.inv_keep : 0.f;
        }
        if (res != nullptr) {
          float r[E];
          unpack(vr[j], r);
#pragma unroll
          for (int i = 0; i < E; ++i) v[j][i] += r[i];
        }
        if (a.z != nullptr)
          store_row_vec<T, RAGGED>(static_cast<T*>(a.z) + base + column(j), v[j], column(j), a.C);
      }
    }
  }
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < VECS; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (valid(column(j) + i)) s += v[j][i];
  const float mu = row_sum<TPR>(s, part[0]) / a.C;
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < VECS; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (inside(j) && valid(column(j) + i)) {
        const float d = v[j][i] - mu;
        q = fmaf(d, d, q);
      }
  const float r = 1.0f / sqrtf(row_sum<TPR>(q, part[1]) / a.C + a.eps);
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    if (inside(j)) {
      float g[E], b[E];
      load_weights<E, RAGGED>(a.gamma, column(j), a.C, a.wdtype, 1.f, g);
      load_weights<E, RAGGED>(a.beta, column(j), a.C, a.wdtype, 0.f, b);
#pragma unroll
      for (int i = 0; i < E; ++i) v[j][i] = fmaf((v[j][i] - mu) * r, g[i], b[i]);
      store_row_vec<T, RAGGED>(static_cast<T*>(a.y) + base + column(j), v[j], column(j), a.C);
    }
  }
  if (active && t == 0) {
    if (a.mean != nullptr) a.mean[row] = mu;
    if (a.rstd != nullptr) a.rstd[row] = r;
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

// Backward: blocks stay and take rows grid apart, so that a thread's columns
// are the same in all of its rows and it sums their weight gradients in
// registers. (RAGGED: the grid is a multiple of 8 blocks, so all of a
// thread's rows start at the same offset within a vector.) Rows come through
// a ring of STAGES in shared memory, filled by asynchronous copies: a thread
// reads back only what it copied itself, so the ring needs no barrier, and
// the loads of the next rows run while this one is reduced.
template <typename T, typename S, int STAGES, bool DROP, bool RAGGED>
__global__ void __launch_bounds__(S::BLOCK) bwd_kernel(BwdArgs a) {
  constexpr int E = Vec<T>::kElems, TPR = S::TPR, VECS = S::VECS, BLOCK = S::BLOCK;
  constexpr int kWarps = TPR > 32 ? TPR / 32 : 1;
  extern __shared__ __align__(16) uint4 ring[];  // [STAGES][2 or 3][VECS][BLOCK]
  __shared__ float2 part[2][kWarps];
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int tensors = a.dz != nullptr ? 3 : 2;
  const T* const src[3] = {static_cast<const T*>(a.dy), static_cast<const T*>(a.z),
                           static_cast<const T*>(a.dz)};
  const long long total = a.rows * a.C;
  const long long first = static_cast<long long>(blockIdx.x) * S::ROWS;
  const long long step = static_cast<long long>(gridDim.x) * S::ROWS;
  const int shift = RAGGED ? static_cast<int>(((first + group) * a.C) % E) : 0;
  auto column = [&](int j) { return (t + j * TPR) * E - shift; };
  auto valid = [&](int c) {
    return !RAGGED || static_cast<unsigned>(c) < static_cast<unsigned>(a.C);
  };
  auto slot = [&](int stage, int q, int j) {
    return &ring[((stage * tensors + q) * VECS + j) * BLOCK + threadIdx.x];
  };
  auto fetch = [&](long long row, int stage) {
    if (row < a.rows) {
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        if (column(j) < a.C) {
          const long long e = row * a.C + column(j);
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            if (q < tensors) {
              if (!RAGGED || e + E <= total)
                copy_async16(slot(stage, q, j), src[q] + e);
              else
                *reinterpret_cast<Vec<T>*>(slot(stage, q, j)) =
                    load_row_vec<T, RAGGED>(src[q] + e, src[q] + total);
            }
          }
        }
      }
    }
    copy_commit();
  };

  float dgamma[VECS][E], dbeta[VECS][E];
#pragma unroll
  for (int j = 0; j < VECS; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i) dgamma[j][i] = dbeta[j][i] = 0.f;
#pragma unroll
  for (int k = 0; k < STAGES - 1; ++k) fetch(first + group + k * step, k);
  // the statistics of the row to come, one row ahead
  float mu = 0.f, r = 0.f;
  if (first + group < a.rows) {
    mu = a.mean[first + group];
    r = a.rstd[first + group];
  }
  int stage = 0, parity = 0;
  for (long long block_row = first; block_row < a.rows; block_row += step) {
    const long long row = block_row + group;
    const bool active = row < a.rows;
    const long long base = row * a.C;
    fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    float mu_next = 0.f, r_next = 0.f;
    if (row + step < a.rows) {
      mu_next = a.mean[row + step];
      r_next = a.rstd[row + step];
    }
    copy_wait<STAGES - 1>();
    float s = 0.f, u = 0.f;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = column(j);
      if (active && c < a.C) {
        float dy[E], h[E], g[E];
        unpack(*reinterpret_cast<const Vec<T>*>(slot(stage, 0, j)), dy);
        unpack(*reinterpret_cast<const Vec<T>*>(slot(stage, 1, j)), h);
        load_weights<E, RAGGED>(a.gamma, c, a.C, a.wdtype, 1.f, g);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if (!valid(c + i)) continue;
          h[i] = (h[i] - mu) * r;
          dgamma[j][i] = fmaf(dy[i], h[i], dgamma[j][i]);
          dbeta[j][i] += dy[i];
          g[i] *= dy[i];
          s += g[i];
          u = fmaf(g[i], h[i], u);
        }
      }
    }
    // both sums over the row's threads
#pragma unroll
    for (int off = (TPR < 32 ? TPR : 32) / 2; off >= 1; off >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, off);
      u += __shfl_xor_sync(0xffffffffu, u, off);
    }
    if (TPR > 32) {
      if ((threadIdx.x & 31) == 0) part[parity][threadIdx.x >> 5] = make_float2(s, u);
      __syncthreads();
      s = u = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        s += part[parity][i].x;
        u += part[parity][i].y;
      }
      parity ^= 1;
    }
    s /= a.C;
    u /= a.C;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = column(j);
      if (active && c < a.C) {
        float dy[E], h[E], g[E];
        unpack(*reinterpret_cast<const Vec<T>*>(slot(stage, 0, j)), dy);
        unpack(*reinterpret_cast<const Vec<T>*>(slot(stage, 1, j)), h);
        load_weights<E, RAGGED>(a.gamma, c, a.C, a.wdtype, 1.f, g);
#pragma unroll
        for (int i = 0; i < E; ++i) dy[i] = r * (g[i] * dy[i] - s - (h[i] - mu) * r * u);
        if (a.dz != nullptr) {
          unpack(*reinterpret_cast<const Vec<T>*>(slot(stage, 2, j)), h);
#pragma unroll
          for (int i = 0; i < E; ++i) dy[i] += h[i];
        }
        store_row_vec<T, RAGGED>(static_cast<T*>(a.dres) + base + c, dy, c, a.C);
        if (a.dx != nullptr) {
          if (DROP) {
            uint32_t w[E / 4][4];
            keep_words<E / 4>(base + c, a.drop, w);
#pragma unroll
            for (int i = 0; i < E; ++i)
              dy[i] = w[i / 4][i % 4] >= a.drop.threshold ? dy[i] * a.drop.inv_keep : 0.f;
          }
          store_row_vec<T, RAGGED>(static_cast<T*>(a.dx) + base + c, dy, c, a.C);
        }
      }
    }
    mu = mu_next;
    r = r_next;
    stage = stage == STAGES - 1 ? 0 : stage + 1;
  }
  copy_wait<0>();
  if (a.workspace == nullptr) return;
  float* out = a.workspace + 2LL * blockIdx.x * a.C;
  if (S::ROWS == 1) {
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = column(j);
      if (c >= a.C) continue;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (!valid(c + i)) continue;
        out[c + i] = dgamma[j][i];
        out[a.C + c + i] = dbeta[j][i];
      }
    }
  } else {
    // the row groups of the block add up in shared memory, one after another
    float* sum = reinterpret_cast<float*>(ring);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.C; i += BLOCK) sum[i] = 0.f;
    for (int k = 0; k < S::ROWS; ++k) {
      __syncthreads();
      if (k != group) continue;
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        const int c = column(j);
        if (c >= a.C) continue;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if (!valid(c + i)) continue;
          sum[c + i] += dgamma[j][i];
          sum[a.C + c + i] += dbeta[j][i];
        }
      }
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

// f(Shape) for the row length: 8 elements a thread up to a warp's width, then
// 16 (32 for the widest), so that the backward's sums stay in registers.
template <typename T, bool BACKWARD, typename F>
int with_shape(int C, F f) {
  constexpr int E = Vec<T>::kElems;
  // a ragged row takes one vector more than its length needs
  const int n = C % E == 0 ? C : C + 2 * E - 2;
  if (n <= 64) return f(Shape<8, 8 / E>{});
  if (n <= 128) return f(Shape<16, 8 / E>{});
  if (n <= 256) return f(Shape<32, 8 / E>{});
  if (n <= 512) return f(Shape<32, 16 / E>{});
  // a warp a row in the backward, whose blocks are few
  if (n <= 1024) return f(Shape<BACKWARD ? 32 : 64, (BACKWARD ? 32 : 16) / E>{});
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

template <typename T, bool DROP, bool RAGGED>
int fwd_rows(const FwdArgs& a, cudaStream_t stream) {
  return with_shape<T, false>(a.C, [&](auto shape) {
    using S = decltype(shape);
    const long long blocks = (a.rows + S::ROWS - 1) / S::ROWS;
    if (blocks > 0x7fffffffLL) return static_cast<int>(ATTN_ERR_TOO_LARGE);
    fwd_kernel<T, S, DROP, RAGGED><<<static_cast<unsigned>(blocks), S::BLOCK, 0, stream>>>(a);
    return launch_status();
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

// Blocks of a kernel that fit an SM at a time (cached per device by the
// caller's record); 0 on error.
template <typename Kernel>
int blocks_per_sm(Kernel kern, int block, int smem, std::atomic<int> (&cache)[kMaxTrackedDevices]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool tracked = dev >= 0 && dev < kMaxTrackedDevices;
  if (tracked && cache[dev].load(std::memory_order_relaxed) > 0)
    return cache[dev].load(std::memory_order_relaxed);
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, block, smem) != cudaSuccess) return 0;
  if (tracked) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <typename T, typename S, int STAGES, bool DROP, bool RAGGED>
int launch_bwd(const BwdArgs& a, cudaStream_t stream) {
  static std::atomic<bool> limit_set[kMaxTrackedDevices];
  static std::atomic<int> resident[2][kMaxTrackedDevices];
  auto kern = bwd_kernel<T, S, STAGES, DROP, RAGGED>;
  const int tensors = a.dz != nullptr ? 3 : 2;
  const int smem = std::max(STAGES * tensors * S::VECS * S::BLOCK * 16,
                            S::ROWS > 1 ? 2 * a.C * 4 : 0);
  if (!set_smem_limit_once(kern, STAGES * 3 * S::VECS * S::BLOCK * 16, limit_set))
    return ATTN_ERR_LAUNCH;
  const int per_sm = blocks_per_sm(kern, S::BLOCK, smem, resident[tensors - 2]);
  if (per_sm <= 0) return ATTN_ERR_LAUNCH;
  long long grid = static_cast<long long>(sm_count() > 0 ? sm_count() : 1) * per_sm;
  grid = std::max(8LL, std::min<long long>(grid, kMaxChunks) / 8 * 8);
  grid = std::min(grid, ((a.rows + S::ROWS - 1) / S::ROWS + 7) / 8 * 8);
  kern<<<static_cast<unsigned>(grid), S::BLOCK, smem, stream>>>(a);
  const int rc = launch_status();
  return rc != ATTN_OK ? rc : static_cast<int>(grid);
}

template <typename T, bool DROP, bool RAGGED>
int bwd_rows(const BwdArgs& a, cudaStream_t stream) {
  return with_shape<T, true>(a.C, [&](auto shape) {
    using S = decltype(shape);
    // at most 192 KB: two stages of three tensors of the widest rows
    constexpr int kStageBytes = 3 * S::VECS * S::BLOCK * 16;
    constexpr int kStages = kStageBytes <= 32768 ? 4 : (kStageBytes * 2 <= 196608 ? 2 : 1);
    return launch_bwd<T, S, kStages, DROP, RAGGED>(a, stream);
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
