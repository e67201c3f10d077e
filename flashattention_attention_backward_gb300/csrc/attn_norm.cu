// Layer norm, dropout with a residual, and the two together, forward and
// backward.
//
//   z = residual + x Z / (1 - p)          (dropout add; Z the keep mask)
//   mu = mean(z), r = (mean((z - mu)^2) + eps)^(-1/2), h = (z - mu) r
//   y = gamma h + beta                    (layer norm over a row's C columns)
// and back, with g = dy gamma:
//   dz = r (g - mean(g) - h mean(g h)) + dz_in
//   dresidual = dz, dx = dz Z / (1 - p)
//   dgamma = sum over rows of dy h, dbeta = sum over rows of dy.
//
// Keep mask: element e (row-major, e = row C + column) is kept iff word
// e mod 4 of Philox4x32-10(counter = (floor(e / 4) mod 2^32,
// floor(e / 2^34), 0, 1), key = (seed mod 2^32, seed >> 32)) is >=
// round(p 2^32). The fourth counter word is 1 where the attention's own
// dropout has 0, so one seed serves both without a common word. Nothing of
// the mask is stored; the backward draws it again.
#include <cmath>
#include <cstdint>

#include "element.cuh"
#include "philox.cuh"

namespace attn {
namespace norm {

constexpr int kThreads = 256;
// Row chunks of the weight gradients' first stage: the workspace holds two
// fp32 sums a column for each.
constexpr int kMaxChunks = 1024;

struct Drop {
  uint32_t seed_lo, seed_hi, threshold;
  float inv_keep;
  int on;
};

inline Drop make_drop(float p, unsigned long long seed) {
  Drop d;
  d.seed_lo = static_cast<uint32_t>(seed);
  d.seed_hi = static_cast<uint32_t>(seed >> 32);
  d.threshold = dropout_threshold(p);
  d.inv_keep = static_cast<float>(1.0 / (1.0 - static_cast<double>(p)));
  d.on = p > 0.0f;
  return d;
}

__device__ __forceinline__ bool kept(long long e, const Drop& d) {
  const PhiloxOut w = philox4x32_10(static_cast<uint32_t>(e >> 2), static_cast<uint32_t>(e >> 34),
                                    0u, 1u, d.seed_lo, d.seed_hi);
  return w.w[e & 3] >= d.threshold;
}

// Keep words of the 4 NB elements from e (a multiple of 4) on.
template <int NB>
__device__ __forceinline__ void keep_words(long long e, const Drop& d, uint32_t (&w)[NB][4]) {
#pragma unroll
  for (int u = 0; u < NB; ++u) {
    const long long c = (e >> 2) + u;
    w[u][0] = static_cast<uint32_t>(c);
    w[u][1] = static_cast<uint32_t>(c >> 32);
    w[u][2] = 0u;
    w[u][3] = 1u;
  }
  philox4x32_10_batch<NB, 10>(w, d.seed_lo, d.seed_hi);
}

// One thread per 16 bytes: a group of 16-byte loads is in flight on every
// lane, and the mask words (two generator calls per 8 elements) are drawn
// behind them.
template <typename T, bool DROP>
__global__ void __launch_bounds__(kThreads)
    dropout_add_kernel(const T* x, const T* residual, T* y, long long n, Drop drop) {
  constexpr int E = Vec<T>::kElems;
  const long long e = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) * E;
  if (e >= n) return;
  const bool whole = e + E <= n;
  float v[E], r[E];
  Vec<T> vx, vr;
  if (whole) {
    vx = load_vec(x + e);
    if (residual != nullptr) vr = load_vec(residual + e);
  }
  uint32_t w[E / 4][4];
  if (DROP) keep_words<E / 4>(e, drop, w);
  if (whole) {
    unpack(vx, v);
    if (residual != nullptr) unpack(vr, r);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      v[i] = e + i < n ? to_f32(x[e + i]) : 0.f;
      r[i] = residual != nullptr && e + i < n ? to_f32(residual[e + i]) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (DROP) v[i] = w[i / 4][i % 4] >= drop.threshold ? v[i] * drop.inv_keep : 0.f;
    if (residual != nullptr) v[i] += r[i];
  }
  if (whole) {
    Vec<T> o;
    pack(v, o);
    store_vec(y + e, o);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (e + i < n) y[e + i] = from_f32<T>(v[i]);
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

struct FwdArgs {
  const void *x, *residual, *gamma, *beta;  // residual NULL: plain layer norm
  void *z, *y;
  float *mean, *rstd;
  long long rows;
  int C, wdtype;
  float eps;
  Drop drop;
};

// One block per row; the row is read three times.
template <typename T>
__global__ void __launch_bounds__(kThreads) fwd_kernel(FwdArgs a) {
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

struct BwdArgs {
  const void *dy, *dz, *z, *gamma;  // dz NULL: nothing to add
  const float *mean, *rstd;
  void *dx, *dres;  // dx: behind the dropout, or NULL; dres: dz itself
  void *dgamma, *dbeta;
  float* workspace;
  long long rows;
  int C, wdtype;
  Drop drop;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) bwd_kernel(BwdArgs a) {
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

// First stage of the weight gradients: 32 columns by a chunk of rows.
template <typename T>
__global__ void __launch_bounds__(kThreads) weights_kernel(BwdArgs a, long long rows_per_chunk) {
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

// Second stage: the chunks of a column, in order.
__global__ void __launch_bounds__(kThreads) weights_sum_kernel(BwdArgs a, int chunks) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= 2 * a.C) return;
  const int c = i < a.C ? i : i - a.C;
  void* out = i < a.C ? a.dgamma : a.dbeta;
  if (out == nullptr) return;
  float v = 0.f;
  for (int k = 0; k < chunks; ++k) v += a.workspace[(2LL * k + (i < a.C ? 0 : 1)) * a.C + c];
  store_as(out, c, a.wdtype, v);
}

int check(long long rows, int C, int dtype, int wdtype) {
  if (rows < 0 || C <= 0) return ATTN_ERR_SHAPE;
  if (!known_dtype(dtype) || !known_dtype(wdtype)) return ATTN_ERR_UNSUPPORTED;
  if (rows >= (1LL << 40) / C) return ATTN_ERR_TOO_LARGE;
  return ATTN_OK;
}

inline bool bad_p(float p) { return !(p >= 0.0f && p < 1.0f); }

inline unsigned grid_for(long long want) {
  const long long cap = static_cast<long long>(sm_count() > 0 ? sm_count() : 1) * 8;
  return static_cast<unsigned>(want < cap ? want : cap);
}

int run_fwd(const FwdArgs& a, int dtype, cudaStream_t stream) {
  if (a.rows == 0) return ATTN_OK;
  return with_dtype(dtype, [&](auto t) {
    fwd_kernel<decltype(t)><<<grid_for(a.rows), kThreads, 0, stream>>>(a);
    return launch_status();
  });
}

inline int chunks_for(long long rows) {
  const long long n = (rows + 63) / 64;
  return static_cast<int>(n < kMaxChunks ? (n > 0 ? n : 1) : kMaxChunks);
}

int run_bwd(const BwdArgs& a, int dtype, cudaStream_t stream) {
  const bool weights = a.dgamma != nullptr || a.dbeta != nullptr;
  if (a.rows == 0 && !weights) return ATTN_OK;
  const int chunks = chunks_for(a.rows);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    if (weights) {
      const long long per = (a.rows + chunks - 1) / chunks;
      const dim3 grid(static_cast<unsigned>((a.C + 31) / 32), static_cast<unsigned>(chunks));
      weights_kernel<T><<<grid, kThreads, 0, stream>>>(a, per);
      weights_sum_kernel<<<(2 * a.C + kThreads - 1) / kThreads, kThreads, 0, stream>>>(a, chunks);
    }
    if (a.rows > 0) bwd_kernel<T><<<grid_for(a.rows), kThreads, 0, stream>>>(a);
    return launch_status();
  });
}

}  // namespace norm
}  // namespace attn

using namespace attn;

extern "C" int attn_layer_norm(const void* x, const void* gamma, const void* beta, void* y,
                               float* mean, float* rstd, long long rows, int C, float eps,
                               int dtype, int wdtype, void* stream) {
  if (rows > 0 && (!x || !y)) return ATTN_ERR_NULL;
  const int rc = norm::check(rows, C, dtype, wdtype);
  if (rc != ATTN_OK) return rc;
  if (!std::isfinite(eps) || eps < 0.0f) return ATTN_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(y) ||
      !aligned16(mean) || !aligned16(rstd))
    return ATTN_ERR_ALIGN;
  norm::FwdArgs a{};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.C = C;
  a.wdtype = wdtype;
  a.eps = eps;
  return norm::run_fwd(a, dtype, as_stream(stream));
}

extern "C" int attn_dropout_add(const void* x, const void* residual, void* y, long long n,
                                float p_drop, unsigned long long seed, int dtype, void* stream) {
  if (n > 0 && (!x || !y)) return ATTN_ERR_NULL;
  if (n < 0 || norm::bad_p(p_drop)) return ATTN_ERR_SHAPE;
  if (!known_dtype(dtype)) return ATTN_ERR_UNSUPPORTED;
  if (n >= (1LL << 40)) return ATTN_ERR_TOO_LARGE;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(y)) return ATTN_ERR_ALIGN;
  if (n == 0) return ATTN_OK;
  const norm::Drop drop = norm::make_drop(p_drop, seed);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const T *xt = static_cast<const T*>(x), *rt = static_cast<const T*>(residual);
    const long long per_block = norm::kThreads * static_cast<long long>(Vec<T>::kElems);
    const unsigned grid = static_cast<unsigned>((n + per_block - 1) / per_block);
    if (drop.on)
      norm::dropout_add_kernel<T, true>
          <<<grid, norm::kThreads, 0, as_stream(stream)>>>(xt, rt, static_cast<T*>(y), n, drop);
    else
      norm::dropout_add_kernel<T, false>
          <<<grid, norm::kThreads, 0, as_stream(stream)>>>(xt, rt, static_cast<T*>(y), n, drop);
    return launch_status();
  });
}

extern "C" int attn_dropout_add_norm(const void* x, const void* residual, const void* gamma,
                                     const void* beta, void* z, void* y, float* mean, float* rstd,
                                     long long rows, int C, float eps, float p_drop,
                                     unsigned long long seed, int dtype, int wdtype,
                                     void* stream) {
  if (rows > 0 && (!x || !residual || !z || !y)) return ATTN_ERR_NULL;
  const int rc = norm::check(rows, C, dtype, wdtype);
  if (rc != ATTN_OK) return rc;
  if (!std::isfinite(eps) || eps < 0.0f || norm::bad_p(p_drop) || (z != nullptr && z == y))
    return ATTN_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(gamma) || !aligned16(beta) ||
      !aligned16(z) || !aligned16(y) || !aligned16(mean) || !aligned16(rstd))
    return ATTN_ERR_ALIGN;
  norm::FwdArgs a{};
  a.x = x;
  a.residual = residual;
  a.gamma = gamma;
  a.beta = beta;
  a.z = z;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.C = C;
  a.wdtype = wdtype;
  a.eps = eps;
  a.drop = norm::make_drop(p_drop, seed);
  return norm::run_fwd(a, dtype, as_stream(stream));
}

extern "C" long long attn_layer_norm_bwd_workspace_bytes(long long rows, int C) {
  const int rc = norm::check(rows, C, ATTN_BF16, ATTN_BF16);
  if (rc != ATTN_OK) return rc;
  return static_cast<long long>(norm::chunks_for(rows)) * 2 * C *
         static_cast<long long>(sizeof(float));
}

extern "C" int attn_layer_norm_bwd(const void* dy, const void* x, const void* gamma,
                                   const float* mean, const float* rstd, void* dx, void* dgamma,
                                   void* dbeta, float* workspace, long long rows, int C, int dtype,
                                   int wdtype, void* stream) {
  if ((rows > 0 && (!dy || !x || !mean || !rstd || !dx)) || ((dgamma || dbeta) && !workspace))
    return ATTN_ERR_NULL;
  const int rc = norm::check(rows, C, dtype, wdtype);
  if (rc != ATTN_OK) return rc;
  if (!aligned16(dy) || !aligned16(x) || !aligned16(gamma) || !aligned16(mean) ||
      !aligned16(rstd) || !aligned16(dx) || !aligned16(dgamma) || !aligned16(dbeta) ||
      !aligned16(workspace))
    return ATTN_ERR_ALIGN;
  norm::BwdArgs a{};
  a.dy = dy;
  a.z = x;
  a.gamma = gamma;
  a.mean = mean;
  a.rstd = rstd;
  a.dres = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.workspace = workspace;
  a.rows = rows;
  a.C = C;
  a.wdtype = wdtype;
  return norm::run_bwd(a, dtype, as_stream(stream));
}

extern "C" int attn_dropout_add_norm_bwd(const void* dy, const void* dz, const void* z,
                                         const void* gamma, const float* mean, const float* rstd,
                                         void* dx, void* dresidual, void* dgamma, void* dbeta,
                                         float* workspace, long long rows, int C, float p_drop,
                                         unsigned long long seed, int dtype, int wdtype,
                                         void* stream) {
  // without dropout dx and dresidual are the same, and dx may be left out
  if ((rows > 0 && (!dy || !z || !mean || !rstd || !dresidual || (!dx && p_drop != 0.0f))) ||
      ((dgamma || dbeta) && !workspace))
    return ATTN_ERR_NULL;
  const int rc = norm::check(rows, C, dtype, wdtype);
  if (rc != ATTN_OK) return rc;
  if (norm::bad_p(p_drop) || (dx != nullptr && dx == dresidual)) return ATTN_ERR_SHAPE;
  if (!aligned16(dy) || !aligned16(dz) || !aligned16(z) || !aligned16(gamma) || !aligned16(mean) ||
      !aligned16(rstd) || !aligned16(dx) || !aligned16(dresidual) || !aligned16(dgamma) ||
      !aligned16(dbeta) || !aligned16(workspace))
    return ATTN_ERR_ALIGN;
  norm::BwdArgs a{};
  a.dy = dy;
  a.dz = dz;
  a.z = z;
  a.gamma = gamma;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  a.dres = dresidual;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.workspace = workspace;
  a.rows = rows;
  a.C = C;
  a.wdtype = wdtype;
  a.drop = norm::make_drop(p_drop, seed);
  return norm::run_bwd(a, dtype, as_stream(stream));
}
