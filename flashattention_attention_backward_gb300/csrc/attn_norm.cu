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

#include "grid_ptx.cuh"
#include "norm_common.cuh"

namespace attn {
namespace norm {

inline Drop make_drop(float p, unsigned long long seed) {
  Drop d;
  for (uint32_t r = 0; r < 10; ++r) {
    d.key[r][0] = static_cast<uint32_t>(seed) + r * 0x9E3779B9u;
    d.key[r][1] = static_cast<uint32_t>(seed >> 32) + r * 0xBB67AE85u;
  }
  d.threshold = dropout_threshold(p);
  d.inv_keep = static_cast<float>(1.0 / (1.0 - static_cast<double>(p)));
  d.on = p > 0.0f;
  return d;
}

// A thread takes 16 bytes: both loads go out first, the mask words (a
// generator call per 4 elements) are drawn behind them, and only then are the
// loads waited for (with their elements widened before, 8192 x 4096 bf16 with a
// residual took 48 us, not 32: 6.3 TB/s). Two groups a thread measured the
// same. Without a residual (29.9 us, floor 20) the generator's multiplies count as
// much as HBM: a call has 19 of 32 x 32 to 64 bits, which issue every fourth
// cycle, and the kernel draws 1.1e12 words a second of the 1.6e12 of a loop that
// does nothing else; multiplies and loads overlap in part.
constexpr int kDropThreads = 128;

template <typename T, bool DROP>
__global__ void __launch_bounds__(kDropThreads)
    dropout_add_kernel(const T* x, const T* residual, T* y, long long n, Drop drop) {
  constexpr int E = Vec<T>::kElems;
  const long long e = (static_cast<long long>(blockIdx.x) * kDropThreads + threadIdx.x) * E;
  if (e >= n) return;
  ptx::grid_dependency_wait();
  const bool whole = e + E <= n, add = residual != nullptr;
  Vec<T> vx, vr;
  if (whole) {
    vx = load_vec(x + e);
    if (add) vr = load_vec(residual + e);
  }
  uint32_t w[E / 4][4];
  if (DROP) {
    long long first[E / 4];
#pragma unroll
    for (int u = 0; u < E / 4; ++u) first[u] = e | (4 * u);
    keep_words<E / 4>(first, drop, w);
  }
  float v[E], r[E];
  if (whole) {
    unpack(vx, v);
    if (add) unpack(vr, r);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      v[i] = e + i < n ? to_f32(x[e + i]) : 0.f;
      r[i] = add && e + i < n ? to_f32(residual[e + i]) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (DROP) v[i] = w[i / 4][i % 4] >= drop.threshold ? v[i] : 0.f;
    if (add)
      v[i] = DROP ? fmaf(v[i], drop.inv_keep, r[i]) : v[i] + r[i];
    else if (DROP)
      v[i] *= drop.inv_keep;
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

// Second stage of the weight gradients: a block takes 32 columns, its 32
// warps every 32nd partial sum of each (kept in flight eight at a time), and
// adds the warps' sums in order. About 2 us at 4096 columns (152 partial sums
// each, 5 MB from L2), mostly the launch and the wait for the first stage; its
// launch overlaps that stage, which saves up to 0.5 us of it in a graph and 2 us
// between calls made back to back.
__global__ void __launch_bounds__(1024) weights_sum_kernel(BwdArgs a, int chunks) {
  __shared__ float part[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + tx;
  float v = 0.f;
  ptx::grid_dependency_wait();  // launched before the first stage has ended
  if (i < 2 * a.C) {
    const float* p = a.workspace + i;
    for (int k = ty; k < chunks; k += 256) {
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        x[u] = k + 32 * u < chunks ? p[2LL * (k + 32 * u) * a.C] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) v += x[u];
    }
  }
  part[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && i < 2 * a.C) {
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += part[k][tx];
    void* out = i < a.C ? a.dgamma : a.dbeta;
    if (out != nullptr) store_as(out, i < a.C ? i : i - a.C, a.wdtype, v);
  }
}

int check(long long rows, int C, int dtype, int wdtype) {
  if (rows < 0 || C <= 0 || !known_dtype(dtype) || !known_dtype(wdtype)) return ATTN_ERR_SHAPE;
  if (C > (1 << 29) || rows >= (1LL << 40) / C) return ATTN_ERR_TOO_LARGE;
  return ATTN_OK;
}

// Partial sums a column that a backward over this many rows may leave.
inline long long max_chunks(long long rows) {
  const long long n = (rows + 7) / 8 * 8;  // blocks come in eights
  return n < kMaxChunks ? (n > 0 ? n : 8) : kMaxChunks;
}

inline bool bad_p(float p) { return !(p >= 0.0f && p < 1.0f); }

int forward(const FwdArgs& a, int dtype, cudaStream_t stream) {
  if (a.rows == 0) return ATTN_OK;
  return with_dtype(dtype, [&](auto t) { return run_fwd<decltype(t)>(a, stream); });
}

int backward(const BwdArgs& a, int dtype, cudaStream_t stream) {
  const bool weights = a.dgamma != nullptr || a.dbeta != nullptr;
  int chunks = 0;
  if (a.rows > 0) {
    chunks = with_dtype(dtype, [&](auto t) { return run_bwd<decltype(t)>(a, stream); });
    if (chunks < 0) return chunks;
  }
  if (!weights || (a.rows > 0 && chunks == 0)) return ATTN_OK;
  return launch_overlapped(weights_sum_kernel, dim3(static_cast<unsigned>((2 * a.C + 31) / 32)),
                           1024, 0, 0, stream, a, chunks);
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
  return norm::forward(a, dtype, as_stream(stream));
}

extern "C" int attn_dropout_add(const void* x, const void* residual, void* y, long long n,
                                float p_drop, unsigned long long seed, int dtype, void* stream) {
  if (n > 0 && (!x || !y)) return ATTN_ERR_NULL;
  if (n < 0 || norm::bad_p(p_drop) || !known_dtype(dtype)) return ATTN_ERR_SHAPE;
  if (n >= (1LL << 40)) return ATTN_ERR_TOO_LARGE;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(y)) return ATTN_ERR_ALIGN;
  if (n == 0) return ATTN_OK;
  const norm::Drop drop = norm::make_drop(p_drop, seed);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const T *xt = static_cast<const T*>(x), *rt = static_cast<const T*>(residual);
    const long long per_block = static_cast<long long>(norm::kDropThreads) * Vec<T>::kElems;
    const unsigned grid = static_cast<unsigned>((n + per_block - 1) / per_block);
    return launch_overlapped(
        drop.on ? norm::dropout_add_kernel<T, true> : norm::dropout_add_kernel<T, false>,
        dim3(grid), norm::kDropThreads, 0, 0, as_stream(stream), xt, rt, static_cast<T*>(y), n,
        drop);
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
  return norm::forward(a, dtype, as_stream(stream));
}

extern "C" long long attn_layer_norm_bwd_workspace_bytes(long long rows, int C) {
  const int rc = norm::check(rows, C, ATTN_BF16, ATTN_BF16);
  if (rc != ATTN_OK) return rc;
  return norm::max_chunks(rows) * 2 * C *
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
  return norm::backward(a, dtype, as_stream(stream));
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
  return norm::backward(a, dtype, as_stream(stream));
}
