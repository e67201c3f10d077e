// Arguments and helpers shared by the layer-norm and dropout kernels
// (attn_norm.cu has the formulas).
#pragma once

#include <cstdint>

#include "element.cuh"
#include "philox.cuh"

namespace attn {
namespace norm {

constexpr int kThreads = 256;
// Blocks of the backward, at most: the workspace holds two fp32 sums a
// column for each.
constexpr int kMaxChunks = 1024;
// Widest row of the kernels that keep a row on chip.
constexpr int kMaxRow = 16384;

struct Drop {
  uint32_t seed_lo, seed_hi, threshold;
  float inv_keep;
  int on;
};

struct FwdArgs {
  const void *x, *residual, *gamma, *beta;  // residual NULL: plain layer norm
  void *z, *y;
  float *mean, *rstd;
  long long rows;
  int C, wdtype;
  float eps;
  Drop drop;
};

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

// One of each per element type (attn_norm_bf16.cu, _fp16.cu, _fp32.cu);
// rows > 0. The backward returns the number of partial sums a column that it
// left in the workspace (0 without a workspace), or a negative error.
template <typename T>
int run_fwd(const FwdArgs& a, cudaStream_t stream);
template <typename T>
int run_bwd(const BwdArgs& a, cudaStream_t stream);

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

}  // namespace norm
}  // namespace attn
