// Arguments and helpers shared by the layer-norm and dropout kernels
// (attn_norm.cu has the formulas).
#pragma once

#include <cstdint>

#include "element.cuh"

namespace attn {
namespace norm {

constexpr int kThreads = 256;
// Blocks of the backward, at most: the workspace holds two fp32 sums a
// column for each.
constexpr int kMaxChunks = 1024;
// Widest row of the kernels that keep a row on chip.
constexpr int kMaxRow = 16384;

struct Drop {
  // the generator's ten round keys: as kernel parameters they are operands of
  // the rounds' exclusive-ors and cost no instruction
  uint32_t key[10][2];
  uint32_t threshold;  // keep iff word >= threshold
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
  float* workspace;  // NULL: no weight gradients
  int finish;        // the grid is one cluster, which finishes the weight gradients itself
  long long rows;
  int C, wdtype;
  Drop drop;
};

// One of each per element type (attn_norm_bf16.cu, _fp16.cu, _fp32.cu);
// rows > 0. The backward returns the number of partial sums a column that it
// left in the workspace (0: none are wanted, or they are added up already), or a
// negative error.
template <typename T>
int run_fwd(const FwdArgs& a, cudaStream_t stream);
template <typename T>
int run_bwd(const BwdArgs& a, cudaStream_t stream);

// Keep words of the 4 NB elements from e on, e a multiple of 4: calls of
// consecutive counters, round by round, so that their multiplies interleave
// (philox.cuh has the generator's definition).
template <int NB>
__device__ __forceinline__ void keep_words(const long long (&e)[NB], const Drop& d,
                                           uint32_t (&w)[NB][4]) {
#pragma unroll
  for (int u = 0; u < NB; ++u) {
    w[u][0] = static_cast<uint32_t>(e[u] >> 2);
    w[u][1] = static_cast<uint32_t>(e[u] >> 34);
    w[u][2] = 0u;
    w[u][3] = 1u;
  }
#pragma unroll
  for (int r = 0; r < 10; ++r) {
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * w[u][0];
      const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * w[u][2];
      w[u][0] = static_cast<uint32_t>(p1 >> 32) ^ w[u][1] ^ d.key[r][0];
      w[u][1] = static_cast<uint32_t>(p1);
      w[u][2] = static_cast<uint32_t>(p0 >> 32) ^ w[u][3] ^ d.key[r][1];
      w[u][3] = static_cast<uint32_t>(p0);
    }
  }
}

__device__ __forceinline__ bool kept(long long e, const Drop& d) {
  const long long first[1] = {e & ~3LL};
  uint32_t w[1][4];
  keep_words<1>(first, d, w);
  const int i = static_cast<int>(e & 3);
  return (i == 0 ? w[0][0] : i == 1 ? w[0][1] : i == 2 ? w[0][2] : w[0][3]) >= d.threshold;
}

// Sets the dropped ones of the E elements from e (a multiple of 4) on to 0.
template <int E>
__device__ __forceinline__ void drop_vec(float (&f)[E], long long e, const Drop& d) {
  long long first[E / 4];
  uint32_t w[E / 4][4];
#pragma unroll
  for (int u = 0; u < E / 4; ++u) first[u] = e | (4 * u);  // e is a multiple of E
  keep_words<E / 4>(first, d, w);
#pragma unroll
  for (int i = 0; i < E; ++i) f[i] = w[i / 4][i % 4] >= d.threshold ? f[i] : 0.f;
}

}  // namespace norm
}  // namespace attn
