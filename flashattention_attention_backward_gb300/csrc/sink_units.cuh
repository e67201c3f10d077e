// How the backward with sinks shares its units of work out: plain C++, for the
// kernels, their launches and a test on the host.
//
// A unit is a key block of one key/value head. The first `with_sinks` units hold
// sinks and visit every query block from their own on, the others their band's.
#pragma once

#ifdef __CUDACC__
#define ATTN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define ATTN_HOST_DEVICE inline
#endif

namespace attn {

// The unit (past the last one: none) that CTA `cta` of `grid` takes in pass r. Without
// sinks, snake order (pass r visits CTAs 0..grid-1 when r is even, grid-1..0 when odd),
// which balances causal units, that shrink. With them, `heavy_passes` passes in which
// every CTA takes a unit with sinks, one in which the first `heavy` do, and those sit
// out the `ahead` passes that the others go on with, about as many units of a band as
// one with sinks is worth (causal GQA under a window of 1024 keys: 128 query tiles
// against 36; snake order alone gives those CTAs 200 to 236 tiles where the average is
// 131, and the step took 0.535 ms, not 0.394).
ATTN_HOST_DEVICE int snake_unit(int r, int cta, int grid) {
  return r * grid + ((r & 1) ? grid - 1 - cta : cta);
}
ATTN_HOST_DEVICE int sinks_unit(int r, int cta, int grid, int heavy_passes, int heavy,
                                int ahead) {
  if (r < heavy_passes) return snake_unit(r, cta, grid);
  r -= heavy_passes;
  const int first = heavy_passes * grid, light = grid - heavy;
  const int behind = first + heavy + ahead * light;
  if (heavy > 0 && cta < heavy) return r == 0 ? first + cta : behind + snake_unit(r - 1, cta, grid);
  return r < ahead ? first + heavy + r * light + cta - heavy
                   : behind + snake_unit(r - ahead, cta, grid);
}

}  // namespace attn
