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

// One call's units: how many hold sinks and how many do not, the query tiles of one of
// each (`most`, `band`), and those of the last unit with sinks, which has the fewest.
struct SinkUnits {
  long long with_sinks, others;
  long long most, band, least;
};

// A unit with sinks that outlasts what an SM has on average is shared by a cluster of
// CTAs, in a launch of its own that the other units' runs beside (1 x 8 heads over 1 x
// 16384 x 128, window 1024: the step takes 357 us, 528 with one launch behind the other,
// 2361 without clusters; 1 x 4 x 8192 x 64, window 512: 51, 67, 149). This returns how
// many CTAs, 1 for no such launch: those with the earliest end, in tiles, where a unit's
// start and epilogue are worth kTurn, clusters that do not run at once go in rounds, and
// the other units begin with the last round, on the SMs that it leaves or, if they need
// more, behind it. (1 x 32 heads over 8 x 16384, window 1024: 8 CTAs, 870 us; as many as
// bring the unit down to the average, 2, took 1134. 1 x 16 over 8 x 8192, window 512, 200
// sinks: 16 clusters of 4, 221 us; of 8, which run 15 at a time, 247.)
// at_once(n): clusters of n CTAs that run at once, 0 if none does.
template <typename AtOnce>
inline int sinks_cluster(const SinkUnits& u, int sms, AtOnce at_once) {
  constexpr long long kTurn = 4;
  const long long all = u.with_sinks * u.most + u.others * u.band;
  if (u.most * sms <= all * 5 / 4) return 1;
  const long long g = u.others < sms ? u.others : sms;
  const long long band = g > 0 ? (u.others + g - 1) / g * (u.band + kTurn) : 0;
  long long best = 0;
  int ctas = 1;
  for (int n = 2; n <= 8 && n <= u.least; n *= 2) {  // a tile for each CTA at least
    const long long fit = at_once(n);
    if (fit <= 0) break;
    const long long heavy = (u.most + n - 1) / n + kTurn;
    const long long before = (u.with_sinks - 1) / fit;  // rounds in front of the last
    const long long last = (u.with_sinks - before * fit) * n;
    const long long both = last + g <= sms ? (heavy > band ? heavy : band) : heavy + band;
    const long long end = before * heavy + both;
    if (ctas > 1 && end > best) continue;
    best = end;
    ctas = n;
  }
  return ctas;
}

// The same for launches of one CTA a unit, whose SMs take what comes next as they get
// free: as many CTAs as bring a unit with sinks down to the average, whatever goes in
// rounds (the step at d = 256, this rule and sinks_cluster: 2 x 8 heads over 1 x 4096,
// window 512, 4 sinks 237 us and 364; 1 x 4 over 1 x 16384, window 64, 1000 sinks 631 and
// 672, with 4 sequences and 200 sinks 826 and 862; 1 x 8 over 2 x 8192, window 1024 368
// and 350), of a size that can run.
template <typename AtOnce>
inline int sinks_cluster_waves(const SinkUnits& u, int sms, AtOnce at_once) {
  const long long all = u.with_sinks * u.most + u.others * u.band;
  int ctas = 1;
  while (ctas < 8 && u.most * sms > all * 5 / 4 * ctas && 2 * ctas <= u.least &&
         at_once(2 * ctas) > 0)
    ctas *= 2;
  return ctas;
}

}  // namespace attn
