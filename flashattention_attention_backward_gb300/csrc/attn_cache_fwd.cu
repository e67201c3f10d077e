// attn_cache_fwd: attention of a ragged batch's new tokens over a paged
// key/value cache, on the tcgen05 tensor cores.
//
// Row t of the batch, at position p of its sequence, and query head h see the keys
// j <= p (or all of the sequence's) with j >= p - left or j < sinks:
//   x_j = logit of q and key j (log2 units),  O = sum_j 2^(x_j - m) v_j / l,
//   l = sum_j 2^(x_j - m),  LSE = (m + log2 l) ln 2
// with a running shift m, the row's maximum (less 9 with fp16, see kHead), and sum l,
// as in attn_fwd: S = Q K^T in fp32 tensor memory, P as 16-bit pairs over it, O
// accumulated in tensor memory and rescaled only when a row's maximum outgrows it (by
// more than 2^8, with fp16 2^6).
//
// Tiles. The G = H / H_kv heads that share a key/value head sit in one tile with
// the tokens: row r of a tile is token r / G and head r mod G, floor(128 / G)
// tokens a tile, so that a decoding step reads each key and value once for all
// of its heads, and a chunk of a prompt fills the 128 rows. The matrix products
// of a tile whose rows are mostly empty cost as much as a full one's, about 0.55
// us per 128 keys and SM at d = 128 against the 1.5 us that an SM's share of the
// memory bandwidth takes to bring those keys and values in; the softmax warps
// without a row do nothing.
//
// Keys come in blocks of 128 positions, gathered by the page table: one TMA box
// of gcd(page size, 128) slots by 64 columns for each piece of a page. A block
// whose end the sequence, or whose start the window, cuts off loads the pieces it
// needs; rows of V that no row of the tile sees are set to zero behind the copy (P
// is zero there, but 0 times what an unused slot holds may be NaN).
//
// Work. All (tile, block) pairs of the batch in the order sequence, key/value
// head, tile, block are one line, cut into equal parts, one a CTA (one CTA an
// SM): lengths differ from sequence to sequence and are known on the device only,
// and a single long sequence still occupies every SM. A tile that two or more
// CTAs share leaves its partial O, m and l in the workspace, and a second, small
// kernel joins them in the order of the blocks: the same bits every time. Each
// CTA finds its part of the line itself, from two sums over the sequences.
//   warp 0      Q of each tile; K in a ring of 4, 2 or 1 stages (d = 64, 128, 256)
//   warp 2      V in the same kind of ring
//   warp 3      zeroes rows of V
//   warp 1      MMA issuer: per tile S(0), then per block S(j + 1), P(j) V
//   warps 4-11  softmax: warpgroup h takes keys 64 h .. 64 h + 63 of each block
//               and columns h d/2 .. of O; then the tile's epilogue
// Every mbarrier wait is bounded, as in attn_fwd.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "cache_common.cuh"
#include "element.cuh"
#include "grid_ptx.cuh"
#include "sm103_ptx.cuh"
#include "softcap_math.cuh"

namespace attn {
namespace cachefwd {

using namespace ptx;
using cache::Batch;

constexpr int kBm = 128;  // rows of a tile (tensor-memory lanes)
constexpr int kBn = 128;  // keys per block
constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
// What a tile costs besides its blocks, in blocks: about 2 us, against 0.9 us a block.
// A prompt of 4096 tokens (32 heads over 8, d = 128, 1024 tiles of 1 to 32 blocks)
// takes 137 us so, 159 with one and 189 with none; 256 requests of up to 300 keys 72,
// 79 and 78.
constexpr int kTileUnits = 2;
constexpr int kMaxCtas = 192;  // parts of the line at most (the workspace's size)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's shift is its maximum less kHead, moved only when that outgrows it by more
// than kRescale (log2 units), so that weights stay below 2^(kHead + kRescale) and the
// largest is 2^kHead or more. bf16 has fp32's exponents. An fp16 operand has eleven
// bits down to 2^-14 only and is 0 below 2^-25: with the shift at the maximum, keys
// that weigh 2^-23 of one large key each lost a seventh of what they weigh together,
// and at 2^-25 all of it, while l kept it. Weights up to 2^15 instead (fp16 ends at
// 2^16) have eleven bits down to 2^-23 of the row's largest, and below an error of 2^-34
// of it. A ragged batch under a window and a softcap takes 70.4 us in fp16 so and 69.9
// in bf16; with 11 and 4 71.9, with 7 and 8 70.3.
template <typename T>
constexpr float kHead = std::is_same<T, __half>::value ? 9.f : 0.f;
template <typename T>
constexpr float kRescale = std::is_same<T, __half>::value ? 6.f : 8.f;
constexpr long long kWaitLimitCycles = 2000000000LL;  // about one second

// The softmax warps' state does not fit in the 168 registers that 384 threads are
// launched with: setmaxnreg moves registers to them from the other four warps.
template <int D>
constexpr int kRegsSoftmax = D == 256 ? 200 : 216;
template <int D>
constexpr int kRegsCtl = D == 256 ? 96 : 72;
static_assert(256 * kRegsSoftmax<256> + 128 * kRegsCtl<256> <= 384 * 168, "register pool");
static_assert(256 * kRegsSoftmax<128> + 128 * kRegsCtl<128> <= 384 * 168, "register pool");

template <int D>
struct Layout {
  static constexpr int kTileBytes = 128 * D * 2;
  // K and V stages: an SM's share of the memory bandwidth wants some 100 KB in flight
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? 2 : 1;
  static constexpr int kQStages = D <= 128 ? 2 : 1;
  static constexpr int kOBufs = D <= 128 ? 2 : 1;  // O accumulators in tensor memory
  // rows of a narrow tile: the 4 copies' O in fp32 fill the warps' stages
  static constexpr int kNarrow = D <= 128 ? 1024 / D : 0;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kQStages * kTileBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  // 2 KB for each softmax warp: rows of O on their way to coalesced stores
  static constexpr int kStage = kV + kStages * kTileBytes;
  // the softmax warpgroups' half-row maxima (two blocks in flight), the row sums
  // of a finished tile: [2][2][128] + [2][128] fp32
  static constexpr int kXchg = kStage + 8 * 2048;
  static constexpr int kBars = kXchg + 6 * 128 * 4;
  static constexpr int kNumBars = 35;
  static constexpr int kSums = kBars + kNumBars * 8;   // [kWarps] long long
  static constexpr int kPart = kSums + kWarps * 8;     // Part
  static constexpr int kTmemSlot = kPart + 48;
  static constexpr int kAbort = kTmemSlot + 4;
  // narrow tiles (d <= 128): the quadrants' shifts, [128] fp32
  static constexpr int kShifts = kAbort + 12;
  static constexpr int kUsed = kShifts + (D <= 128 ? 512 : 0);
  // more than half of the SM's shared memory, so that a second CTA never waits
  // on the first one's tensor memory
  static constexpr int kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
};
static_assert(Layout<128>::kBytes <= 232448, "shared memory budget");
static_assert(Layout<256>::kBytes <= 232448, "shared memory budget");

enum Bar {
  BAR_Q_FULL = 0,    // + Q stage
  BAR_Q_EMPTY = 2,   // + Q stage: the tile's last S GEMM has read it
  BAR_K_FULL = 4,    // + stage
  BAR_V_FULL = 8,    // + stage
  BAR_V_EDGE = 12,   // + stage: copies of a V block some of whose rows are then zeroed
  BAR_S_DONE = 16,   // + block parity: S of the block written, its K read
  BAR_P_FULL = 18,   // + block parity: P of the block written (and O rescaled if needed)
  BAR_O_DONE = 20,   // + block parity: P V of the block completed, its V read
  BAR_O_LAST = 22,   // + O buffer: the tile's last P V completed
  BAR_O_FREE = 24,   // + O buffer: the tile's epilogue has read O
  BAR_K_EMPTY = 26,  // + stage, where there are more than two: its K read
  BAR_V_EMPTY = 30,  // + stage, where there are more than two: its V read
  BAR_DRAIN = 34,    // abort path only: completion of everything issued
};

__device__ int g_status;

// What a part leaves for the joining kernel if its last tile goes on in the parts
// behind it: how many parts share the tile (0: none), and the tile.
struct Shared {
  int parts, row0, kvh, rows;
};
// The workspace: Shared[kMaxCtas]; then per part two slots (0: of a tile that
// began in a part before, 1: of one that begins here) of m [128], l [128] and O
// [128][d], fp32.
constexpr long long kSharedBytes = kMaxCtas * static_cast<long long>(sizeof(Shared));
__host__ __device__ constexpr long long slot_floats(int d) { return 256 + 128LL * d; }

struct Params {
  Batch batch;
  void* o;
  float* lse;
  long long o_token, o_head;
  char* workspace;
  int H, H_kv, G, tokens;  // tokens of a full tile: 128 / G
  int narrow;              // rows of a narrow tile's copy of the queries, 0: none narrow
  int box;                 // slots of one TMA box: gcd(page_size, 128)
  int cap;                 // positions that the page table holds
  int whole;               // parts end at tiles' ends: no tile is shared, nothing to join
  float scale, softcap;
  int causal, left, sinks;  // left < 0: no bound
};

struct Ctx {
  uint32_t bars;
  volatile int* abort;
};

__device__ __forceinline__ uint32_t bar_addr(const Ctx& c, int i) { return c.bars + 8u * i; }
__device__ __noinline__ void record_status(int code) { atomicCAS(&g_status, 0, code); }

__device__ __forceinline__ bool wait(const Ctx& c, int bar, uint32_t parity) {
  const uint32_t a = bar_addr(c, bar);
  if (mbar_try_wait(a, parity)) return true;
  const long long t0 = clock64();
  uint32_t n = 0;
  while (!mbar_try_wait(a, parity)) {
    if ((++n & 63u) == 0) {
      if (*c.abort) return false;
      if (clock64() - t0 > kWaitLimitCycles) {
        *c.abort = 1;
        record_status(ATTN_ERR_DEVICE_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_warp(const Ctx& c, int bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(c, bar, parity));
}
__device__ __forceinline__ void wait_drain(const Ctx& c, int bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar_addr(c, bar), parity)) {
    if (clock64() - t0 > kWaitLimitCycles) return;
  }
}

// ------------------------------------------------------------------ the line of work
struct Seq {
  int row0, n;    // its rows of the batch
  int length;     // positions that the page table holds of it
  int pos0;       // position of row row0 (negative: more new tokens than positions)
  int tiles;
};
__device__ __forceinline__ Seq seq_of(const Params& p, int b) {
  const Batch& c = p.batch;
  Seq s;
  s.row0 = min(max(c.starts[b], 0), c.T);
  s.n = min(max(c.starts[b + 1], s.row0), c.T) - s.row0;
  const int length = max(c.lengths[b], 0);
  s.length = min(length, p.cap);
  s.pos0 = length - s.n;
  s.tiles = (s.n + p.tokens - 1) / p.tokens;
  return s;
}

// The keys that any row of a tile sees: j <= hi and (j >= lo or j < sinks), and
// its nt key blocks, the first ns of the sequence (sinks before the band), then j0,
// j0 + 1, ... A tile that sees nothing has one block, all hidden.
struct Tile {
  int pos0, count;  // position of its first token, its tokens
  int lo, hi, sinks;
  int j0, ns, nt;
  __device__ __forceinline__ int units() const { return nt + kTileUnits; }
  __device__ __forceinline__ int block(int t) const { return t < ns ? t : j0 + t - ns; }
};
__device__ __forceinline__ Tile tile_of(const Params& p, const Seq& s, int tile) {
  Tile t;
  t.pos0 = s.pos0 + tile * p.tokens;
  t.count = min(p.tokens, s.n - tile * p.tokens);
  const int last = t.pos0 + t.count - 1;
  t.hi = p.causal ? min(last, s.length - 1) : s.length - 1;
  t.lo = p.left < 0 ? 0 : max(0, t.pos0 - p.left);
  t.sinks = max(0, min(p.sinks, t.hi + 1));
  if (t.sinks >= t.lo) t.lo = 0;
  t.j0 = t.lo / kBn;
  const int sink_blocks = (t.sinks + kBn - 1) / kBn;
  if (t.lo <= t.hi) {
    t.ns = min(t.j0, sink_blocks);
    t.nt = t.ns + t.hi / kBn - t.j0 + 1;
  } else {  // no band: only sinks, if any
    t.ns = sink_blocks;
    t.nt = max(1, sink_blocks);
    t.j0 = 0;
    t.lo = 1 << 30;  // above every key
  }
  return t;
}

// A narrow tile (with a softcap; at most 8 rows at d = 128, 16 at d = 64) has four
// copies of its queries, in rows 0, 32, 64 and 96 of the tile, and the warps of each
// quadrant of tensor memory take a quarter of every block's keys. With its rows in
// one quadrant the softmax of a block is two warps' work, the others idle: with the
// softcap's tanh that takes longer than the block's loads (64 requests of up to 8192
// keys, 32 heads over 8, d = 128: 253 us, 183 narrow). Without a softcap the loads
// take longer either way (183 and 182 us), and short sequences pay for the joining
// of the copies (256 requests of up to 300 keys 71 us, 74 narrow).
template <int D, bool SOFTCAP>
constexpr bool kHasNarrow = SOFTCAP && D <= 128;
template <int D, bool SOFTCAP>
__device__ __forceinline__ bool is_narrow(const Params& p, const Tile& t) {
  return kHasNarrow<D, SOFTCAP> && t.count * p.G <= p.narrow;
}

// The line is measured in units: a block is one, and a tile has kTileUnits in
// front of its first (its queries, its epilogue). Units of one key/value head's
// tiles of a sequence, summed by a whole warp:
__device__ __forceinline__ long long head_units(const Params& p, const Seq& s) {
  const int lane = threadIdx.x & 31;
  long long sum = 0;
  for (int i = lane; i < s.tiles; i += 32) sum += tile_of(p, s, i).units();
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  return sum;
}

// The same for sequence b0 + lane (0 past the end), a whole warp together:
// sequences of one tile in parallel, longer ones one by one.
__device__ __forceinline__ long long lane_units(const Params& p, int b0, int end) {
  const int lane = threadIdx.x & 31;
  Seq s{};
  if (b0 + lane < end) s = seq_of(p, b0 + lane);
  long long units = s.tiles == 1 ? tile_of(p, s, 0).units() : 0;
  uint32_t more = __ballot_sync(0xffffffffu, s.tiles > 1);
  while (more != 0) {
    const int src = __ffs(more) - 1;
    more &= more - 1;
    Seq o;
    o.row0 = __shfl_sync(0xffffffffu, s.row0, src);
    o.n = __shfl_sync(0xffffffffu, s.n, src);
    o.length = __shfl_sync(0xffffffffu, s.length, src);
    o.pos0 = __shfl_sync(0xffffffffu, s.pos0, src);
    o.tiles = __shfl_sync(0xffffffffu, s.tiles, src);
    const long long sum = head_units(p, o);
    if (lane == src) units = sum;
  }
  return units;
}

// A CTA's part of the line: the tile and the unit of it where it begins, how many
// units it has, how many a full part has, and the units before it.
struct Part {
  int b, kvh, tile, at;
  long long count, share, first;
};

// Finds the CTA's part (every thread of the CTA calls; `sums` and `part` in
// shared memory). Warp w sums the units of its chunk of the sequences, 32 at a
// time; the warp whose chunk holds the part's first unit then looks for it there
// (a chunk of up to 32 sequences, so up to 384 in all, is not summed again).
__device__ __forceinline__ void find_part(const Params& p, long long* sums, Part* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int B = p.batch.B;
  const int chunk = (B + kWarps - 1) / kWarps;
  const int first = min(B, warp * chunk), end = min(B, first + chunk);
  long long sum = 0, mine = 0;
  for (int b = first; b < end; b += 32) sum += mine = lane_units(p, b, end);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) sums[warp] = sum * p.H_kv;
  if (threadIdx.x == 0) part->count = 0;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  const long long share = (total + gridDim.x - 1) / gridDim.x;
  const long long u0 = blockIdx.x * share;
  if (u0 < total && u0 >= before && u0 < before + sums[warp]) {
    long long at = u0 - before;  // within this warp's chunk
    for (int b = first; b < end; b += 32) {
      const long long units = (chunk <= 32 ? mine : lane_units(p, b, end)) * p.H_kv;
      long long upto = units;  // inclusive sum over the lanes
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, upto > at);
      if (past == 0) {
        at -= __shfl_sync(0xffffffffu, upto, 31);
        continue;
      }
      const int src = __ffs(past) - 1;
      const long long per_head = __shfl_sync(0xffffffffu, units, src) / p.H_kv;
      at -= __shfl_sync(0xffffffffu, upto - units, src);
      const int kvh = static_cast<int>(at / per_head);
      at -= kvh * per_head;
      const Seq s = seq_of(p, b + src);
      for (int i = 0; i < s.tiles; i += 32) {
        const int here = i + lane < s.tiles ? tile_of(p, s, i + lane).units() : 0;
        int sum_to = here;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, sum_to, off);
          if (lane >= off) sum_to += v;
        }
        const uint32_t in = __ballot_sync(0xffffffffu, sum_to > at);
        if (in == 0) {
          at -= __shfl_sync(0xffffffffu, sum_to, 31);
          continue;
        }
        const int t = __ffs(in) - 1;
        at -= __shfl_sync(0xffffffffu, sum_to - here, t);
        if (lane == 0) {
          part->b = b + src;
          part->kvh = kvh;
          part->tile = i + t;
          part->at = static_cast<int>(at);
          part->share = share;
          part->first = u0;
          part->count = min(share, total - u0);
        }
        break;
      }
      break;
    }
  }
  __syncthreads();
}

// Walks the tiles of a part; every role has its own and one call of step(), whose
// code is long and inlined.
struct Walk {
  int b, kvh, next, at, left;  // what comes: a tile, from which unit of it on; units left
  int tile, blk, take;         // the tile's blocks blk .. blk + take - 1 are the part's
  Seq s;
  Tile t;
  __device__ __forceinline__ Walk(const Params& p, const Part& part)
      : b(part.b), kvh(part.kvh), next(part.tile), at(part.at),
        left(static_cast<int>(part.count)) {
    if (left > 0) s = seq_of(p, b);
  }
  // The next tile; false behind the last. A part that ends in the units before a
  // tile's first block leaves the tile to the next one.
  __device__ __forceinline__ bool step(const Params& p) {
    bool skip;
    do {
      if (left <= 0) return false;
      if (next == s.tiles) {
        next = 0;
        if (++kvh == p.H_kv) {
          kvh = 0;
          do {  // left > 0: a sequence with tiles follows
            s = seq_of(p, ++b);
          } while (s.tiles == 0 && b + 1 < p.batch.B);
        }
      }
      tile = next++;
      t = tile_of(p, s, tile);
      blk = max(0, at - kTileUnits);
      take = max(0, (p.whole ? t.nt : min(t.nt, at + left - kTileUnits)) - blk);
      left -= t.units() - at;  // below 0: the tile goes on in the next part
      skip = p.whole && at > 0;  // a whole tile belongs to the part that holds its first unit
      at = 0;
    } while (skip);
    return take > 0;
  }
};

// ------------------------------------------------------------------ loaders
// The pieces of a key block that a tile needs: lane i < 128 / box holds the page
// (or -1) and the slot of the box of keys n0 + i box.
struct Pieces {
  int page, slot;
  uint32_t needed;  // a bit per lane
};
__device__ __forceinline__ Pieces pieces_of(const Params& p, const Walk& w, int blk) {
  const int lane = threadIdx.x & 31;
  const int key = w.t.block(blk) * kBn + lane * p.box;
  const bool need = lane * p.box < kBn &&
                    ((key <= w.t.hi && key + p.box > w.t.lo) || key < w.t.sinks);
  Pieces x;
  x.needed = __ballot_sync(0xffffffffu, need);
  x.page = x.slot = 0;
  if (need) {
    const uint32_t k = static_cast<uint32_t>(key), n = static_cast<uint32_t>(p.batch.page_size);
    x.page = p.batch.pages[static_cast<long long>(w.b) * p.batch.max_pages + k / n];
    x.slot = static_cast<int>(k % n);
  }
  return x;
}

// Loads the needed pieces of one block into the stage at dst, completing on bar.
template <int D>
__device__ __forceinline__ void load_pieces(const Ctx& c, const Params& p, const Pieces& x,
                                            int kvh, uint32_t dst, const CUtensorMap* map,
                                            int bar) {
  const int lane = threadIdx.x & 31;
  if (lane == 0)
    mbar_arrive_expect_tx(bar_addr(c, bar), __popc(x.needed) * p.box * (D * 2));
  __syncwarp();
  if ((x.needed >> lane) & 1u) {
    int page = x.page;
    if (page < 0 || page >= p.batch.n_pages) {
      page = p.batch.n_pages;  // outside the tensor: filled with zeros
      record_status(ATTN_ERR_PAGE);
    }
#pragma unroll
    for (int cb = 0; cb < D / 64; ++cb)
      tma_load_4d(dst + cb * 16384 + lane * p.box * 128, map, bar_addr(c, bar), 64 * cb, kvh,
                  x.slot, page);
  }
  __syncwarp();
}

// Waits until stage g mod kS of K or of V has been read by block g - kS. With two
// stages or one the barriers of the products serve: no block of that parity behind
// g - kS can have completed, so that the phase is that block's.
template <int D, bool IS_V>
__device__ __forceinline__ bool wait_stage(const Ctx& c, int g) {
  constexpr int kS = Layout<D>::kStages;
  const int before = g - kS;
  if (before < 0) return true;
  if (kS > 2)
    return wait_warp(c, (IS_V ? BAR_V_EMPTY : BAR_K_EMPTY) + g % kS, (before / kS) & 1);
  return wait_warp(c, (IS_V ? BAR_O_DONE : BAR_S_DONE) + (before & 1), (before >> 1) & 1);
}

// Whether a block of a tile has keys that no row of the tile sees.
__device__ __forceinline__ bool is_cut(const Tile& t, int n0) {
  return n0 + kBn - 1 > t.hi || (n0 < t.lo && n0 + kBn > t.sinks);
}

// Warp 0: Q of each tile and its K blocks; warp 2: the V blocks. Each ring waits
// for its own stages, in the order the tensor cores finish them.
template <int D, bool SOFTCAP, bool IS_V>
__device__ void loader_role(const Ctx& c, const Params& p, const Part& part, uint32_t sbase,
                            const CUtensorMap* tq, const CUtensorMap* tqn,
                            const CUtensorMap* tkv) {
  using L = Layout<D>;
  constexpr int kS = L::kStages, kQS = L::kQStages;
  const int lane = threadIdx.x & 31;
  const int bar_full = IS_V ? BAR_V_FULL : BAR_K_FULL;
  const int ring = IS_V ? L::kV : L::kK;
  int g = 0, i = 0;  // blocks and tiles issued
  bool ok = true;
  Walk w(p, part);
  for (; ok && w.step(p); ++i) {
    if (!IS_V) {
      const int qs = i % kQS;
      if (i >= kQS && !(ok = wait_warp(c, BAR_Q_EMPTY + qs, ((i / kQS) - 1) & 1))) break;
      if (lane == 0) {
        if (p.batch.lengths[w.b] > p.cap) record_status(ATTN_ERR_PAGE);
        const bool narrow = is_narrow<D, SOFTCAP>(p, w.t);
        const int rows = narrow ? 4 * p.narrow : p.tokens * p.G;
        mbar_arrive_expect_tx(bar_addr(c, BAR_Q_FULL + qs), rows * (D * 2));
        for (int copy = 0; copy < (narrow ? 4 : 1); ++copy)
          for (int cb = 0; cb < D / 64; ++cb)
            tma_load_4d(sbase + L::kQ + qs * L::kTileBytes + cb * 16384 + copy * 4096,
                        narrow ? tqn : tq, bar_addr(c, BAR_Q_FULL + qs), 64 * cb, 0, w.kvh,
                        w.s.row0 + w.tile * p.tokens);
      }
      __syncwarp();
    }
    // the page numbers of the next block are on their way while this one waits
    // for its stage
    Pieces next = pieces_of(p, w, w.blk);
    for (int t = 0; t < w.take; ++t, ++g) {
      const Pieces x = next;
      if (t + 1 < w.take) next = pieces_of(p, w, w.blk + t + 1);
      if (!(ok = wait_stage<D, IS_V>(c, g))) break;
      const int st = g % kS;
      const bool cut = IS_V && is_cut(w.t, w.t.block(w.blk + t) * kBn);
      // what zero_role finishes completes on a barrier of its own, if at all
      if (!cut || x.needed != 0)
        load_pieces<D>(c, p, x, w.kvh, sbase + ring + st * L::kTileBytes, tkv,
                       cut ? BAR_V_EDGE + st : bar_full + st);
    }
  }
  // When aborting, the copies in flight must land before the CTA exits (a phase
  // that was never begun ends the wait by its limit).
  if (!ok || *c.abort) {
    for (int st = 0; st < kS; ++st)
      wait_drain(c, bar_full + st, ((g + kS - st) / kS - 1) & 1);
    if (!IS_V)
      for (int st = 0; st < kQS; ++st) wait_drain(c, BAR_Q_FULL + st, (i / kQS) & 1);
  }
}

// Warp 3: sets the rows of V that no row of the tile sees to zero, in the blocks
// that have such rows, once their copies have landed, and hands the stage on.
template <int D>
__device__ void zero_role(const Ctx& c, const Params& p, const Part& part, uint8_t* smem) {
  using L = Layout<D>;
  constexpr int kS = L::kStages;
  const int lane = threadIdx.x & 31;
  uint32_t parity = 0;  // bit st: that of the stage's next copies
  int g = 0;
  bool ok = true;
  Walk w(p, part);
  while (ok && w.step(p)) {
    for (int t = 0; t < w.take; ++t, ++g) {
      const int n0 = w.t.block(w.blk + t) * kBn, st = g % kS;
      if (!is_cut(w.t, n0)) continue;
      const int key = n0 + 4 * lane;  // any of the block's keys visible: it has copies
      const bool seen = (key <= w.t.hi && key + 3 >= w.t.lo) || key < w.t.sinks;
      if (__any_sync(0xffffffffu, seen)) {
        if (!(ok = wait_warp(c, BAR_V_EDGE + st, (parity >> st) & 1))) break;
        parity ^= 1u << st;
      } else if (!(ok = wait_stage<D, true>(c, g))) {
        break;
      }
      for (int r = lane >> 3; r < kBn; r += 4) {  // 8 lanes a row
        const int k = n0 + r;
        if (k <= w.t.hi && (k >= w.t.lo || k < w.t.sinks)) continue;
#pragma unroll
        for (int cb = 0; cb < D / 64; ++cb)
          *reinterpret_cast<uint4*>(smem + L::kV + st * L::kTileBytes + cb * 16384 + r * 128 +
                                    (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_addr(c, BAR_V_FULL + st));
    }
  }
  if (!ok || *c.abort)
    for (int st = 0; st < kS; ++st) wait_drain(c, BAR_V_EDGE + st, (parity >> st) & 1);
}

// ------------------------------------------------------------------ MMA issuer
// fp16 operands have format 0 where make_idesc_bf16 sets 1 (bits 7 and 10).
template <typename T>
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn_major) {
  return make_idesc_bf16(M, N, false, b_mn_major) &
         ~(std::is_same<T, __half>::value ? (1u << 7) | (1u << 10) : 0u);
}

// S runs one block ahead of P V: S(g + 1) goes into the other S buffer (its P(g -
// 1) was read by P(g - 1) V, issued before), also where block g + 1 begins the next
// tile and two Q stages hold both tiles' queries, so that the softmax finds its
// scores behind the epilogue; then P(g) V into the tile's O buffer once the
// softmax has written P(g). One thread does all of it: few MMAs can be queued, so
// what it spends between the last MMA of one product and the first of the next is
// time of the tensor cores (with the whole warp in the loop, votes behind every
// wait and a commit for each of the loaders, a chunk of 2048 tokens over 18432 keys
// took 468 us, 419 so).
template <typename T, int D>
__device__ __forceinline__ void issue_mmas(const Ctx& c, const Params& p, const Part& part,
                                           uint32_t sbase, uint32_t tmem) {
  using L = Layout<D>;
  constexpr int kS = L::kStages, kQS = L::kQStages, kOB = L::kOBufs;
  constexpr uint32_t kIdS = idesc<T>(kBm, kBn, false);  // S = Q K^T
  constexpr uint32_t kIdO = idesc<T>(kBm, D, true);     // O += P V
  auto kmaj = [](int k) { return static_cast<uint32_t>(((k >> 2) * 16384 + (k & 3) * 32) >> 4); };
  auto mnmaj = [](int k) { return static_cast<uint32_t>((2048 * k) >> 4); };
  const uint32_t q_0 = sdesc_lo(sbase + L::kQ, 16), k_0 = sdesc_lo(sbase + L::kK, 16);
  const uint32_t v_0 = sdesc_lo(sbase + L::kV, 16384);
  constexpr uint32_t kStep = L::kTileBytes >> 4;  // from one stage's descriptor to the next
  // S of block g of tile i; `first`, `last` of the tile's blocks
  auto issue_s = [&](int g, int i, bool first, bool last) -> bool {
    const int st = g % kS, qs = i % kQS;
    if (first && !wait(c, BAR_Q_FULL + qs, (i / kQS) & 1)) return false;
    if (!wait(c, BAR_K_FULL + st, (g / kS) & 1)) return false;
    const uint32_t q_lo = q_0 + qs * kStep, k_lo = k_0 + st * kStep, s_to = tmem + (g & 1) * 128;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      mma_ss(s_to, sdesc_from_lo(q_lo + kmaj(k)), sdesc_from_lo(k_lo + kmaj(k)), kIdS, k > 0);
    mma_commit(bar_addr(c, BAR_S_DONE + (g & 1)));
    if (kS > 2) mma_commit(bar_addr(c, BAR_K_EMPTY + st));
    if (last) mma_commit(bar_addr(c, BAR_Q_EMPTY + qs));
    return true;
  };
  bool ok = true;
  Walk w(p, part);
  // block g, number t of the nt of tile i, is the next P V; none yet at -1
  int g = -1, i = -1, t = 0, nt = 0;
  for (;;) {
    const bool last = t + 1 >= nt;
    const bool more = last ? w.step(p) : true;
    const int next_nt = w.take;
    const bool ahead = kQS >= 2 || !last || g < 0;
    if (more && ahead &&
        !(ok = issue_s(g + 1, last ? i + 1 : i, last, last ? next_nt == 1 : t + 2 == nt)))
      break;
    if (g >= 0) {
      const int vs = g % kS, ob = i % kOB;
      const uint32_t v_lo = v_0 + vs * kStep, p_at = tmem + (g & 1) * 128;
      const uint32_t o_to = tmem + 256 + ob * D;
      if (!(ok = wait(c, BAR_V_FULL + vs, (g / kS) & 1))) break;
      if (t == 0 && i >= kOB && !(ok = wait(c, BAR_O_FREE + ob, ((i / kOB) - 1) & 1))) break;
      if (!(ok = wait(c, BAR_P_FULL + (g & 1), (g >> 1) & 1))) break;
      tc_fence_after();
      // A = P (pairs in the S buffer of block g: keys 0-63 in columns 0-31,
      // keys 64-127 in columns 64-95, one half per softmax warpgroup)
#pragma unroll
      for (int k = 0; k < kBn / 16; ++k)
        mma_ts(o_to, p_at + 8 * k + (k >= 4 ? 32 : 0), sdesc_from_lo(v_lo + mnmaj(k)), kIdO,
               (t > 0 || k > 0) ? 1u : 0u);
      mma_commit(bar_addr(c, BAR_O_DONE + (g & 1)));
      if (kS > 2) mma_commit(bar_addr(c, BAR_V_EMPTY + vs));
      if (last) mma_commit(bar_addr(c, BAR_O_LAST + ob));
    }
    if (!more) break;
    if (!ahead && !(ok = issue_s(g + 1, i + 1, true, next_nt == 1))) break;
    if (last) {
      nt = next_nt;
      t = 0;
      ++i;
    } else {
      ++t;
    }
    ++g;
  }
  if (!ok || *c.abort != 0) {
    // completion of everything issued before tensor memory is released
    mma_commit(bar_addr(c, BAR_DRAIN));
    wait_drain(c, BAR_DRAIN, 0);
  }
}

// ------------------------------------------------------------------ softmax
template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack_pair<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Bit e of word e / 32 set where key key0 + e (e < 64) is visible to a row that
// sees keys up to hi from lo on, and the first `sinks`.
__device__ __forceinline__ uint2 visible_bits(int key0, int lo, int hi, int sinks) {
  auto below = [](int n) {  // bits 0 .. n - 1
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
  };
  const unsigned long long v = below(hi - key0 + 1) & (~below(lo - key0) | below(sinks - key0));
  return make_uint2(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32));
}
__device__ __forceinline__ bool bit_of(uint2 bits, int e) {
  return ((e < 32 ? bits.x : bits.y) >> (e & 31)) & 1u;
}

// Factors on a raw score s: its logit without a softcap (tau log2e); with one, u =
// tau s / c, 2 u log2e, and what tanh(u) is multiplied by (c log2e).
struct Factors {
  float plain, u, in, out;
};

// The capped logit c tanh(u), log2 units, less the shift, of two scores, by one of
// three forms of tanh. Up to 1/4 its Taylor sum to u^7, multiplied into the logit at
// once: the first term left out is 62/2835 u^9, 8.4e-8 or less, the polynomial's error;
// both shrink with u, so that a logit far below the cap is off by 2^-20 of itself. The
// form through exp2 is off by 1e-7 of the cap: it serves warps that have a score beyond
// 1, whose logit is three quarters of the cap or more.
enum { kTanhMufu = 0, kTanhPoly = 1, kTanhTaylor = 2 };
constexpr float kTaylorMax = 0.25f;
template <int FORM>
__device__ __forceinline__ uint64_t cap_pair(const Factors& f, uint64_t s2, uint64_t nsh2) {
  if (FORM == kTanhTaylor) {
    const uint64_t u2 = f2_mul(s2, f2_make(f.u, f.u)), x2 = f2_mul(u2, u2);
    uint64_t w2 = f2_fma(x2, f2_make(-5.3968254e-2f, -5.3968254e-2f),
                         f2_make(1.3333333e-1f, 1.3333333e-1f));
    w2 = f2_fma(w2, x2, f2_make(-3.3333333e-1f, -3.3333333e-1f));
    w2 = f2_fma(w2, x2, f2_make(1.f, 1.f));
    return f2_fma(f2_mul(s2, f2_make(f.plain, f.plain)), w2, nsh2);
  }
  const uint64_t th2 = FORM == kTanhPoly ? softcap::tanh_poly2(f2_mul(s2, f2_make(f.u, f.u)))
                                         : softcap::tanh_mufu2(f2_mul(s2, f2_make(f.in, f.in)));
  return f2_fma(th2, f2_make(f.out, f.out), nsh2);
}
// Calls body with the form that serves every score of the warp, `most` the lane's
// largest in size. A lane whose row is none of the tile's (`mine` false: another
// sequence's query, or one of no sequence) has no say, so that what it holds changes no
// bit of the others.
template <typename F>
__device__ __forceinline__ void with_form(const Factors& f, float most, bool mine, F body) {
  most *= f.u;
  if (!__any_sync(0xffffffffu, mine && most > kTaylorMax))
    body(std::integral_constant<int, kTanhTaylor>{});
  else if (!__any_sync(0xffffffffu, mine && most > softcap::kPolyMax))
    body(std::integral_constant<int, kTanhPoly>{});
  else
    body(std::integral_constant<int, kTanhMufu>{});
}

// P = 2^(x - shift) of 64 keys as 16-bit pairs into tensor-memory columns dst ..
// dst + 31; returns their sum (fp32, before rounding).
template <typename T, bool SOFTCAP>
__device__ __forceinline__ float chunk_p(const Factors& f, const uint32_t (&raw)[64],
                                         uint32_t dst, bool masked, uint2 visible, float shift,
                                         bool mine) {
  const uint64_t nsh2 = f2_make(-shift, -shift), plain2 = f2_make(f.plain, f.plain);
  uint64_t sum2 = f2_make(0.f, 0.f);
  uint32_t packed[32];
  auto p_group = [&](auto form) {
#pragma unroll
    for (int u = 0; u < 32; ++u) {
      const uint64_t s2 = f2_make(raw[2 * u], raw[2 * u + 1]);
      const uint64_t y2 =
          SOFTCAP ? cap_pair<decltype(form)::value>(f, s2, nsh2) : f2_fma(s2, plain2, nsh2);
      float y0 = f2_lo(y2), y1 = f2_hi(y2);
      if (SOFTCAP && masked) {
        if (!bit_of(visible, 2 * u)) y0 = -INFINITY;
        if (!bit_of(visible, 2 * u + 1)) y1 = -INFINITY;
      }
      const float p0 = ex2_approx(y0), p1 = ex2_approx(y1);
      sum2 = f2_add(sum2, f2_make(p0, p1));
      packed[u] = pack_pair<T>(p0, p1);
    }
  };
  if constexpr (SOFTCAP)
    with_form(f, softcap::max_abs(raw), mine, p_group);
  else
    p_group(std::integral_constant<int, 0>{});
  uint32_t lo[16], hi[16];
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    lo[u] = packed[u];
    hi[u] = packed[16 + u];
  }
  tmem_st16(dst, lo);
  tmem_st16(dst + 16, hi);
  return f2_lo(sum2) + f2_hi(sum2);
}

constexpr int kBarBoth = 3;  // named barrier of both softmax warpgroups

// O (this warp's lanes, D / 2 columns from tO on) times f, 32 columns at a time.
template <int D>
__device__ __forceinline__ void scale_o(uint32_t tO, float f) {
  const uint64_t f2 = f2_make(f, f);
#pragma unroll
  for (int c32 = 0; c32 < D / 64; ++c32) {
    uint32_t o[32];
    tmem_ld32(tO + c32 * 32, o);
    uint32_t a[16], b[16];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint64_t v = f2_mul(f2_make(o[2 * u], o[2 * u + 1]), f2);
      const uint64_t x = f2_mul(f2_make(o[16 + 2 * u], o[17 + 2 * u]), f2);
      a[2 * u] = static_cast<uint32_t>(v);
      a[2 * u + 1] = static_cast<uint32_t>(v >> 32);
      b[2 * u] = static_cast<uint32_t>(x);
      b[2 * u + 1] = static_cast<uint32_t>(x >> 32);
    }
    tmem_st16(tO + c32 * 32, a);
    tmem_st16(tO + c32 * 32 + 16, b);
  }
}

// The sum of a row that sees nothing is 0 (of one that does 2^kHead or more, but for
// roundings), and NaN where one of its logits is, and then O and LSE are NaN too.
__device__ __forceinline__ float inverse_of(float total) {
  return total == 0.f ? 0.f : 1.f / total;
}
__device__ __forceinline__ float lse_of(float m, float total) {
  return total == 0.f ? -INFINITY : (m + __log2f(total)) * kLn2;
}

// One row's running shift (log2 units) and the sum of its weights above it.
struct Stats {
  float m, l;
};

// Takes the block's row maximum of raw scores in: moves the shift when the maximum
// outgrows it by more than kRescale, and then scales l and, once P V of block g - 1
// has completed, O. Returns the shift to use.
template <typename T, int D, bool SOFTCAP>
__device__ __forceinline__ float take_max(const Ctx& c, Stats& x, float smax, const Factors& fac,
                                          bool has_o, int g, uint32_t tO, bool& ok) {
  float m_tile = -INFINITY;  // the shift of this block's row maximum (log2 units)
  if (smax > -INFINITY) {
    // the weights' forms but the polynomial: above 1/4 an error of 1e-7 of the cap is
    // one of 2^-20 of the logit
    m_tile = smax * fac.plain;
    if (SOFTCAP) {
      const uint64_t s2 = f2_make(smax, smax), zero2 = f2_make(0.f, 0.f);
      m_tile = f2_lo(cap_pair<kTanhTaylor>(fac, s2, zero2));
      if (fabsf(smax) * fac.u > kTaylorMax) m_tile = f2_lo(cap_pair<kTanhMufu>(fac, s2, zero2));
    }
    m_tile -= kHead<T>;
  }
  const bool need = m_tile > x.m + kRescale<T>;
  if (__any_sync(0xffffffffu, need)) {
    const float m_new = need ? m_tile : x.m;
    const float f = need ? ex2_approx(x.m - m_new) : 1.f;  // 0 while m = -inf
    // a wait that gives up is voted on at the next barrier
    if (__any_sync(0xffffffffu, need && x.m > -INFINITY) && has_o) {
      if (!wait_warp(c, BAR_O_DONE + ((g - 1) & 1), ((g - 1) >> 1) & 1)) ok = false;
      if (ok) {
        tc_fence_after();
        scale_o<D>(tO, f);
      }
    }
    x.l *= f;
    x.m = m_new;
  }
  return x.m > -INFINITY ? x.m : 0.f;
}

// Writes 64 bytes of each of the warp's 32 rows through `stage` (2 KB of the
// warp's own), so that neighbouring lanes store neighbouring pieces of a row: lane
// r comes with row r's pieces and its address, 0 for none.
__device__ __forceinline__ void store_rows(uint8_t* stage, const uint32_t (&v)[16],
                                           unsigned long long address) {
  const int lane = threadIdx.x & 31;
  // piece j of row r at 4 r + (j ^ (r / 2 mod 4)): eight neighbouring lanes, on
  // either side, are on all banks
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(stage + (lane * 4 + (j ^ ((lane >> 1) & 3))) * 16) =
        make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
  const int j = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 8 * i + (lane >> 2);
    const unsigned long long to = __shfl_sync(0xffffffffu, address, row);
    if (to != 0)
      reinterpret_cast<uint4*>(to)[j] =
          *reinterpret_cast<const uint4*>(stage + (row * 4 + (j ^ ((row >> 1) & 3))) * 16);
  }
  __syncwarp();
}

// What the epilogue of a tile needs: this row's statistics, the part's blocks of the
// tile, its place in the batch.
struct Done {
  Stats x;
  int take, blk, nt, left;
  int row0, kvh, rows;
  bool narrow;
};

// Writes out O and LSE of tile i of the part, or what the part has of them, once
// the tile's last P V has completed. That has a barrier of its own for each O
// buffer: by now the next tile's blocks may have completed too, which moves O_DONE
// on, but the tile after that waits for this epilogue to free the buffer.
template <typename T, int D, bool SOFTCAP>
__device__ __forceinline__ bool epilogue(const Ctx& c, const Params& p, const Part& part,
                                         const Done& d, bool ok, int i, int h, uint32_t lanes,
                                         float* xsum, float* shifts, uint8_t* smem,
                                         uint8_t* stage, int token) {
  using L = Layout<D>;
  const int lane = threadIdx.x & 31;
  const int quadrant = (threadIdx.x >> 5) & 3;
  const int r = (quadrant << 5) + lane;
  const uint32_t tO = lanes + 256 + (i % L::kOBufs) * D + h * (D / 2);
  const int row = d.narrow ? lane : r;
  const bool idle = !d.narrow && (r & ~31) >= d.rows;
  if (ok) ok = wait(c, BAR_O_LAST + i % L::kOBufs, (i / L::kOBufs) & 1);
  xsum[h * 128 + r] = d.x.l;
  if (kHasNarrow<D, SOFTCAP> && d.narrow && h == 0) shifts[r] = d.x.m;
  if (!named_bar_and(kBarBoth, 256, ok)) return false;
  tc_fence_after();
  const bool whole = d.blk == 0 && d.take == d.nt;
  const int head = d.kvh * p.G + row - token * p.G;
  const long long out_row = static_cast<long long>(d.row0) + token;
  float* partial = reinterpret_cast<float*>(p.workspace + kSharedBytes) +
                   (2LL * blockIdx.x + (d.blk == 0 ? 1 : 0)) * slot_floats(D);
  if (kHasNarrow<D, SOFTCAP> && d.narrow) {
    // the quadrants' shifts and sums of a row
    auto join = [&](int at, float& M, float& total) {
      M = -INFINITY;
      total = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) M = fmaxf(M, shifts[32 * k + at]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        total = fmaf(xsum[32 * k + at] + xsum[128 + 32 * k + at],
                     shifts[32 * k + at] > -INFINITY ? ex2_approx(shifts[32 * k + at] - M) : 1.f,
                     total);  // without a maximum the sum is 0, or NaN
    };
    float M, total;
    join(lane, M, total);
    const float f = d.x.m > -INFINITY ? ex2_approx(d.x.m - M) : 0.f;
    if (quadrant == 0 && h == 0 && lane < d.rows) {
      if (!whole) {
        partial[lane] = M;
        partial[128 + lane] = total;
      } else if (p.lse != nullptr) {
        p.lse[out_row * p.H + head] = lse_of(M, total);
      }
    }
    // [quadrant][row][column] fp32 over all of the warps' stages, then the quadrants
    // added in order
    float* sum = reinterpret_cast<float*>(smem + L::kStage);
#pragma unroll
    for (int c0 = 0; c0 < D / 2; c0 += 32) {
      uint32_t o[32];
      tmem_ld32(tO + c0, o);
      if (lane < d.rows) {
        float4* to = reinterpret_cast<float4*>(sum + (quadrant * p.narrow + lane) * D +
                                               h * (D / 2) + c0);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          to[u] = f > 0.f ? make_float4(__uint_as_float(o[4 * u]) * f,
                                        __uint_as_float(o[4 * u + 1]) * f,
                                        __uint_as_float(o[4 * u + 2]) * f,
                                        __uint_as_float(o[4 * u + 3]) * f)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    named_bar_sync(kBarBoth, 256);
    const int k = static_cast<int>(threadIdx.x) - 128;  // rows * D / 4 <= 256
    if (k < d.rows * (D / 4)) {
      const int at = k / (D / 4), col = (k % (D / 4)) * 4;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 v = *reinterpret_cast<const float4*>(sum + (q * p.narrow + at) * D + col);
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
      }
      if (!whole) {
        *reinterpret_cast<float4*>(partial + 256 + at * D + col) = o;
      } else {
        join(at, M, total);
        const float inv = inverse_of(total);
        const int tok = at / p.G;
        T* out = static_cast<T*>(p.o) + (static_cast<long long>(d.row0) + tok) * p.o_token +
                 (d.kvh * p.G + at - tok * p.G) * p.o_head + col;
        *reinterpret_cast<uint2*>(out) =
            make_uint2(pack_pair<T>(o.x * inv, o.y * inv), pack_pair<T>(o.z * inv, o.w * inv));
      }
    }
  } else if (!idle) {
    const bool mine = r < d.rows;
    const float total = xsum[r] + xsum[128 + r];
    if (whole) {
      T* out = static_cast<T*>(p.o) + out_row * p.o_token + head * p.o_head + h * (D / 2);
      const float inv = inverse_of(total);
      const uint64_t inv2 = f2_make(inv, inv);
#pragma unroll
      for (int c0 = 0; c0 < D / 2; c0 += 32) {
        uint32_t raw[32], packed[16];
        tmem_ld32(tO + c0, raw);
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const uint64_t v = f2_mul(f2_make(raw[2 * u], raw[2 * u + 1]), inv2);
          // a row that sees nothing: its P V was 0 times what V held
          packed[u] = total != 0.f ? pack_pair<T>(f2_lo(v), f2_hi(v)) : 0u;
        }
        store_rows(stage, packed, mine ? reinterpret_cast<unsigned long long>(out + c0) : 0ull);
      }
      if (mine && h == 0 && p.lse != nullptr)
        p.lse[out_row * p.H + head] = lse_of(d.x.m, total);
    } else {
      if (mine && h == 0) {
        partial[r] = d.x.m;
        partial[128 + r] = total;
      }
      float* to = partial + 256 + r * D + h * (D / 2);
#pragma unroll
      for (int c0 = 0; c0 < D / 2; c0 += 16) {
        uint32_t raw[16];
        tmem_ld16(tO + c0, raw);
        store_rows(stage, raw, mine ? reinterpret_cast<unsigned long long>(to + c0) : 0ull);
      }
    }
  }
  if (d.blk == 0 && d.take < d.nt && threadIdx.x == 128) {
    // the tile goes on in the parts behind: the last of them holds its last unit
    const long long end = part.first + part.count - d.left;
    Shared s;
    s.parts = static_cast<int>((end - 1) / part.share) - static_cast<int>(blockIdx.x) + 1;
    s.row0 = d.row0;
    s.kvh = d.kvh;
    s.rows = d.rows;
    reinterpret_cast<Shared*>(p.workspace)[blockIdx.x] = s;
  }
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar_addr(c, BAR_O_FREE + i % L::kOBufs));
  return true;
}

// Thread r of each warpgroup owns row r; the warpgroups exchange the half-row
// maxima through shared memory once per block, so that both take the same shift.
// Warps without a row of the tile only keep the barriers' count. In a narrow tile
// lane r of every quadrant owns row r and has sums of its own over the quadrant's
// keys, joined at the end.
template <typename T, int D, bool SOFTCAP>
__device__ void softmax_role(const Ctx& c, const Params& p, const Part& part, uint8_t* smem,
                             uint32_t tmem) {
  using L = Layout<D>;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int h = (warp - 4) >> 2;  // which half of the keys (and of O's columns)
  const int quadrant = warp & 3;
  const int r = (quadrant << 5) + lane;
  const uint32_t lane_base = static_cast<uint32_t>(r & ~31) << 16;
  float* xmax = reinterpret_cast<float*>(smem + L::kXchg);  // [block parity][half][row]
  float* xsum = xmax + 4 * 128;                              // [half][row]
  float* shifts = reinterpret_cast<float*>(smem + L::kShifts);
  uint8_t* stage = smem + L::kStage + (warp - 4) * 2048;
  const int wide_token = r / p.G, narrow_token = lane / p.G;
  const Factors fac{p.scale * kLog2e, SOFTCAP ? p.scale / p.softcap : 0.f,
                    SOFTCAP ? 2.f * kLog2e * p.scale / p.softcap : 0.f,
                    SOFTCAP ? p.softcap * kLog2e : 0.f};
  bool ok = true;
  int g = 0;  // blocks of all tiles before
  int i = 0;
  Walk w(p, part);
  for (; ok && w.step(p); ++i) {
    const int nt = w.take;
    const int rows = w.t.count * p.G;
    const bool narrow = is_narrow<D, SOFTCAP>(p, w.t);
    const int token = narrow ? narrow_token : wide_token;
    const bool idle = !narrow && (r & ~31) >= rows;  // the warp has no row
    const uint32_t tO = tmem + lane_base + 256 + (i % L::kOBufs) * D + h * (D / 2);
    // the keys that this row sees, and those that every row of the tile sees
    const int pos = w.t.pos0 + token;
    const int hi = p.causal ? min(pos, w.s.length - 1) : w.s.length - 1;
    const int lo = p.left < 0 ? 0 : pos - p.left;
    const int all_hi = p.causal ? min(w.t.pos0, w.s.length - 1) : w.s.length - 1;
    const int all_lo = p.left < 0 ? 0 : w.t.pos0 + w.t.count - 1 - p.left;
    Stats x{-INFINITY, 0.f};
    if (kHasNarrow<D, SOFTCAP> && narrow) {
      for (int t = 0; t < nt; ++t) {
        const int gb = g + t;
        const int n0 = w.t.block(w.blk + t) * kBn;
        const uint32_t tS = tmem + lane_base + (gb & 1) * 128;
        const bool masked = n0 + kBn - 1 > all_hi || (n0 < all_lo && n0 + kBn > p.sinks);
        const bool got = wait(c, BAR_S_DONE + (gb & 1), (gb >> 1) & 1);
        float* slot = xmax + (gb & 1) * 256;
        // keys 32 quadrant + 16 h .. + 15 of the block
        const int key0 = n0 + 32 * quadrant + 16 * h;
        uint32_t raw[16];
        uint32_t visible = 0xffffu;
        float hmax = -INFINITY, most = 0.f;
        if (got) {
          tc_fence_after();
          tmem_ld16(tS + 32 * quadrant + 16 * h, raw);
          if (masked) visible = visible_bits(key0, lo, hi, p.sinks).x;
          if (lane >= rows) visible = 0;  // these lanes' scores are of no row
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const bool seen = (visible >> e) & 1u;
            if (seen) hmax = fmaxf(hmax, __uint_as_float(raw[e]));
            if (seen) most = fmaxf(most, fabsf(__uint_as_float(raw[e])));
          }
        }
        slot[h * 128 + r] = hmax;
        ok = named_bar_and(kBarBoth, 256, ok && got);
        if (!ok) break;
        const float smax = fmaxf(hmax, slot[(1 - h) * 128 + r]);
        const float shift = take_max<T, D, SOFTCAP>(c, x, smax, fac, t > 0, gb, tO, ok);
        // P of the warp's 16 keys; 0 for the keys of the other quadrants: of the
        // 64 pair columns (0 .. 31 and 64 .. 95), in groups of 8 (16 keys),
        // warpgroup h writes groups h, 2 + h, 4 + h, 6 + h, its keys' one among them
        uint32_t pairs[8], zeros[8];
        with_form(fac, most, true, [&](auto form) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            // the logit of what a hidden score holds is not used
            const uint64_t y2 = cap_pair<decltype(form)::value>(
                fac, f2_make(raw[2 * u], raw[2 * u + 1]), f2_make(-shift, -shift));
            const float p0 = ex2_approx((visible >> (2 * u)) & 1u ? f2_lo(y2) : -INFINITY);
            const float p1 = ex2_approx((visible >> (2 * u + 1)) & 1u ? f2_hi(y2) : -INFINITY);
            x.l += p0 + p1;
            pairs[u] = pack_pair<T>(p0, p1);
            zeros[u] = 0u;
          }
        });
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int group = 2 * j + h;
          const uint32_t dst = tS + 8 * group + (group >= 4 ? 32 : 0);
          if (j == quadrant)
            tmem_st8(dst, pairs);
          else
            tmem_st8(dst, zeros);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_addr(c, BAR_P_FULL + (gb & 1)));  // one arrival per warp
      }
    } else {
      for (int t = 0; t < nt; ++t) {
        const int gb = g + t;
        const int n0 = w.t.block(w.blk + t) * kBn;
        const int key0 = n0 + 64 * h;
        const uint32_t tS = tmem + lane_base + (gb & 1) * 128;
        const bool masked =
            n0 + kBn - 1 > all_hi || (n0 < all_lo && n0 + kBn > p.sinks);
        const bool got = wait(c, BAR_S_DONE + (gb & 1), (gb >> 1) & 1);
        uint32_t raw[64];
        uint2 visible = make_uint2(~0u, ~0u);
        float hmax = -INFINITY;
        if (got && !idle) {
          tc_fence_after();
          tmem_ld32x2(tS + 64 * h, tS + 64 * h + 32, raw);
          float m0 = -INFINITY, m1 = -INFINITY;
          if (masked) {
            visible = visible_bits(key0, lo, hi, p.sinks);
            // hidden scores become -inf; with a softcap 0, which keeps them out of
            // the choice of tanh's form (chunk_p hides the logits)
#pragma unroll
            for (int e = 0; e < 64; ++e) {
              const bool seen = bit_of(visible, e);
              if (SOFTCAP) {
                if (seen) m0 = fmaxf(m0, __uint_as_float(raw[e]));
                if (!seen) raw[e] = 0u;
              } else if (!seen) {
                raw[e] = 0xff800000u;
              }
            }
          }
          if (!SOFTCAP || !masked) {
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              m0 = fmaxf(m0, __uint_as_float(raw[e]));
              m1 = fmaxf(m1, __uint_as_float(raw[e + 1]));
            }
          }
          hmax = fmaxf(m0, m1);
        }
        float* slot = xmax + (gb & 1) * 256;
        slot[h * 128 + r] = hmax;
        ok = named_bar_and(kBarBoth, 256, ok && got);
        if (!ok) break;
        if (!idle) {
          const float smax = fmaxf(hmax, slot[(1 - h) * 128 + r]);
          const float shift = take_max<T, D, SOFTCAP>(c, x, smax, fac, t > 0, gb, tO, ok);
          x.l +=
              chunk_p<T, SOFTCAP>(fac, raw, tS + 64 * h, masked, visible, shift, r < rows);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_addr(c, BAR_P_FULL + (gb & 1)));  // one arrival per warp
      }
    }
    const Done done{x, nt, w.blk, w.t.nt, w.left, w.s.row0 + w.tile * p.tokens,
                    w.kvh, rows, narrow};
    ok = epilogue<T, D, SOFTCAP>(c, p, part, done, ok, i, h, tmem + lane_base, xsum, shifts,
                                 smem, stage, token);
    g += nt;
  }
}

// ------------------------------------------------------------------ kernels
template <typename T, int D, bool SOFTCAP>
__global__ void __launch_bounds__(kThreads, 1)
    cache_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_qn,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  Ctx c;
  c.bars = sbase + L::kBars;
  c.abort = reinterpret_cast<volatile int*>(smem + L::kAbort);
  Part* part = reinterpret_cast<Part*>(smem + L::kPart);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(bar_addr(c, i), 1);
    for (int sl = 0; sl < 2; ++sl) {
      mbar_init(bar_addr(c, BAR_P_FULL + sl), 8);  // one arrival per softmax warp
      mbar_init(bar_addr(c, BAR_O_FREE + sl), 8);
    }
    *c.abort = (sbase & 1023u) != 0;  // the swizzle atoms need 1024-byte alignment
    if (sbase & 1023u) record_status(ATTN_ERR_DEVICE);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(sbase + L::kTmemSlot, 512);
    tmem_relinquish();
  }
  if (warp == 2 && (threadIdx.x & 31) == 0) {
    prefetch_tmap(p.narrow > 0 ? &tm_qn : &tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // rows that no tile's copy fills hold zeros, not what shared memory held before
  const int unused = kBm - p.tokens * p.G;
  for (int i = threadIdx.x; i < L::kQStages * (D / 64) * unused * 8; i += kThreads) {
    const int row = kBm - 1 - (i >> 3) % unused, box = (i >> 3) / unused;
    *reinterpret_cast<uint4*>(smem + L::kQ + box * 16384 + row * 128 + (i & 7) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  grid_dependency_wait();
  grid_dependency_launch();
  if (threadIdx.x == 0) reinterpret_cast<Shared*>(p.workspace)[blockIdx.x].parts = 0;
  tc_fence_before();
  find_part(p, reinterpret_cast<long long*>(smem + L::kSums), part);
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kTmemSlot);
  if (*c.abort == 0) {
    if (warp < 4) {
      setmaxnreg_dec<kRegsCtl<D>>();
      if (warp == 0)
        loader_role<D, SOFTCAP, false>(c, p, *part, sbase, &tm_q, &tm_qn, &tm_k);
      if (warp == 1) {
        if (elect_one_sync()) issue_mmas<T, D>(c, p, *part, sbase, tmem);
        __syncwarp();
      }
      if (warp == 2)
        loader_role<D, SOFTCAP, true>(c, p, *part, sbase, &tm_q, &tm_qn, &tm_v);
      if (warp == 3) zero_role<D>(c, p, *part, smem);
    } else {
      setmaxnreg_inc<kRegsSoftmax<D>>();
      softmax_role<T, D, SOFTCAP>(c, p, *part, smem, tmem);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the tile that begins in part blockIdx.x and goes on behind
// it: M = max m_i, L = sum l_i 2^(m_i - M), O = sum O_i 2^(m_i - M) / L. One warp a
// row, D / 32 columns a lane, parts in order; where a tile has more than kJoinFew
// parts the warps of a block share a row, warp k takes parts k, k + 8, ... and the
// warps' sums are added in order (one token over 131072 keys, one key/value head:
// 147 parts, 86 us with a warp a row, 32 so).
constexpr int kJoinWarps = 8, kJoinSplit = 128 / kJoinWarps, kJoinFew = 8;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) cache_join_kernel(const Params p) {
  grid_dependency_wait();
  const Shared s = reinterpret_cast<const Shared*>(p.workspace)[blockIdx.x];
  if (s.parts == 0) return;
  const bool few = s.parts <= kJoinFew;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = few ? 0 : warp, step = few ? 1 : kJoinWarps;
  constexpr int E = D / 32;
  __shared__ float2 sums[kJoinWarps][32][E / 2];
  __shared__ float totals[kJoinWarps];
  const float* slots = reinterpret_cast<const float*>(p.workspace + kSharedBytes) +
                       2LL * blockIdx.x * slot_floats(D);
  // part i of the tile: slot 1 of the first CTA, slot 0 of the ones behind
  auto slot = [&](int i) { return slots + (i == 0 ? 1 : 2 * i) * slot_floats(D); };
  constexpr int kAhead = 4;  // parts whose O is on its way before the weights are known
  // every warp of a block that shares its rows goes through the same ones
  for (int r = few ? blockIdx.y * kJoinWarps + warp : blockIdx.y; r < s.rows;
       r += few ? 128 : kJoinSplit) {
    float2 v[kAhead][E / 2];
    auto load = [&](int i, float2 (&to)[E / 2]) {
      const float* from = slot(i) + 256 + r * D + lane * E;
#pragma unroll
      for (int e = 0; e < E / 2; ++e) to[e] = reinterpret_cast<const float2*>(from)[e];
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (first + u * step < s.parts) load(first + u * step, v[u]);
    float M = -INFINITY;
    for (int i = lane; i < s.parts; i += 32) M = fmaxf(M, slot(i)[r]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    const float shift = M > -INFINITY ? M : 0.f;
    float2 o[E / 2];
    float total = 0.f;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) o[e] = make_float2(0.f, 0.f);
    for (int i0 = first; i0 < s.parts; i0 += kAhead * step) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * step;
        if (i >= s.parts) break;
        const float f = ex2_approx(slot(i)[r] - shift), l = slot(i)[128 + r];
        total = fmaf(l, f, total);
        if (f > 0.f) {  // a part that saw nothing holds no numbers
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            o[e].x = fmaf(v[u][e].x, f, o[e].x);
            o[e].y = fmaf(v[u][e].y, f, o[e].y);
          }
        }
        if (i + kAhead * step < s.parts) load(i + kAhead * step, v[u]);
      }
    }
    if (!few) {
      __syncthreads();  // the row before has been read
#pragma unroll
      for (int e = 0; e < E / 2; ++e) sums[warp][lane][e] = o[e];
      if (lane == 0) totals[warp] = total;
      __syncthreads();
      if (warp != 0) continue;
      for (int k = 1; k < kJoinWarps; ++k) {
        total += totals[k];
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          o[e].x += sums[k][lane][e].x;
          o[e].y += sums[k][lane][e].y;
        }
      }
    }
    const float inv = inverse_of(total);
    const int token = r / p.G, head = s.kvh * p.G + r - token * p.G;
    const long long row = static_cast<long long>(s.row0) + token;
    T* out = static_cast<T*>(p.o) + row * p.o_token + head * p.o_head + lane * E;
#pragma unroll
    for (int e = 0; e < E / 2; ++e)
      reinterpret_cast<uint32_t*>(out)[e] = pack_pair<T>(o[e].x * inv, o[e].y * inv);
    if (lane == 0 && p.lse != nullptr)
      p.lse[row * p.H + head] = lse_of(M, total);
  }
}

// ------------------------------------------------------------------ host
// 4-D tensor map over 2-byte elements, innermost d; strides in elements of the
// outer dimensions (0 for those of one element), box {64, box[0..2]}, 128-byte
// swizzle, zero fill outside the tensor.
template <typename T>
bool encode_4d(CUtensorMap* map, const void* base, int d, const long long (&extent)[3],
               const long long (&stride)[3], const int (&box)[3]) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d)}, strides[3];
  cuuint32_t boxes[4] = {64}, es[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = static_cast<cuuint64_t>(extent[i]);
    strides[i] = static_cast<cuuint64_t>(stride[i] > 0 ? stride[i] : d) * 2;
    boxes[i + 1] = static_cast<cuuint32_t>(box[i]);
  }
  const CUresult r = enc(
      map, std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
      4, const_cast<void*>(base), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B,
      d == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

struct Tensors {
  const void *q, *k, *v;
  long long q_in[2], k_in[3], v_in[3];
};

template <typename T, int D, bool SOFTCAP>
int launch(const CUtensorMap (&maps)[4], const Params& p, int ctas, bool join,
           cudaStream_t stream) {
  auto kern = cache_fwd_kernel<T, D, SOFTCAP>;
  static std::atomic<bool> configured[kMaxTrackedDevices];
  if (!set_smem_limit_once(kern, Layout<D>::kBytes, configured)) return ATTN_ERR_LAUNCH;
  const int rc = launch_overlapped(kern, dim3(static_cast<unsigned>(ctas)), kThreads,
                                   Layout<D>::kBytes, 0, stream, maps[0], maps[1], maps[2],
                                   maps[3], p);
  if (rc != ATTN_OK || !join) return rc;
  return launch_overlapped(cache_join_kernel<T, D>,
                           dim3(static_cast<unsigned>(ctas), kJoinSplit), 32 * kJoinWarps, 0, 0,
                           stream, p);
}

template <typename T>
int run(const Tensors& x, const Params& given, int d, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_LAUNCH;
  CUtensorMap maps[4];  // Q, Q of narrow tiles, K, V
  const Batch& c = given.batch;
  const long long q_extent[3] = {given.G, given.H_kv, c.T};
  const long long q_stride[3] = {x.q_in[1], x.q_in[1] * given.G, x.q_in[0]};
  const long long extent[3] = {given.H_kv, c.page_size, c.n_pages};
  const long long k_stride[3] = {x.k_in[2], x.k_in[1], x.k_in[0]};
  const long long v_stride[3] = {x.v_in[2], x.v_in[1], x.v_in[0]};
  const int narrow_tokens = given.narrow > 0 ? given.narrow / given.G : 1;
  if (!encode_4d<T>(&maps[0], x.q, d, q_extent, q_stride, {given.G, 1, given.tokens}) ||
      (given.narrow > 0 &&
       !encode_4d<T>(&maps[1], x.q, d, q_extent, q_stride, {given.G, 1, narrow_tokens})) ||
      !encode_4d<T>(&maps[2], x.k, d, extent, k_stride, {1, given.box, 1}) ||
      !encode_4d<T>(&maps[3], x.v, d, extent, v_stride, {1, given.box, 1}))
    return ATTN_ERR_LAUNCH;
  if (given.narrow == 0) maps[1] = maps[0];  // not used
  // as many parts as there can be blocks, one an SM at most
  const long long tiles = (c.T / given.tokens + static_cast<long long>(c.B)) * given.H_kv;
  const long long blocks = (given.cap + kBn - 1) / kBn;
  // Where the page table holds few blocks, tiles are left whole: walking them one
  // behind another costs less than the second kernel does. One token, 32 heads
  // over 8, in a graph, whole against cut: d = 128, 240 keys 7.4 us against 9.0,
  // 499 keys 8.8 against 9.8, 1000 keys 11.9 against 10.9; d = 256, whose one stage
  // makes a block take twice as long, 400 keys 13.3 against 11.2. 1.7 us less of
  // the host's time, too.
  Params p = given;
  p.whole = blocks <= (d == 256 ? 2 : 6);
  const long long pieces = p.whole ? tiles : tiles * blocks;
  const int most = sms < kMaxCtas ? sms : kMaxCtas;
  const int ctas = tiles >= most || pieces >= most ? most : static_cast<int>(pieces);
  const bool join = !p.whole;
  const bool cap = p.softcap > 0.f;
  if (d == 64)
    return cap ? launch<T, 64, true>(maps, p, ctas, join, stream)
               : launch<T, 64, false>(maps, p, ctas, join, stream);
  if (d == 128)
    return cap ? launch<T, 128, true>(maps, p, ctas, join, stream)
               : launch<T, 128, false>(maps, p, ctas, join, stream);
  return cap ? launch<T, 256, true>(maps, p, ctas, join, stream)
             : launch<T, 256, false>(maps, p, ctas, join, stream);
}

// Sizes that both entry points check.
int check_sizes(int T, int B, int H, int H_kv, int d) {
  if (T < 0 || B < 0 || H < 0 || H_kv < 1 || H % H_kv != 0 || d < 1) return ATTN_ERR_SHAPE;
  if (d != 64 && d != 128 && d != 256) return ATTN_ERR_UNSUPPORTED;
  if (H / H_kv > 128) return ATTN_ERR_UNSUPPORTED;
  if (H > 16384 || T > (1 << 29) || B > (1 << 29) ||
      static_cast<long long>(T) * H >= (1LL << 40) / d)
    return ATTN_ERR_TOO_LARGE;
  return ATTN_OK;
}

}  // namespace cachefwd

int cache_fwd_status(int* status, bool clear) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, cachefwd::g_status, sizeof(int)) != cudaSuccess)
    return ATTN_ERR_LAUNCH;
  *status = v;
  const int zero = 0;
  if (clear && v != 0 &&
      cudaMemcpyToSymbol(cachefwd::g_status, &zero, sizeof(int)) != cudaSuccess)
    return ATTN_ERR_LAUNCH;
  return ATTN_OK;
}

}  // namespace attn

using namespace attn;

extern "C" long long attn_cache_fwd_workspace_bytes(int T, int B, int H, int H_kv, int d) {
  const int rc = cachefwd::check_sizes(T, B, H, H_kv, d);
  if (rc != ATTN_OK) return rc;
  return cachefwd::kSharedBytes + cachefwd::kMaxCtas * 2LL * cachefwd::slot_floats(d) * 4;
}

extern "C" int attn_cache_fwd(const void* q, const void* k_cache, const void* v_cache, void* o,
                              float* lse, const int* starts, const int* lengths, const int* pages,
                              void* workspace, int T, int B, int H, int H_kv, int d,
                              int page_size, int max_pages, int n_pages, float scale, int causal,
                              float softcap, int window_left, int sinks, int dtype,
                              const long long* strides, void* stream) {
  cachefwd::Params p{};
  p.batch = {starts, lengths, pages, T, B, page_size, max_pages, n_pages};
  int rc = cache::check_batch(p.batch);
  if (rc != ATTN_OK) return rc;
  rc = cachefwd::check_sizes(T, B, H, H_kv, d);
  if (rc != ATTN_OK) return rc;
  if (!std::isfinite(scale) || !(scale > 0.f) || std::isnan(softcap) || sinks < 0)
    return ATTN_ERR_SHAPE;
  if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_SHAPE;
  if (page_size % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  const bool empty = T == 0 || B == 0 || H == 0;
  if (!empty && n_pages < 1) return ATTN_ERR_SHAPE;
  if (!empty && (!q || !k_cache || !v_cache || !o || !workspace)) return ATTN_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
      !aligned16(lse) || !aligned16(workspace))
    return ATTN_ERR_ALIGN;
  cachefwd::Tensors x{q, k_cache, v_cache, {}, {}, {}};
  long long o_to[2];
  auto at = [&](int i) { return strides != nullptr ? strides + i : nullptr; };
  // no broadcast inputs either: a tensor map's strides are positive
  if ((rc = cache::row_strides(x.q_in, at(0), T, H, d, true)) != ATTN_OK ||
      (rc = cache::row_strides(o_to, at(2), T, H, d, true)) != ATTN_OK ||
      (rc = cache::cache_strides(x.k_in, at(4), p.batch, H_kv, d, true)) != ATTN_OK ||
      (rc = cache::cache_strides(x.v_in, at(7), p.batch, H_kv, d, true)) != ATTN_OK)
    return rc;
  long long bits = 0;
  for (int i = 0; i < 2; ++i) bits |= x.q_in[i] | o_to[i];
  for (int i = 0; i < 3; ++i) bits |= x.k_in[i] | x.v_in[i];
  if (bits % 8 != 0) return ATTN_ERR_ALIGN;
  if (empty) return ATTN_OK;
  p.o = o;
  p.lse = lse;
  p.o_token = o_to[0];
  p.o_head = o_to[1];
  p.workspace = static_cast<char*>(workspace);
  p.H = H;
  p.H_kv = H_kv;
  p.G = H / H_kv;
  p.tokens = cachefwd::kBm / p.G;
  p.box = cachefwd::kBn;
  while (page_size % p.box != 0) p.box /= 2;
  const long long cap = static_cast<long long>(max_pages) * page_size;
  p.cap = cap < (1LL << 30) ? static_cast<int>(cap) : 1 << 30;
  p.scale = scale;
  p.softcap = softcap > 0.f ? softcap : 0.f;
  p.narrow = (!(softcap > 0.f) ? 0
              : d == 64        ? cachefwd::Layout<64>::kNarrow
              : d == 128       ? cachefwd::Layout<128>::kNarrow
                               : 0) /
             p.G * p.G;  // whole tokens
  p.causal = causal != 0;
  p.left = window_left > (1 << 30) ? 1 << 30 : window_left;
  p.sinks = sinks;
  return dtype == ATTN_BF16 ? cachefwd::run<__nv_bfloat16>(x, p, d, as_stream(stream))
                            : cachefwd::run<__half>(x, p, d, as_stream(stream));
}
