// attn_cache_fwd: attention of a ragged batch's new tokens over a paged
// key/value cache, on the tcgen05 tensor cores.
//
// Row t of the batch, at position p of its sequence, and query head h see the keys
// j <= p (or all of the sequence's) with j >= p - left or j < sinks:
//   x_j = logit of q and key j (log2 units),  O = sum_j 2^(x_j - m) v_j / l,
//   l = sum_j 2^(x_j - m),  LSE = (m + log2 l) ln 2
// with a running maximum m and sum l, as in attn_fwd: S = Q K^T in fp32 tensor
// memory, P as 16-bit pairs over it, O accumulated in tensor memory and rescaled
// only when a row's maximum grows by more than 2^8.
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
//   warp 0      Q of each tile; K in a ring of 2 stages (d <= 128) or 1
//   warp 2      V in the same kind of ring
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
constexpr int kMaxCtas = 192;  // parts of the line at most (the workspace's size)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.f;  // move the shift only when the maximum grows by more
constexpr long long kWaitLimitCycles = 2000000000LL;  // about one second

// The softmax warps' state does not fit in the 168 registers that 384 threads are
// launched with: setmaxnreg moves registers to them from the loaders and the MMA
// warp.
constexpr int kRegsSoftmax = 216, kRegsCtl = 72;
static_assert(256 * kRegsSoftmax + 128 * kRegsCtl <= 384 * 168, "register pool");

template <int D>
struct Layout {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kStages = D <= 128 ? 2 : 1;   // of K, of V, of Q
  static constexpr int kOBufs = D <= 128 ? 2 : 1;    // O accumulators in tensor memory
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kStages * kTileBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  // the softmax warpgroups' half-row maxima (two blocks in flight) and row sums:
  // [2][2][128] + [2][128] fp32
  static constexpr int kXchg = kV + kStages * kTileBytes;
  static constexpr int kBars = kXchg + 6 * 128 * 4;
  static constexpr int kNumBars = 24;
  static constexpr int kSums = kBars + kNumBars * 8;   // [kWarps] long long
  static constexpr int kPart = kSums + kWarps * 8;     // Part
  static constexpr int kTmemSlot = kPart + 48;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kUsed = kAbort + 12;
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
  BAR_K_EMPTY = 6,   // + stage
  BAR_V_FULL = 8,    // + stage
  BAR_V_EMPTY = 10,  // + stage
  BAR_S_FULL = 12,   // + S buffer (block parity): S of the block written
  BAR_P_FULL = 14,   // + S buffer: P of the block written (and O rescaled if needed)
  BAR_O_DONE = 16,   // P V of a block completed (one phase per key block)
  BAR_O_LAST = 17,   // the tile's last P V completed (one phase per tile)
  BAR_O_FREE = 18,   // + O buffer: the tile's epilogue has read O
  BAR_V_EDGE = 20,   // + stage: copies of a V block some of whose rows are then zeroed
  BAR_DRAIN = 22,    // abort path only: completion of everything issued
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
  } else {
    t.ns = sink_blocks;
    t.nt = max(1, sink_blocks);
    t.j0 = 0;
  }
  return t;
}

// Blocks of one key/value head's tiles of a sequence, summed by a whole warp.
__device__ __forceinline__ long long head_blocks(const Params& p, const Seq& s) {
  const int lane = threadIdx.x & 31;
  long long sum = 0;
  for (int i = lane; i < s.tiles; i += 32) sum += tile_of(p, s, i).nt;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  return sum;
}

// Blocks of one key/value head for sequence b0 + lane (0 past the end), a whole
// warp together: sequences of one tile in parallel, longer ones one by one.
__device__ __forceinline__ long long lane_blocks(const Params& p, int b0, int end) {
  const int lane = threadIdx.x & 31;
  Seq s{};
  if (b0 + lane < end) s = seq_of(p, b0 + lane);
  long long blocks = s.tiles == 1 ? tile_of(p, s, 0).nt : 0;
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
    const long long sum = head_blocks(p, o);
    if (lane == src) blocks = sum;
  }
  return blocks;
}

// A CTA's part of the line: where it begins, how many blocks it has, and how many
// a full part has.
struct Part {
  int b, kvh, tile, blk;
  long long count, share, first;
};

// Finds the CTA's part (every thread of the CTA calls; `sums` and `part` in
// shared memory). Warp w sums the blocks of its chunk of the sequences, 32 at a
// time; the warp whose chunk holds the part's first block then looks for it there
// (a chunk of up to 32 sequences, so up to 384 in all, is not summed again).
__device__ __forceinline__ void find_part(const Params& p, long long* sums, Part* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int B = p.batch.B;
  const int chunk = (B + kWarps - 1) / kWarps;
  const int first = min(B, warp * chunk), end = min(B, first + chunk);
  long long sum = 0, mine = 0;
  for (int b = first; b < end; b += 32) sum += mine = lane_blocks(p, b, end);
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
      const long long blocks = (chunk <= 32 ? mine : lane_blocks(p, b, end)) * p.H_kv;
      long long upto = blocks;  // inclusive sum over the lanes
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
      const long long per_head = __shfl_sync(0xffffffffu, blocks, src) / p.H_kv;
      at -= __shfl_sync(0xffffffffu, upto - blocks, src);
      const int kvh = static_cast<int>(at / per_head);
      at -= kvh * per_head;
      const Seq s = seq_of(p, b + src);
      for (int i = 0; i < s.tiles; i += 32) {
        const int nt = i + lane < s.tiles ? tile_of(p, s, i + lane).nt : 0;
        int sum_to = nt;
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
        at -= __shfl_sync(0xffffffffu, sum_to - nt, t);
        if (lane == 0) {
          part->b = b + src;
          part->kvh = kvh;
          part->tile = i + t;
          part->blk = static_cast<int>(at);
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

// Walks the tiles of a part; every role has its own.
struct Walk {
  int b, kvh, tile, blk, take, left;
  Seq s;
  Tile t;
  __device__ __forceinline__ void begin(const Params& p, const Part& part) {
    b = part.b;
    kvh = part.kvh;
    tile = part.tile;
    blk = part.blk;
    left = static_cast<int>(part.count);
    if (left > 0) {
      s = seq_of(p, b);
      t = tile_of(p, s, tile);
      take = min(t.nt - blk, left);
      if (p.whole) {  // a tile belongs to the part that holds its first block
        if (blk > 0)
          next(p);
        else
          take = t.nt;
      }
    }
  }
  __device__ __forceinline__ void next(const Params& p) {
    left -= take;
    if (left <= 0) return;
    blk = 0;
    if (++tile == s.tiles) {
      tile = 0;
      if (++kvh == p.H_kv) {
        kvh = 0;
        do {  // left > 0: a sequence with tiles follows
          s = seq_of(p, ++b);
        } while (s.tiles == 0 && b + 1 < p.batch.B);
      }
    }
    t = tile_of(p, s, tile);
    take = p.whole ? t.nt : min(t.nt, left);
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

// A V block with rows that no row of its tile sees, on its way into stage st.
struct Edge {
  int st = -1, n0 = 0, lo = 0, hi = 0, sinks = 0;
  bool copied = false;  // some of its pieces are loaded
};
// Zeroes those rows once the copies have landed and hands the stage over. Bit st of
// `parity` is that of the stage's next copies.
template <int D>
__device__ __forceinline__ bool finish_edge(const Ctx& c, Edge& e, uint32_t& parity,
                                            uint8_t* ring) {
  if (e.st < 0) return true;
  const int lane = threadIdx.x & 31;
  if (e.copied) {
    if (!wait_warp(c, BAR_V_EDGE + e.st, (parity >> e.st) & 1)) return false;
    parity ^= 1u << e.st;
  }
  for (int r = lane >> 3; r < kBn; r += 4) {  // 8 lanes a row
    const int key = e.n0 + r;
    if (key <= e.hi && (key >= e.lo || key < e.sinks)) continue;
#pragma unroll
    for (int cb = 0; cb < D / 64; ++cb)
      *reinterpret_cast<uint4*>(ring + e.st * Layout<D>::kTileBytes + cb * 16384 + r * 128 +
                                (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(bar_addr(c, BAR_V_FULL + e.st));
  e.st = -1;
  return true;
}

// Warp 0: Q of each tile and its K blocks; warp 2: the V blocks. Each ring waits
// for its own stages, in the order the tensor cores finish them. A V block whose
// rows are to be zeroed is finished behind the next block's request, so that its
// copies' latency does not leave the ring empty.
template <int D, bool IS_V>
__device__ void loader_role(const Ctx& c, const Params& p, const Part& part, uint8_t* smem,
                            uint32_t sbase, const CUtensorMap* tq, const CUtensorMap* tkv) {
  using L = Layout<D>;
  constexpr int kS = L::kStages;
  const int lane = threadIdx.x & 31;
  const int bar_full = IS_V ? BAR_V_FULL : BAR_K_FULL;
  const int bar_empty = IS_V ? BAR_V_EMPTY : BAR_K_EMPTY;
  const int ring = IS_V ? L::kV : L::kK;
  int g = 0, i = 0;  // blocks and tiles issued
  Edge edge;
  uint32_t edge_parity = 0;
  bool ok = true;
  Walk w;
  for (w.begin(p, part); ok && w.left > 0; w.next(p), ++i) {
    if (!IS_V) {
      const int qs = i % kS;
      if (i >= kS && !(ok = wait_warp(c, BAR_Q_EMPTY + qs, ((i / kS) - 1) & 1))) break;
      if (lane == 0) {
        if (p.batch.lengths[w.b] > p.cap) record_status(ATTN_ERR_PAGE);
        mbar_arrive_expect_tx(bar_addr(c, BAR_Q_FULL + qs), p.tokens * p.G * (D * 2));
        for (int cb = 0; cb < D / 64; ++cb)
          tma_load_4d(sbase + L::kQ + qs * L::kTileBytes + cb * 16384, tq,
                      bar_addr(c, BAR_Q_FULL + qs), 64 * cb, 0, w.kvh,
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
      const int st = g % kS;
      // with one stage the block before has to be finished first
      if (IS_V && kS == 1 && !(ok = finish_edge<D>(c, edge, edge_parity, smem + ring))) break;
      if (g >= kS && !(ok = wait_warp(c, bar_empty + st, ((g / kS) - 1) & 1))) break;
      const uint32_t dst = sbase + ring + st * L::kTileBytes;
      const int n0 = w.t.block(w.blk + t) * kBn;
      const bool cut = IS_V && (n0 + kBn - 1 > w.t.hi || (n0 < w.t.lo && n0 + kBn > w.t.sinks));
      if (!cut || x.needed != 0)
        load_pieces<D>(c, p, x, w.kvh, dst, tkv, cut ? BAR_V_EDGE + st : bar_full + st);
      if (IS_V) {
        if (!(ok = finish_edge<D>(c, edge, edge_parity, smem + ring))) break;
        if (cut) {
          edge.st = st;
          edge.n0 = n0;
          edge.lo = w.t.lo;
          edge.hi = w.t.hi;
          edge.sinks = w.t.sinks;
          edge.copied = x.needed != 0;
        }
      }
    }
  }
  if (IS_V && ok) ok = finish_edge<D>(c, edge, edge_parity, smem + ring);
  // When aborting, the copies in flight must land before the CTA exits (a phase
  // that was never begun ends the wait by its limit).
  if (!ok || *c.abort) {
    for (int st = 0; st < kS; ++st) {
      const int uses = (g + kS - st) / kS;  // blocks that went to this stage, or one more
      wait_drain(c, bar_full + st, (uses > 0 ? uses - 1 : 0) & 1);
      if (IS_V) wait_drain(c, BAR_V_EDGE + st, (edge_parity >> st) & 1);
      if (!IS_V) wait_drain(c, BAR_Q_FULL + st, (i / kS) & 1);
    }
  }
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
// softmax has written P(g).
template <typename T, int D>
__device__ void mma_role(const Ctx& c, const Params& p, const Part& part, uint32_t sbase,
                         uint32_t tmem) {
  using L = Layout<D>;
  constexpr int kS = L::kStages, kOB = L::kOBufs;
  const bool leader = elect_one_sync() != 0;
  constexpr uint32_t kIdS = idesc<T>(kBm, kBn, false);  // S = Q K^T
  constexpr uint32_t kIdO = idesc<T>(kBm, D, true);     // O += P V
  auto kmaj = [](int k) { return static_cast<uint32_t>(((k >> 2) * 16384 + (k & 3) * 32) >> 4); };
  auto mnmaj = [](int k) { return static_cast<uint32_t>((2048 * k) >> 4); };
  // S of block g of tile i; `first`, `last` of the tile's blocks
  auto issue_s = [&](int g, int i, bool first, bool last) -> bool {
    const int st = g % kS, qs = i % kS;
    if (first && !wait_warp(c, BAR_Q_FULL + qs, (i / kS) & 1)) return false;
    if (!wait_warp(c, BAR_K_FULL + st, (g / kS) & 1)) return false;
    tc_fence_after();
    if (leader) {
      const uint32_t q_lo = sdesc_lo(sbase + L::kQ + qs * L::kTileBytes, 16);
      const uint32_t k_lo = sdesc_lo(sbase + L::kK + st * L::kTileBytes, 16);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss(tmem + (g & 1) * 128, sdesc_from_lo(q_lo + kmaj(k)), sdesc_from_lo(k_lo + kmaj(k)),
               kIdS, k > 0);
      mma_commit(bar_addr(c, BAR_S_FULL + (g & 1)));
      mma_commit(bar_addr(c, BAR_K_EMPTY + st));
      if (last) mma_commit(bar_addr(c, BAR_Q_EMPTY + qs));
    }
    return true;
  };
  bool ok = true;
  Walk w;
  w.begin(p, part);
  if (w.left > 0) {
    int nt = w.take, next_nt = 0;
    ok = issue_s(0, 0, true, nt == 1);
    for (int g = 0, i = 0, t = 0; ok; ++g) {
      const bool last = t + 1 == nt;
      bool more = !last;
      if (last) {
        w.next(p);
        more = w.left > 0;
        next_nt = w.take;
      }
      const bool ahead = kS >= 2 || !last;
      if (more && ahead &&
          !(ok = issue_s(g + 1, last ? i + 1 : i, last, last ? next_nt == 1 : t + 2 == nt)))
        break;
      if (!(ok = wait_warp(c, BAR_P_FULL + (g & 1), (g >> 1) & 1))) break;
      const int vs = g % kS, ob = i % kOB;
      if (!(ok = wait_warp(c, BAR_V_FULL + vs, (g / kS) & 1))) break;
      if (t == 0 && i >= kOB && !(ok = wait_warp(c, BAR_O_FREE + ob, ((i / kOB) - 1) & 1)))
        break;
      tc_fence_after();
      if (leader) {
        const uint32_t v_mn = sdesc_lo(sbase + L::kV + vs * L::kTileBytes, 16384);
        // A = P (pairs in the S buffer of block g: keys 0-63 in columns 0-31,
        // keys 64-127 in columns 64-95, one half per softmax warpgroup)
#pragma unroll
        for (int k = 0; k < kBn / 16; ++k)
          mma_ts(tmem + 256 + ob * D, tmem + (g & 1) * 128 + 8 * k + (k >= 4 ? 32 : 0),
                 sdesc_from_lo(v_mn + mnmaj(k)), kIdO, (t > 0 || k > 0) ? 1u : 0u);
        mma_commit(bar_addr(c, BAR_O_DONE));
        mma_commit(bar_addr(c, BAR_V_EMPTY + vs));
        if (last) mma_commit(bar_addr(c, BAR_O_LAST));
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
    }
  }
  if (__any_sync(0xffffffffu, !ok || *c.abort != 0)) {
    // completion of everything issued before tensor memory is released
    if (leader) mma_commit(bar_addr(c, BAR_DRAIN));
    wait_drain(c, BAR_DRAIN, 0);
  }
  __syncwarp();
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

// P = 2^(x - shift) of 64 keys as 16-bit pairs into tensor-memory columns dst ..
// dst + 31; returns their sum (fp32, before rounding).
template <typename T, bool SOFTCAP>
__device__ __forceinline__ float chunk_p(const Params& p, const uint32_t (&raw)[64], uint32_t dst,
                                         bool masked, uint2 visible, float c_log2, float cap_in,
                                         float cap_out, float shift) {
  const uint64_t c2v = f2_make(SOFTCAP ? cap_in : c_log2, SOFTCAP ? cap_in : c_log2);
  const uint64_t out2 = f2_make(cap_out, cap_out);
  const float cap_u = SOFTCAP ? p.scale / p.softcap : 0.f;  // u = tau s / c
  const uint64_t cu2 = f2_make(cap_u, cap_u);
  const uint64_t nsh2 = f2_make(-shift, -shift);
  uint64_t sum2 = f2_make(0.f, 0.f);
  uint32_t packed[32];
  auto p_group = [&](auto fast_tag) {
    constexpr bool FAST = decltype(fast_tag)::value;
#pragma unroll
    for (int u = 0; u < 32; ++u) {
      const uint64_t s2 = f2_make(raw[2 * u], raw[2 * u + 1]);
      uint64_t y2;
      if (SOFTCAP) {
        const uint64_t th2 = FAST ? softcap::tanh_poly2(f2_mul(s2, cu2))
                                  : softcap::tanh_mufu2(f2_mul(s2, c2v));
        y2 = f2_fma(th2, out2, nsh2);
      } else {
        y2 = f2_fma(s2, c2v, nsh2);
      }
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
  if constexpr (SOFTCAP) {
    if (__all_sync(0xffffffffu, softcap::max_abs(raw) * cap_u <= softcap::kPolyMax))
      p_group(std::true_type{});
    else
      p_group(std::false_type{});
  } else {
    p_group(std::false_type{});
  }
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

// Thread r of each warpgroup owns row r; the warpgroups exchange the half-row
// maxima through shared memory once per block, so that both take the same shift.
// Warps without a row of the tile only keep the barriers' count.
template <typename T, int D, bool SOFTCAP>
__device__ void softmax_role(const Ctx& c, const Params& p, const Part& part, uint8_t* smem,
                             uint32_t tmem) {
  using L = Layout<D>;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int h = (warp - 4) >> 2;  // which half of the keys (and of O's columns)
  const int r = ((warp & 3) << 5) + lane;
  const int token = r / p.G;
  const uint32_t lane_base = static_cast<uint32_t>(r & ~31) << 16;
  float* xmax = reinterpret_cast<float*>(smem + L::kXchg);  // [block parity][half][row]
  float* xsum = xmax + 4 * 128;                              // [half][row]
  const float c_log2 = p.scale * kLog2e;
  const float cap_in = SOFTCAP ? 2.f * kLog2e * p.scale / p.softcap : 0.f;
  const float cap_out = SOFTCAP ? p.softcap * kLog2e : 0.f;
  bool ok = true;
  int g = 0;  // blocks of all tiles before
  int i = 0;
  Walk w;
  for (w.begin(p, part); ok && w.left > 0; w.next(p), ++i) {
    const int nt = w.take;
    const int ob = i % L::kOBufs;
    const uint32_t tO = tmem + lane_base + 256 + ob * D + h * (D / 2);
    const int rows = w.t.count * p.G;
    const bool idle = (r & ~31) >= rows;  // the warp has no row
    // the keys that this row sees, and those that every row of the tile sees
    const int pos = w.t.pos0 + token;
    const int hi = p.causal ? min(pos, w.s.length - 1) : w.s.length - 1;
    const int lo = p.left < 0 ? 0 : pos - p.left;
    const int all_hi = p.causal ? min(w.t.pos0, w.s.length - 1) : w.s.length - 1;
    const int all_lo = p.left < 0 ? 0 : w.t.pos0 + w.t.count - 1 - p.left;
    float m_used = -INFINITY, l = 0.f;
    for (int t = 0; t < nt; ++t) {
      const int gb = g + t;
      const int n0 = w.t.block(w.blk + t) * kBn;
      const int key0 = n0 + 64 * h;
      const uint32_t tS = tmem + lane_base + (gb & 1) * 128;
      const bool masked =
          n0 + kBn - 1 > all_hi || (n0 < all_lo && n0 + kBn > p.sinks);
      const bool got = wait(c, BAR_S_FULL + (gb & 1), (gb >> 1) & 1);
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
        float m_tile = -INFINITY;  // row maximum of the logits (log2 units) over this block
        if (smax > -INFINITY) {
          if (SOFTCAP) {
            const float ex = ex2_approx(smax * cap_in);
            m_tile = (1.f - 2.f * rcp_approx(ex + 1.f)) * cap_out;
          } else {
            m_tile = smax * c_log2;
          }
        }
        const bool need = m_tile > m_used + kRescale;
        if (__any_sync(0xffffffffu, need)) {
          const float m_new = need ? m_tile : m_used;
          const float f = need ? ex2_approx(m_used - m_new) : 1.f;  // 0 while m_used = -inf
          // this half of the O row, once P(t - 1) V has completed; a wait that
          // gives up is voted on at the next barrier
          if (__any_sync(0xffffffffu, need && m_used > -INFINITY) && t > 0) {
            if (!wait_warp(c, BAR_O_DONE, (gb - 1) & 1)) ok = false;
            if (ok) {
              tc_fence_after();
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
          }
          l *= f;
          m_used = m_new;
        }
        const float shift = m_used > -INFINITY ? m_used : 0.f;
        l += chunk_p<T, SOFTCAP>(p, raw, tS + 64 * h, masked, visible, c_log2, cap_in, cap_out,
                                 shift);
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_addr(c, BAR_P_FULL + (gb & 1)));  // one arrival per warp
    }
    // ---- epilogue, once the tile's last P V has completed (on a barrier of its
    // own, one phase per tile: both of the last phases of O_DONE may be behind)
    if (ok) ok = wait(c, BAR_O_LAST, i & 1);
    xsum[h * 128 + r] = l;
    if (!named_bar_and(kBarBoth, 256, ok)) break;
    tc_fence_after();
    const float lt = xsum[r] + xsum[128 + r];
    const bool whole = w.blk == 0 && nt == w.t.nt;
    if (!idle) {
      const bool mine = r < rows;
      if (whole) {
        const int head = w.kvh * p.G + r - token * p.G;
        const long long row = w.s.row0 + w.tile * p.tokens + token;
        T* out = static_cast<T*>(p.o) + row * p.o_token + head * p.o_head + h * (D / 2);
        const float inv = lt > 0.f ? 1.f / lt : 0.f;
        const uint64_t inv2 = f2_make(inv, inv);
#pragma unroll
        for (int c16 = 0; c16 < D / 32; ++c16) {
          uint32_t raw[16];
          tmem_ld16(tO + c16 * 16, raw);
          uint32_t packed[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint64_t v = f2_mul(f2_make(raw[2 * u], raw[2 * u + 1]), inv2);
            packed[u] = pack_pair<T>(f2_lo(v), f2_hi(v));
          }
          // a row that sees nothing: its P V was 0 times what V held
          if (!(lt > 0.f)) {
#pragma unroll
            for (int u = 0; u < 8; ++u) packed[u] = 0u;
          }
          if (mine) {
            uint4* to = reinterpret_cast<uint4*>(out + c16 * 16);
            to[0] = make_uint4(packed[0], packed[1], packed[2], packed[3]);
            to[1] = make_uint4(packed[4], packed[5], packed[6], packed[7]);
          }
        }
        if (mine && h == 0 && p.lse != nullptr)
          p.lse[row * p.H + head] = lt > 0.f ? (m_used + __log2f(lt)) * kLn2 : -INFINITY;
      } else {
        float* to = reinterpret_cast<float*>(p.workspace + kSharedBytes) +
                    (2LL * blockIdx.x + (w.blk == 0 ? 1 : 0)) * slot_floats(D);
        if (mine && h == 0) {
          to[r] = m_used;
          to[128 + r] = lt;
        }
        to += 256 + r * D + h * (D / 2);
#pragma unroll
        for (int c16 = 0; c16 < D / 32; ++c16) {
          uint32_t raw[16];
          tmem_ld16(tO + c16 * 16, raw);
          if (mine) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              reinterpret_cast<uint4*>(to + c16 * 16)[u] =
                  make_uint4(raw[4 * u], raw[4 * u + 1], raw[4 * u + 2], raw[4 * u + 3]);
          }
        }
      }
    }
    if (w.blk == 0 && nt < w.t.nt && threadIdx.x == 128) {
      // the tile goes on in the parts behind: the last of them holds its last block
      const long long end = part.first + part.count + (w.t.nt - nt);
      Shared s;
      s.parts = static_cast<int>((end - 1) / part.share) - static_cast<int>(blockIdx.x) + 1;
      s.row0 = w.s.row0 + w.tile * p.tokens;
      s.kvh = w.kvh;
      s.rows = rows;
      reinterpret_cast<Shared*>(p.workspace)[blockIdx.x] = s;
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_addr(c, BAR_O_FREE + ob));
    g += nt;
  }
}

// ------------------------------------------------------------------ kernels
template <typename T, int D, bool SOFTCAP>
__global__ void __launch_bounds__(kThreads, 1)
    cache_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
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
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // rows that no tile's copy fills hold zeros, not what shared memory held before
  const int unused = kBm - p.tokens * p.G;
  for (int i = threadIdx.x; i < L::kStages * (D / 64) * unused * 8; i += kThreads) {
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
      setmaxnreg_dec<kRegsCtl>();
      if (warp == 0)
        loader_role<D, false>(c, p, *part, smem, sbase, &tm_q, &tm_k);
      else if (warp == 1)
        mma_role<T, D>(c, p, *part, sbase, tmem);
      else if (warp == 2)
        loader_role<D, true>(c, p, *part, smem, sbase, &tm_q, &tm_v);
    } else {
      setmaxnreg_inc<kRegsSoftmax>();
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
// it: M = max m_i, L = sum l_i 2^(m_i - M), O = sum O_i 2^(m_i - M) / L, in the
// order of the parts. One warp a row, D / 32 columns a lane.
constexpr int kJoinWarps = 8, kJoinSplit = 128 / kJoinWarps;
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) cache_join_kernel(const Params p) {
  grid_dependency_wait();
  const Shared s = reinterpret_cast<const Shared*>(p.workspace)[blockIdx.x];
  const int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  if (s.parts == 0 || r >= s.rows) return;
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const float* slots = reinterpret_cast<const float*>(p.workspace + kSharedBytes) +
                       2LL * blockIdx.x * slot_floats(D);
  // part i of the tile: slot 1 of the first CTA, slot 0 of the ones behind
  auto slot = [&](int i) { return slots + (i == 0 ? 1 : 2 * i) * slot_floats(D); };
  constexpr int kAhead = 4;  // parts whose O is on its way before the weights are known
  float2 v[kAhead][E / 2];
  auto load = [&](int i, float2 (&to)[E / 2]) {
    const float* from = slot(i) + 256 + r * D + lane * E;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) to[e] = reinterpret_cast<const float2*>(from)[e];
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (i < s.parts) load(i, v[i]);
  float M = -INFINITY;
  for (int i = lane; i < s.parts; i += 32) M = fmaxf(M, slot(i)[r]);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float shift = M > -INFINITY ? M : 0.f;
  float2 o[E / 2];
  float total = 0.f;
#pragma unroll
  for (int e = 0; e < E / 2; ++e) o[e] = make_float2(0.f, 0.f);
  for (int i0 = 0; i0 < s.parts; i0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u;
      if (i >= s.parts) break;
      const float f = ex2_approx(slot(i)[r] - shift);
      if (f > 0.f) {  // a part that saw nothing holds no numbers
        total = fmaf(slot(i)[128 + r], f, total);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          o[e].x = fmaf(v[u][e].x, f, o[e].x);
          o[e].y = fmaf(v[u][e].y, f, o[e].y);
        }
      }
      if (i + kAhead < s.parts) load(i + kAhead, v[u]);
    }
  }
  const float inv = total > 0.f ? 1.f / total : 0.f;
  const int token = r / p.G, head = s.kvh * p.G + r - token * p.G;
  const long long row = s.row0 + token;
  T* out = static_cast<T*>(p.o) + row * p.o_token + head * p.o_head + lane * E;
#pragma unroll
  for (int e = 0; e < E / 2; ++e)
    reinterpret_cast<uint32_t*>(out)[e] = pack_pair<T>(o[e].x * inv, o[e].y * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[row * p.H + head] = total > 0.f ? (M + __log2f(total)) * kLn2 : -INFINITY;
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
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

struct Tensors {
  const void *q, *k, *v;
  long long q_in[2], k_in[3], v_in[3];
};

template <typename T, int D, bool SOFTCAP>
int launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const Params& p,
           int ctas, bool join, cudaStream_t stream) {
  auto kern = cache_fwd_kernel<T, D, SOFTCAP>;
  static std::atomic<bool> configured[kMaxTrackedDevices];
  if (!set_smem_limit_once(kern, Layout<D>::kBytes, configured)) return ATTN_ERR_LAUNCH;
  const int rc = launch_overlapped(kern, dim3(static_cast<unsigned>(ctas)), kThreads,
                                   Layout<D>::kBytes, 0, stream, tq, tk, tv, p);
  if (rc != ATTN_OK || !join) return rc;
  return launch_overlapped(cache_join_kernel<T, D>,
                           dim3(static_cast<unsigned>(ctas), kJoinSplit), 32 * kJoinWarps, 0, 0,
                           stream, p);
}

template <typename T>
int run(const Tensors& x, const Params& given, int d, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return ATTN_ERR_LAUNCH;
  CUtensorMap tq, tk, tv;
  const Batch& c = given.batch;
  const long long q_extent[3] = {given.G, given.H_kv, c.T};
  const long long q_stride[3] = {x.q_in[1], x.q_in[1] * given.G, x.q_in[0]};
  const long long extent[3] = {given.H_kv, c.page_size, c.n_pages};
  const long long k_stride[3] = {x.k_in[2], x.k_in[1], x.k_in[0]};
  const long long v_stride[3] = {x.v_in[2], x.v_in[1], x.v_in[0]};
  if (!encode_4d<T>(&tq, x.q, d, q_extent, q_stride, {given.G, 1, given.tokens}) ||
      !encode_4d<T>(&tk, x.k, d, extent, k_stride, {1, given.box, 1}) ||
      !encode_4d<T>(&tv, x.v, d, extent, v_stride, {1, given.box, 1}))
    return ATTN_ERR_LAUNCH;
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
    return cap ? launch<T, 64, true>(tq, tk, tv, p, ctas, join, stream)
               : launch<T, 64, false>(tq, tk, tv, p, ctas, join, stream);
  if (d == 128)
    return cap ? launch<T, 128, true>(tq, tk, tv, p, ctas, join, stream)
               : launch<T, 128, false>(tq, tk, tv, p, ctas, join, stream);
  return cap ? launch<T, 256, true>(tq, tk, tv, p, ctas, join, stream)
             : launch<T, 256, false>(tq, tk, tv, p, ctas, join, stream);
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
  p.causal = causal != 0;
  p.left = window_left > (1 << 30) ? 1 << 30 : window_left;
  p.sinks = sinks;
  return dtype == ATTN_BF16 ? cachefwd::run<__nv_bfloat16>(x, p, d, as_stream(stream))
                            : cachefwd::run<__half>(x, p, d, as_stream(stream));
}
