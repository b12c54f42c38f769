// paged_tc.cu -- attention of a chunk over the paged cache on tcgen05,
// CTA-pair (2-SM) form: bf16 queries, head_dim 256, pages in bf16 or e4m3.
//
// A cluster of two CTAs computes 256-row query tiles: 256 / G new tokens x the
// G query heads of one key/value head, 128 rows per CTA, against tiles of 128
// keys (cached tiles first, then the chunk's own).  Per key tile
//   S = Q K^T   tcgen05.mma.cta_group::2, M = 256: K split by keys (64 per CTA)
//   P           fp32 online softmax, two threads per row, P rounded to bf16 once
//   O += P V    tcgen05.mma.cta_group::2: V split by columns (128 per CTA)
// as in the dense kernel (tc_pair.cu).  What differs is how keys arrive and how
// the work is shared out.
//
// Loading, by two warps per CTA and operand into the 128-byte-swizzled layout:
//   bf16, tiles whose 128 keys are all seen by some query: TMA, one box of
//     min(page, 64) rows per page (all columns of the item at once from 64-token
//     pages on, else one 64-column block each), asynchronous to everything else.
//   Other tiles (the ragged last one, the window's edges, the chunk's own):
//     cp.async row by row, and zeros for rows past the length, outside the
//     window or of padding tokens, so that whatever a stale slot holds (NaN)
//     meets P = 0 as 0.  (Gathering every tile this way held a CTA to 11 bytes
//     a cycle, about 5700 cycles a tile.)
//   e4m3: raw rows by TMA into a staging half ahead of their use, then rebuilt as
//     bf16 by the loader warps, exactly, as the scale is a power of two: no
//     rounding beside the cache's own.  Chunks of four query tiles and more read
//     rows that cache.cu rebuilt once into the workspace (expanded_bytes).
//
// Work.  Unit = (sequence, kv head, query tile).  Lengths differ by sequence
// and live on the device, so each cluster derives the schedule itself from
// cache_lens: a nominal tile count per unit (its cached tiles in the window
// plus all chunk tiles).  If one unit per cluster and round leaves the clusters
// busy, units run whole; else the concatenation of all units' tiles is cut into
// equal ranges, one per cluster, and units that were cut leave fp32 partials
// that paged_combine_kernel merges by the log-sum-exp rule.  No atomics: the
// result does not depend on timing.
//
// Warp roles per CTA (512 threads):
//   warps 0..7   softmax, O correction, epilogue: warp w has the 32 rows of
//                TMEM quarter w % 4 and half w / 4 of the columns.  Two warps per
//                quarter keep the exponentials (1024 cycles of the special-
//                function units per tile) under the MMAs' time; each row's two
//                threads exchange their maxima through S's columns.
//   warps 8, 9   load Q and K;  warps 10, 11 load V
//   warp 12      TMEM allocation; QK issue (even CTA)
//   warp 13      PV issue (even CTA)
//   warp 14      scheduler: derives the segments this cluster runs and hands
//                them to the other warps through a two-entry ring
// TMEM per CTA (512 columns): O fp32 [0,256) | S0 [256,384) | S1 [384,512).
// Shared memory per CTA: Q 64 KB | K ring 2 x 32 KB | V ring 4 x 16 KB, or 2 and
// 32 KB of raw e4m3 rows | P 32 KB (also the output staging area) | control | codes
// of up to 512 chunk tokens (longer chunks: in the workspace).
// Every wait is bounded (DevCtl); counters that index barriers and ring slots
// run across segments.
//
// Measured: 512 tokens x 8 heads against four bf16 sequences of 15000 tokens 231 us
// (1144 TFLOP/s of 1655), against e4m3 ones 247 us (the rebuilding pass and fp32
// partials included); 51 tokens of 32 sequences of 816 tokens 27.6 us, the smallest
// call 12.4 us.  A tile takes about 4000 cycles where its MMAs need 2048: the
// softmax warps' chain (score read, maxima met across the pair of warps, 1024 cycles
// of exponentials, P stored) bounds it, the MMAs wait.
#include <cfloat>

#include "launch.h"
#include "paged.cuh"

namespace piattn {

namespace {

constexpr int kThreads = 512;
constexpr int kBM = 128;                    // query rows per CTA (256 per pair)
constexpr int kRowsTile = 2 * kBM;
constexpr int kBN = 128;                    // keys per key tile
constexpr int kD = 256;
constexpr int kQBlk = kBM * 128;            // [128 rows x 64 bf16]
constexpr int kQBytes = 4 * kQBlk;
constexpr int kKBlk = 64 * 128;             // [64 keys x 64 d]
constexpr int kKItem = 4 * kKBlk;           // this CTA's 64 keys x 256 d
constexpr int kVItem = 2 * kKBlk;           // 64 keys x this CTA's 128 columns
constexpr int kPBlk = kBM * 128;            // [128 rows x 64 keys]
constexpr int kPBytes = 2 * kPBlk;
constexpr int kOffQ = 0;
constexpr int kOffK = kQBytes;
constexpr int kNK = 2;                      // K ring slots
constexpr float kRescaleThreshold = 8.0f;   // log2 units: P stays <= 256
constexpr int kSmemLimit = 232448;

constexpr uint32_t kIdescQK = idesc_bf16_f32(2 * kBM, kBN, false, false);
constexpr uint32_t kIdescPV = idesc_bf16_f32(2 * kBM, kD, false, true);
constexpr uint32_t kColO = 0, kColS = 256;
constexpr int kGroup = kPagedTcGroup;
constexpr int kSegs = 2;                     // segment ring
constexpr int kSegUsers = 14;                // warps that read it


// A run of key tiles of one unit on this cluster.
struct Segment {
  int b, g, tile;            // sequence (absolute), kv head, query tile
  int tq0, tq1;              // its first / last new token
  int len;                   // cached tokens
  int lo0, lo1;              // window start (cached positions) of the first token that is
                             // not padding / of the last
  int sink_tiles, win_tile;  // cached tiles [0, sink_tiles) and [win_tile, ...)
  int n_cached, c0;          // number of cached tiles; first chunk tile
  int it0, n;                // this run: tiles [it0, it0 + n) of the unit's list
  int slot;                  // partial slot, -1: the unit runs whole here
  uint32_t csq0, csq1;       // block index of the first / last token
  int any_e;                 // an expert among the tokens
};

// bf16 pages: four V halves.  e4m3: two, and as much room for raw rows: each loader
// warp has two pieces, K of 16 keys x 256 bytes, V of 32 keys x 128 bytes.
constexpr int kRawPiece = 4096;
template <bool kE4M3>
struct Layout {
  static constexpr int kNV = kE4M3 ? 2 : 4;
  static constexpr int kOffV = kOffK + kNK * kKItem;
  static constexpr int kOffRaw = kOffV + kNV * kVItem;
  static constexpr int kOffP = kOffRaw + (kE4M3 ? 8 * kRawPiece : 0);
  static constexpr int kOffCtl = kOffP + kPBytes;
};
constexpr int kTiles = (kMaxTokens + kBN - 1) / kBN;
// What a chunk tile holds (tile_fast; a padding token is FAST too).
constexpr uint32_t kTileFast = 1u, kTilePad = 2u;
// Codes of longer chunks live in the workspace (one copy per CTA).
constexpr int kSmemTokens = 512;

// The schedule's inputs: nominal tiles before each sequence's units, lengths.
struct Plan {
  int cum[kGroup + 1];
  int len[kGroup];
  int max_nom;
};

template <class L>
struct __align__(8) Smem {
  uint64_t q_full, q_empty;
  uint64_t k_full[kNK], k_empty[kNK];
  uint64_t v_full[L::kNV], v_empty[L::kNV];
  uint64_t s_full[2], s_free[2];
  uint64_t p_full, o_done, o_free;
  uint64_t drain_qk, drain_pv;
  uint64_t pair[4];                 // a quarter's two warps meet
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t raw_full[8];             // e4m3: the loader warps' raw pieces
  uint32_t tmem_base;
  int abort;
  Plan plan;
  Segment seg[kSegs];
  uint16_t tile_cs_first[kTiles];
  uint16_t tile_cs_last[kTiles];
  uint8_t tile_fast[kTiles];
};

template <class L>
__host__ __device__ constexpr int off_codes() {
  return L::kOffCtl + ((int)sizeof(Smem<L>) + 127) / 128 * 128;
}
__host__ __device__ constexpr int pad_tokens(int n) { return (n + 127) / 128 * 128; }
template <class L>
__host__ __device__ constexpr int layout_bytes() {
  return off_codes<L>() + kSmemTokens * 2;
}
static_assert(layout_bytes<Layout<false>>() <= kSmemLimit, "layout too large");
static_assert(layout_bytes<Layout<true>>() <= kSmemLimit, "layout too large");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Code size matters in this kernel: a dozen warps in seven roles share the
// instruction caches, and with everything inlined and unrolled each role's loop
// waited for its own instructions (a third of all stalls, and 1.6 times the
// time with e4m3 pages).  What is rare or long is out of line.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int* abort, int* status,
                                       unsigned long long limit) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*(volatile int*)abort) return false;
    if ((unsigned long long)(clock64() - t0) > limit) {
      atomicCAS(status, 0, kStatusTimeout);
      *(volatile int*)abort = 1;
      return false;
    }
  }
  return true;
}

// After a wait ran out in either CTA, when neither starts anything more.  A loader
// that was ahead of its partner has copies under way whose barrier, in the even CTA,
// lacks the partner's arrivals and never completes: no wait covers them.  They come
// from this GPU's own memory, within microseconds; this is about half a millisecond.
__device__ __noinline__ void settle() {
  const long long t0 = clock64();
  while (clock64() - t0 < (1ll << 20)) __nanosleep(1000);
}

// Warp-uniform bounded wait: every lane polls, all get the same answer.
template <class SmemT>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, SmemT& sm,
                                          const DevCtl& ctl) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_slow(bar, parity, &sm.abort, ctl.status, ctl.wait_limit));
}

// ------------------------------------------------------------ the schedule

// Nominal key tiles of each unit of a sequence with n cached tokens: an upper
// bound over its query tiles, at least 1.
__device__ __forceinline__ int nominal_tiles(const PagedTcParams& p, int n) {
  int t = (n + kBN - 1) / kBN;
  if (p.window > 0) {
    const long long w = ((long long)p.window + p.tok_per_tile + kBN - 1) / kBN + 1 +
                        ((long long)p.sinks + kBN - 1) / kBN;
    t = (int)min((long long)t, w);
  }
  return t + (p.Sq + kBN - 1) / kBN;
}

// Warp-collective: the plan of this launch's sequences, from cache_lens.  (The
// host keeps the total below 2^31 by the size of a group.)
__device__ __forceinline__ void make_plan(const PagedTcParams& p, const DevCtl& ctl, Plan& plan,
                                          int lane) {
  const int units = p.Hkv * p.n_tiles;
  int carry = 0, top = 0;
  bool bad = false;
  for (int base = 0; base < p.nb; base += 32) {
    const int b = base + lane;
    int nom = 0, n = 0;
    if (b < p.nb) {
      n = cached_len(p.lens, p.b0 + b, p.max_pages, p.page_shift, bad);
      nom = nominal_tiles(p, n);
    }
    top = max(top, nom);
    int x = units * nom;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (b < p.nb) {
      plan.cum[b + 1] = carry + x;
      plan.len[b] = n;
    }
    carry += __shfl_sync(0xffffffffu, x, 31);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (lane == 0) {
    plan.cum[0] = 0;
    plan.max_nom = top;
  }
  if (bad && blockIdx.x == 0) record_status(ctl, kStatusArg);
  __syncwarp();
}

// Tiles per cluster when the tiles are cut into equal ranges; 0: units run
// whole, unit u on cluster u % n_clusters.  A cut costs a cluster about five
// tiles' time (partials written and merged: measured against whole units at 32
// sequences of 816 + 51 tokens), so units stay whole unless cutting saves that.
__device__ __forceinline__ int tiles_per_cluster(const PagedTcParams& p, const Plan& plan) {
  if (!p.may_cut) return 0;
  const int n_units = p.nb * p.Hkv * p.n_tiles;
  const int per = max((plan.cum[p.nb] + p.n_clusters - 1) / p.n_clusters, 2);
  const int rounds = (n_units + p.n_clusters - 1) / p.n_clusters;
  return (long long)rounds * plan.max_nom <= per + 5 ? 0 : per;
}

// The next segment's place in the schedule: unit (b, g, tile) and the nominal
// range [s0, s1) of its nom tiles.  pos: a tile of the cluster's range, or with
// per == 0 a unit.  Returns the position after it.
struct Place {
  int b, g, tile, slot, s0, s1, nom;
};
__device__ __forceinline__ int next_place(const PagedTcParams& p, const Plan& plan, int per,
                                          int pos, int end, Place& x) {
  const int units = p.Hkv * p.n_tiles;
  int b, u;
  if (per == 0) {
    b = pos / units;
    u = pos - b * units;
    x.nom = (plan.cum[b + 1] - plan.cum[b]) / units;
    x.s0 = 0;
    x.s1 = x.nom;
    x.slot = -1;
    pos += p.n_clusters;
  } else {
    int lo = 0, hi = p.nb - 1;               // largest b with cum[b] <= pos
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (plan.cum[mid] <= pos) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    x.nom = (plan.cum[b + 1] - plan.cum[b]) / units;
    const int rem = pos - plan.cum[b];
    u = rem / x.nom;
    x.s0 = rem - u * x.nom;
    x.s1 = min(x.nom, x.s0 + (end - pos));
    // A run that begins mid-unit is its cluster's first: slot 0, else slot 1.
    x.slot = x.s0 == 0 && x.s1 == x.nom ? -1 : (pos / per) * 2 + (x.s0 > 0 ? 0 : 1);
    pos += x.s1 - x.s0;
  }
  x.b = b;
  x.g = u / p.n_tiles;
  x.tile = u - x.g * p.n_tiles;
  return pos;
}

__device__ __forceinline__ int window_lo(const PagedTcParams& p, int len, int i) {
  return p.window <= 0 ? 0 : min(max(len + i - p.window + 1, 0), len);
}

// Warp-collective: what the unit's query tokens see, and this run's part of
// its tile list: the cached tiles that hold a key inside the window or a sink,
// then the chunk's tiles from the window's first to the last whose first key
// the last token's block admits.  (FAST and padding holes are masked per
// element.)  A unit of padding rows has no tile.
template <class SmemT>
__device__ __forceinline__ void fill_segment(const PagedTcParams& p, const SmemT& sm,
                                          const uint16_t* codes, const Place& pl, Segment& out,
                                          int lane) {
  Segment x;
  x.b = p.b0 + pl.b;
  x.g = pl.g;
  x.tile = pl.tile;
  x.slot = pl.slot;
  x.tq0 = x.tile * p.tok_per_tile;
  x.tq1 = min(x.tq0 + p.tok_per_tile, p.Sq) - 1;
  x.len = sm.plan.len[pl.b];
  int any_e = 0;
  uint32_t first = ~0u;                      // first token that is not padding
  for (int t = x.tq0 + lane; t <= x.tq1; t += 32) {
    const uint32_t c = codes[t];
    any_e |= (c >> 1) & 1;
    if (!is_pad(c)) first = min(first, (uint32_t)t);
  }
  x.any_e = __any_sync(0xffffffffu, any_e);
  first = __reduce_min_sync(0xffffffffu, first);
  const bool live = first != ~0u;
  x.csq0 = codes[x.tq0] >> 2;
  x.csq1 = codes[x.tq1] >> 2;
  x.lo0 = window_lo(p, x.len, live ? (int)first : x.tq0);
  x.lo1 = window_lo(p, x.len, x.tq1);
  const int n_ct = (x.len + kBN - 1) / kBN;
  x.sink_tiles = p.window > 0 ? (min(p.sinks, x.lo0) + kBN - 1) / kBN : 0;
  x.win_tile = max(x.lo0 / kBN, x.sink_tiles);
  x.n_cached = x.sink_tiles + max(n_ct - x.win_tile, 0);
  x.c0 = 0;
  if (p.window > 0 && x.len >= p.sinks) x.c0 = max(x.tq0 - p.window + 1, 0) / kBN;
  const int n_chunk = (p.Sq + kBN - 1) / kBN;
  int c1 = 0;                                // chunk tiles whose first key is admitted
  for (int t0 = 0; t0 < n_chunk; t0 += 32) {
    const unsigned m = __ballot_sync(0xffffffffu,
                                     t0 + lane < n_chunk && sm.tile_cs_first[t0 + lane] <= x.csq1);
    c1 += __popc(m);
  }
  const int total = live ? x.n_cached + max(c1 - x.c0, 0) : 0;
  x.it0 = (int)((long long)pl.s0 * total / pl.nom);
  x.n = (int)((long long)pl.s1 * total / pl.nom) - x.it0;
  if (lane == 0) out = x;
}

struct KeyTile {
  int tile;
  bool chunk;
};
__device__ __forceinline__ KeyTile key_tile(const Segment& x, int idx) {
  if (idx >= x.n_cached) return {x.c0 + idx - x.n_cached, true};
  return {idx < x.sink_tiles ? idx : x.win_tile + idx - x.sink_tiles, false};
}
// Whether every key of a cached tile is seen by some query of the segment.
__device__ __forceinline__ bool whole_tile(const PagedTcParams& p, const Segment& x,
                                           const KeyTile& kt) {
  const int k0 = kt.tile * kBN;
  return !kt.chunk && k0 + kBN <= x.len && (p.window <= 0 || k0 >= x.lo0 || k0 + kBN <= p.sinks);
}

// Warp-collective: the codes of sequence b's chunk and each tile's summary, a
// tile of 128 tokens at a time.  (A short loop: its code is fetched cold by
// every call, and the whole kernel waits for it.)
template <class SmemT>
__device__ __forceinline__ void scan_codes(const PagedTcParams& p, SmemT& sm, uint16_t* codes,
                                           int b, int lane) {
  const uint8_t* ar = p.ar + (long long)b * p.mask_bs;
  const int32_t* seg = p.seg ? p.seg + (long long)b * p.mask_bs : nullptr;
  uint32_t cs = 0;
#pragma unroll 1
  for (int t0 = 0; t0 < p.Sq; t0 += kBN) {
    uint32_t on[4];
    int sg[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 32 * i + lane;
      on[i] = t < p.Sq ? ar[t] : 0u;
      sg[i] = t < p.Sq && seg ? seg[t] : 0;
    }
    uint32_t any_f = 0, any_p = 0;
    uint32_t first = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 32 * i + lane;
      const uint32_t m = __ballot_sync(0xffffffffu, on[i] != 0u);
      const uint32_t code =
          t < p.Sq ? make_code(cs + __popc(m & (0xffffffffu >> (31 - lane))), sg[i]) : 0xFFFFu;
      codes[t] = (uint16_t)code;
      if (i == 0) first = cs + (m & 1u);
      cs += __popc(m);
      const uint32_t live = __ballot_sync(0xffffffffu, t < p.Sq);
      const uint32_t f = __ballot_sync(0xffffffffu, (code & 1u) != 0u) & live;
      const uint32_t q = __ballot_sync(0xffffffffu, is_pad(code)) & live;
      any_f |= f;
      any_p |= q;
    }
    if (lane == 0) {
      sm.tile_cs_first[t0 / kBN] = (uint16_t)first;
      sm.tile_cs_last[t0 / kBN] = (uint16_t)cs;
      sm.tile_fast[t0 / kBN] = (uint8_t)((any_f ? kTileFast : 0u) | (any_p ? kTilePad : 0u));
    }
  }
  __syncwarp();
}

// Which of the 64 keys from tile offset 64 * half a query row sees, one bit
// each.  tok: the row's token (its code cq).
__device__ __noinline__ uint2 row_mask(const PagedTcParams& p, const uint16_t* codes,
                                       const Segment& x, bool chunk, int h0, int tok, uint32_t cq) {
  const int lane = threadIdx.x & 31;
  uint32_t vm[2] = {~0u, ~0u};
  int a, e, s;                               // visible: [a, e) and [0, s) from h0
  if (chunk) {
    e = 0;                                   // keys whose block the row admits: a prefix
#pragma unroll 1
    for (int step = 64; step >= 1; step >>= 1) {
      const int probe = e + step;
      if (probe <= 64 && (uint32_t)(codes[h0 + probe - 1] >> 2) <= (cq >> 2)) e = probe;
    }
    e = min(e, p.Sq - h0);
    a = p.window > 0 ? tok - p.window + 1 - h0 : 0;
    s = p.window > 0 ? min(max(p.sinks - x.len, 0) - h0, e) : 0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      // FAST bit (padding keys carry it too) and padding, per key
      const uint32_t ck = codes[h0 + 32 * w + lane];
      const uint32_t fw = __ballot_sync(0xffffffffu, (ck & 1u) != 0u);
      const uint32_t pw = __ballot_sync(0xffffffffu, is_pad(ck));
      vm[w] = ~((cq & 2u) ? fw : pw);
    }
  } else {
    e = x.len - h0;
    a = window_lo(p, x.len, tok) - h0;       // below: sinks only
    s = p.window > 0 ? min(p.sinks, x.len) - h0 : 0;
  }
#pragma unroll
  for (int w = 0; w < 2; ++w)
    vm[w] &= (bits_below(e - 32 * w) & ~bits_below(a - 32 * w)) | bits_below(s - 32 * w);
  return make_uint2(vm[0], vm[1]);
}

// ------------------------------------------------------------- the loaders

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  // src-size 0 writes zeros and reads nothing
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Cached position x: the page id that holds it, kNoRow if no query of the
// segment sees it.  Loaded a tile before row_of() uses it.
constexpr int kNoRow = -2147483647 - 1;
__device__ __forceinline__ int page_of(const PagedTcParams& p, const Segment& s, int x) {
  if (x >= s.len || (p.window > 0 && x < s.lo0 && x >= p.sinks)) return kNoRow;
  if (p.in_order) return s.b * p.max_pages + (x >> p.page_shift);
  return p.table[(long long)s.b * p.max_pages + (x >> p.page_shift)];
}
// Whether some query of the segment sees cached position x.
__device__ __forceinline__ bool row_seen(const PagedTcParams& p, const Segment& s, int x) {
  return x < s.len && (p.window <= 0 || x >= s.lo0 || x < p.sinks);
}
// The page id at x if some query sees a row of that page inside x's tile (the
// table may hold anything for others).
__device__ __forceinline__ int page_seen(const PagedTcParams& p, const Segment& s, int x) {
  const int w = min(1 << p.page_shift, kBN), x0 = x & -w;
  if (x0 >= s.len || (p.window > 0 && x0 + w <= s.lo0 && x0 >= p.sinks)) return kNoRow;
  return p.table[(long long)s.b * p.max_pages + (x0 >> p.page_shift)];
}
// Its slot; -1 if there is none (a page id out of range is noted in bad).
__device__ __forceinline__ int slot_of(const PagedTcParams& p, int x, int page, bool& bad) {
  if (page >= 0 && page < p.num_pages)
    return (page << p.page_shift) + (x & ((1 << p.page_shift) - 1));
  bad = bad || page != kNoRow;
  return -1;
}

// The row of chunk key j in [B * Sq], -1 if it is padding, out of the chunk or
// hidden from every query of the segment.
__device__ __forceinline__ int chunk_row(const PagedTcParams& p, const Segment& s,
                                         const uint16_t* codes, int j) {
  if (j >= p.Sq) return -1;
  const uint32_t c = codes[j];
  if (is_pad(c) || (c >> 2) > s.csq1 || !in_window(s.len, s.tq0, j, p.window, p.sinks)) return -1;
  return s.b * p.Sq + j;
}

// n rows of an item by cp.async, zeros where there is none: row row0 + i * step
// is row __shfl(mine, lane0 + i * lane_step) of the tensor at base.
__device__ __noinline__ void copy_rows(int mine, const uint8_t* base, uint32_t pitch, uint32_t dst,
                                       int n, int row0, int step, int lane0, int lane_step) {
  const int c = threadIdx.x & 7;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 8) {
    int r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = __shfl_sync(0xffffffffu, mine, lane0 + (i0 + i) * lane_step);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = row0 + (i0 + i) * step;
      cp_async16(dst + row * 128 + ((c ^ (row & 7)) << 4),
                 base + (unsigned long long)(uint32_t)max(r[i], 0) * pitch, r[i] >= 0);
    }
  }
}

// Where a lane's first 16 bytes lie in a raw piece: rows of 256 bytes (two a pass) or
// 128 bytes (four a pass); a pass is 512 bytes.
__device__ __forceinline__ uint32_t lane_src(int rows, int sub, int c16) {
  return (uint32_t)(sub * (512 / rows) + c16 * 16);
}
// Multiplies the eight rebuilt pieces of a lane (see rebuild) by rest_scale.
__device__ __noinline__ void rescale_rows(uint32_t base, int rows, uint32_t cs, int l0, uint32_t e) {
  const uint32_t m = rest_scale(e);
#pragma unroll 1
  for (int it = 0; it < 8; ++it) {
    const uint32_t r = __shfl_sync(0xffffffffu, m, l0 + it * rows);
    const uint32_t a0 = base + it * rows * 128 + ((cs ^ ((it * rows) & 7)) << 4);
    for (int k = 0; k < 2; ++k) {
      uint4 w = ld_shared_v4(a0 ^ (16 * k));
      w = make_uint4(mul_bf16x2(w.x, r), mul_bf16x2(w.y, r), mul_bf16x2(w.z, r), mul_bf16x2(w.w, r));
      st_shared_v4(a0 ^ (16 * k), w);
    }
  }
  __syncwarp();
}
// The exponent byte of row r, loaded by the lane that looked the row up.
__device__ __forceinline__ uint32_t row_exp(const PagedTcParams& p, const uint8_t* exps, int r, int g) {
  return r >= 0 ? (uint32_t)__ldg(exps + (unsigned long long)(uint32_t)r * (uint32_t)p.Hkv + g) : kNoExp;
}

template <bool kE4M3>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedTcParams p, const DevCtl ctl) {
  using L = Layout<kE4M3>;
  using SmemT = Smem<L>;
  constexpr int kNV = L::kNV;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // Both CTAs see the same base offset, so both leave here or neither does.
  if ((int)(smem - smem_raw) + layout_bytes<L>() > p.smem_bytes) {
    pdl_wait();
    if (threadIdx.x == 0) record_status(ctl, kStatusUnsupported);
    return;
  }
  SmemT& sm = *reinterpret_cast<SmemT*>(smem + L::kOffCtl);
  uint16_t* codes = p.Sq <= kSmemTokens
                        ? reinterpret_cast<uint16_t*>(smem + off_codes<L>())
                        : p.codes + (long long)blockIdx.x * pad_tokens(p.Sq);
  uint8_t* sQ = smem + kOffQ;
  uint8_t* kring = smem + kOffK;
  uint8_t* vring = smem + L::kOffV;
  uint8_t* sP = smem + L::kOffP;

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cluster = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 4);
    mbar_init(&sm.q_empty, 1);
    for (int s = 0; s < kNK; ++s) {
      mbar_init(&sm.k_full[s], 4);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kNV; ++s) {
      mbar_init(&sm.v_full[s], 4);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.s_free[s], 16);
    }
    mbar_init(&sm.p_full, 16);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.o_free, 16);
    mbar_init(&sm.drain_qk, 1);
    mbar_init(&sm.drain_pv, 1);
    for (int s = 0; s < 4; ++s) mbar_init(&sm.pair[s], 2);
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(&sm.seg_full[s], 1);
      mbar_init(&sm.seg_empty[s], kSegUsers);
    }
    for (int s = 0; s < 8; ++s) mbar_init(&sm.raw_full[s], 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  cluster_sync();                             // both CTAs' barriers exist
  if (warp == 12) {
    tmem_alloc_pair(&sm.tmem_base, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_launch_dependents();

  // Every other warp takes the scheduler's segments in order; null at the end
  // (or after a failure).
  bool ok = true;
  uint32_t n_seg = 0;
  auto next_segment = [&]() -> const Segment* {
    if (n_seg > 0) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.seg_empty[(n_seg - 1) % kSegs]);
    }
    const int i = (int)(n_seg % kSegs);
    if (!ok || !warp_wait(&sm.seg_full[i], (n_seg / kSegs) & 1, sm, ctl)) return nullptr;
    ++n_seg;
    return sm.seg[i].n < 0 ? nullptr : &sm.seg[i];
  };

  const uint32_t tmem = sm.tmem_base;
  const uint32_t tO = tmem + kColO, tS = tmem + kColS;      // S[b] at +128 b

  if (warp >= 12) {
    auto commit_both = [&](uint64_t* bar) {
      umma_commit_pair(mapa_shared(smem_u32(bar), 0));
      umma_commit_pair(mapa_shared(smem_u32(bar), 1));
    };
    uint32_t gt = 0, nu = 0;      // key tiles and segments processed
    if (warp == 12) {
      const uint64_t qdesc0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t kdesc0 = sdesc_sw128(smem_u32(kring), 16, 1024);
      while (const Segment* px = next_segment()) {
        const Segment& x = *px;
        if (!leader || x.n == 0) continue;
        ok = warp_wait(&sm.q_full, nu & 1, sm, ctl);
        ++nu;
        for (int j = 0; j < x.n && ok; ++j, ++gt) {
          const int s = (int)(gt % kNK);
          ok = warp_wait(&sm.k_full[s], (gt / kNK) & 1, sm, ctl);
          // S[gt % 2] was last read by the softmax of tile gt - 2.
          if (ok && gt >= 2) ok = warp_wait(&sm.s_free[gt & 1], ((gt - 2) >> 1) & 1, sm, ctl);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t kd = kdesc0 + (uint64_t)((s * kKItem) >> 4);
#pragma unroll 4
            for (int kk = 0; kk < kD / 16; ++kk) {
              const uint32_t qoff = (uint32_t)((kk >> 2) * kQBlk + (kk & 3) * 32);
              const uint32_t koff = (uint32_t)((kk >> 2) * kKBlk + (kk & 3) * 32);
              umma_pair_ss(tS + 128 * (gt & 1), qdesc0 + (uint64_t)(qoff >> 4),
                           kd + (uint64_t)(koff >> 4), kIdescQK, kk > 0 ? 1u : 0u);
            }
            commit_both(&sm.k_empty[s]);
            commit_both(&sm.s_full[gt & 1]);
            if (j == x.n - 1) commit_both(&sm.q_empty);
          }
          __syncwarp();
        }
      }
      if (leader) {
        if (lane == 0) umma_commit_pair(smem_u32(&sm.drain_qk));
        __syncwarp();
        (void)mbar_wait(&sm.drain_qk, 0, ctl);
      }
    } else if (warp == 13) {
      const uint64_t pdesc0 = sdesc_sw128(smem_u32(sP), 16, 1024);
      const uint64_t vdesc0 = sdesc_sw128(smem_u32(vring), kKBlk, 1024);
      uint32_t uv = 0;
      while (const Segment* px = next_segment()) {
        const Segment& x = *px;
        if (!leader || x.n == 0) continue;
        ++nu;
        for (int j = 0; j < x.n && ok; ++j, ++gt) {
          // V arrives before P: wait for it first, off the critical path.
          ok = warp_wait(&sm.v_full[uv % kNV], (uv / kNV) & 1, sm, ctl) &&
               warp_wait(&sm.p_full, gt & 1, sm, ctl);
          // The first PV overwrites O: the previous epilogue must have read it.
          if (ok && j == 0 && nu > 1) ok = warp_wait(&sm.o_free, (nu - 2) & 1, sm, ctl);
          for (int h = 0; h < 2 && ok; ++h) {
            const int s = (int)(uv % kNV);
            if (h == 1) ok = warp_wait(&sm.v_full[s], (uv / kNV) & 1, sm, ctl);
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
              const uint64_t vd = vdesc0 + (uint64_t)((s * kVItem) >> 4);
#pragma unroll
              for (int k4 = 0; k4 < 4; ++k4) {
                const uint32_t poff = (uint32_t)(h * kPBlk + k4 * 32);
                umma_pair_ss(tO, pdesc0 + (uint64_t)(poff >> 4), vd + (uint64_t)((k4 * 2048) >> 4),
                             kIdescPV, (j > 0 || h > 0 || k4 > 0) ? 1u : 0u);
              }
              commit_both(&sm.v_empty[s]);
              if (h == 1) commit_both(&sm.o_done);
            }
            __syncwarp();
            ++uv;
          }
        }
      }
      if (leader) {
        if (lane == 0) umma_commit_pair(smem_u32(&sm.drain_pv));
        __syncwarp();
        (void)mbar_wait(&sm.drain_pv, 0, ctl);
      }
    } else if (warp == 14) {
      // ------------------------------------------------------ scheduler
      if (p.mask_bs == 0) scan_codes(p, sm, codes, 0, lane);
      make_plan(p, ctl, sm.plan, lane);
      const int per = tiles_per_cluster(p, sm.plan);
      const int step = per == 0 ? p.nb * p.Hkv * p.n_tiles : sm.plan.cum[p.nb];
      int pos = per == 0 ? cluster : min((int)min((long long)cluster * per, (long long)step), step);
      const int end = per == 0 ? step : (int)min((long long)pos + per, (long long)step);
      int codes_b = -1;
      // A ring entry is free once the users of the segment kSegs back are done.
      auto released = [&](uint32_t k) {      // segment k's entry, by its users
        return warp_wait(&sm.seg_empty[k % kSegs], (k / kSegs) & 1, sm, ctl);
      };
      for (;;) {
        if (n_seg >= kSegs && !released(n_seg - kSegs)) break;
        Segment& out = sm.seg[n_seg % kSegs];
        const bool done = pos >= end;
        if (done) {
          if (lane == 0) out.n = -1;
        } else {
          Place pl;
          pos = next_place(p, sm.plan, per, pos, end, pl);
          if (p.mask_bs != 0 && pl.b != codes_b) {
            // Nobody may still read the old codes.
            if (n_seg > 0 && !released(n_seg - 1)) break;
            scan_codes(p, sm, codes, p.b0 + pl.b, lane);
            codes_b = pl.b;
          }
          fill_segment(p, sm, codes, pl, out, lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.seg_full[n_seg % kSegs]);
        ++n_seg;
        if (done) break;
      }
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------- loaders
    // Warps 8 and 9 bring Q and K, warps 10 and 11 V: a warp that waits for its
    // copies to land must not hold back the other operand's.
    const int lw = warp & 1;
    Segment x;                                // the current segment, in registers
    x.it0 = x.n = 0;
    bool bad = false;
    // Full barriers (even CTA) of the cp.async items in flight, oldest first.
    uint32_t pend0 = 0, pend1 = 0;
    int n_pend = 0;
    auto signal = [&](uint32_t bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(bar);
    };
    auto flush = [&]() {                      // every item in flight lands and is announced
      cp_wait<0>();
      if (n_pend > 0) signal(pend0);
      if (n_pend > 1) signal(pend1);
      n_pend = 0;
    };
    auto push = [&](uint32_t bar) {
      cp_commit();
      if (n_pend == 2) {
        cp_wait<2>();
        signal(pend0);
        pend0 = pend1;
        pend1 = bar;
      } else {
        (n_pend == 0 ? pend0 : pend1) = bar;
        ++n_pend;
      }
    };
    // A slot that is not free yet may wait for an item not announced yet.
    auto acquire = [&](uint64_t* bar, uint32_t use) -> bool {   // use: earlier fills of the slot
      if (use == 0) return true;
      const uint32_t parity = (use - 1) & 1;
      if (n_pend > 0) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        flush();
      }
      return warp_wait(bar, parity, sm, ctl);
    };
    // Waits (bounded) for the last phase of a ring's full barriers, so that no
    // copy into either CTA is in flight when the cluster leaves; phases that the
    // consumer has waited for return at once.
    auto land = [&](uint64_t* full, int slots, uint32_t used) {
      flush();
      if (leader && lw == 0 && lane == 0)
        for (int s = 0; s < slots; ++s) {
          const uint32_t n = used > (uint32_t)s ? (used - (uint32_t)s + slots - 1) / slots : 0;
          if (n > 0) (void)mbar_wait(&full[s], (n - 1) & 1, ctl);
        }
      __syncwarp();
    };
    auto bar_full = [&](uint64_t* bar) { return mapa_shared(smem_u32(bar), 0); };

    // Row lookup: lane l looks up the l-th of the 32 rows (of 64) that this warp
    // copies of an item; rows of 512 bytes take all 32 lanes, of 256 bytes 16
    // lanes.  (e4m3: rows 32 lw + l.)  Page ids are loaded a tile ahead (peek), so
    // that their latency does not delay the copies.
    const int row32 = lane * 2 + lw;                               // 32 lanes per row
    const int row16 = (lane >> 1) * 4 + lw * 2 + (lane & 1);       // 16
    // TMA tiles: lane l has the page of box l.
    const int box = min(1 << p.page_shift, 64);                    // rows per box
    const int boxes = 64 / box;                                    // per 64 keys
    auto peek = [&](int idx, int row, int tma_row) -> int {
      if (idx >= x.it0 + x.n) return kNoRow;
      const KeyTile kt = key_tile(x, idx);
      if (kt.chunk) return kNoRow;
      const int at = kt.tile * kBN;
      if (kE4M3) return page_seen(p, x, at + row);
      const bool tma = p.use_tma && whole_tile(p, x, kt);
      return page_of(p, x, at + (tma ? tma_row : row));
    };
    // e4m3.  A warp copies (TMA) and rebuilds rows of its own, 32 of K or of a V half
    // item, in two pieces: a piece's next copy starts as soon as it has been read and
    // lands while the other is rebuilt.  All rows come of a page that holds a row
    // some query sees, zeros for others (a coordinate past the pool); a row that
    // nobody sees gets scale 0, and every byte dequantises to a finite number.
    const uint32_t raw_u = smem_u32(smem + L::kOffRaw) + (warp - 8) * 2 * kRawPiece;
    uint64_t* const raw_full = &sm.raw_full[(warp - 8) * 2];
    uint32_t used = 0;                        // tiles whose pieces have been used up
    // Piece h's copy: its rows, from the slots of lanes l0 and l0 + 16 (V in pages of
    // 16 tokens: two boxes).
    auto copy_raw = [&](const CUtensorMap* map, int h, int slot, int l0, int col, int bytes) {
      if (!p.use_tma) return;
      const int past = p.num_pages << p.page_shift;
      const int s0 = __shfl_sync(0xffffffffu, slot, l0), s1 = __shfl_sync(0xffffffffu, slot, 16);
      if (lane == 0) {
        mbar_arrive_expect_tx(&raw_full[h], kRawPiece);
        tma_load_3d_at(raw_u + h * kRawPiece, map, &raw_full[h], col, s0 < 0 ? past : s0, x.g);
        if (bytes < kRawPiece)
          tma_load_3d_at(raw_u + h * kRawPiece + bytes, map, &raw_full[h], col, s1 < 0 ? past : s1, x.g);
      }
      __syncwarp();
    };
    // Rebuilds piece h into rows row0 .. of an item: a pass has `rows` rows (2 of K, 4
    // of V), this lane 16 bytes (piece c16) of row `sub`; each eight lanes hold four
    // pieces of two adjacent rows, whose bf16 chunks fall on eight different bank
    // groups.  The exponent of row i sits in lane l0 + i.
    auto rebuild = [&](int h, uint32_t item, int rows, int sub, int c16, int l0, uint32_t e) -> bool {
      if (p.use_tma && !warp_wait(&raw_full[h], used & 1, sm, ctl)) return false;
      const uint32_t src0 = raw_u + h * kRawPiece + lane_src(rows, sub, c16);
      const uint32_t base = item + sub * 128 + (c16 >> 2) * kKBlk;
      const uint32_t cs = (uint32_t)(((c16 & 3) * 2) ^ sub);     // chunk, swizzled by the row's low bits
      const uint32_t m = main_scale(e);
      uint4 wa = ld_shared_v4(src0), wb = ld_shared_v4(src0 + 512);
#pragma unroll 1
      for (int it = 0; it < 8; it += 2) {
        const uint32_t ma = __shfl_sync(0xffffffffu, m, l0 + it * rows + sub);
        const uint32_t mb = __shfl_sync(0xffffffffu, m, l0 + (it + 1) * rows + sub);
        const uint2 qa[4] = {dequant4(wa.x, ma, p.spread), dequant4(wa.y, ma, p.spread),
                             dequant4(wa.z, ma, p.spread), dequant4(wa.w, ma, p.spread)};
        const uint2 qb[4] = {dequant4(wb.x, mb, p.spread), dequant4(wb.y, mb, p.spread),
                             dequant4(wb.z, mb, p.spread), dequant4(wb.w, mb, p.spread)};
        if (it < 6) {
          wa = ld_shared_v4(src0 + (it + 2) * 512);
          wb = ld_shared_v4(src0 + (it + 3) * 512);
        }
        const uint32_t ra = it * rows, rb = ra + rows;
        const uint32_t a0 = base + ra * 128 + ((cs ^ (ra & 7)) << 4);
        const uint32_t b0 = base + rb * 128 + ((cs ^ (rb & 7)) << 4);
        st_shared_v4(a0, make_uint4(qa[0].x, qa[0].y, qa[1].x, qa[1].y));
        st_shared_v4(a0 ^ 16, make_uint4(qa[2].x, qa[2].y, qa[3].x, qa[3].y));
        st_shared_v4(b0, make_uint4(qb[0].x, qb[0].y, qb[1].x, qb[1].y));
        st_shared_v4(b0 ^ 16, make_uint4(qb[2].x, qb[2].y, qb[3].x, qb[3].y));
      }
      __syncwarp();
      // what scales above 2^7 (values above 448 * 2^7) lack
      if (__any_sync(0xffffffffu, e > 134u && e < 255u))
        rescale_rows(base, rows, cs, l0 + sub, e);
      return true;
    };
    // After the last use: a bounded wait for pieces still on their way.
    auto land_raw = [&](uint32_t asked) {
      if (kE4M3 && p.use_tma && lane == 0 && asked > 0)
        for (int h = 0; h < 2; ++h) (void)mbar_wait(&raw_full[h], (asked - 1) & 1, ctl);
      __syncwarp();
    };
    const int odd = (lane >> 2) & 1;
    const int sub2 = odd, piece2 = (lane & 3) + 4 * (lane >> 3);
    const int sub4 = odd + 2 * (lane >> 4), piece4 = (lane & 3) + 4 * ((lane >> 3) & 1);
    // The boxes of one item: `blocks` 64-column blocks from block c0 of the
    // head, keys from position x0; lane l brings box l / blocks, block l % blocks
    // (pages of 64 tokens and more: one box of all blocks).  A page id out of
    // range reads past the pool, which TMA fills with zeros.
    auto tma_item = [&](const CUtensorMap* map, uint64_t* bar, uint32_t item, int blk0, int blocks,
                        int x0, int page) {
      const uint32_t full = bar_full(bar);
      if (leader && lw == 0 && lane == 0)
        mbar_arrive_expect_tx(bar, (uint32_t)(2 * blocks * kKBlk));
      __syncwarp();
      if (lw == 0) {
        const int per = boxes == 1 ? 1 : blocks;
        const int i = lane / per, blk = boxes == 1 ? 0 : lane % per;
        if (lane < boxes * per) {
          const int slot = slot_of(p, x0 + i * box, page, bad);
          tma_load_3d_pair(item + blk * kKBlk + i * box * 128, map, full, 0,
                           slot < 0 ? p.num_pages << p.page_shift : slot, blk0 + blk);
        }
      }
      __syncwarp();
      if (lane == 0 && !(leader && lw == 0)) mbar_arrive_remote(full);
    };
    const uint32_t pitch = (uint32_t)p.Hkv * (kD * 2);             // bf16 rows
    if (warp < 10) {
      const uint32_t kring_u = smem_u32(kring);
      const int my_row = 64 * (int)rank + (kE4M3 ? 32 * lw + lane : row32);
      const int tma_row = 64 * (int)rank + (boxes == 1 ? 0 : min(lane >> 2, boxes - 1) * box);
      uint32_t uk = 0, nq = 0;
      int page = kNoRow;
      auto copy_k = [&](const KeyTile& kt, uint32_t item) {
        const int at = kt.tile * kBN;
        const int mine = kt.chunk ? chunk_row(p, x, codes, at + 64 * (int)rank + row32)
                                  : slot_of(p, at + my_row, page, bad);
        const uint8_t* base =
            static_cast<const uint8_t*>(kt.chunk ? p.k : p.kp) + (x.g * (kD * 2) + lane * 16);
        copy_rows(mine, base, pitch, item + (lane >> 3) * kKBlk, 32, lw, 2, 0, 1);
      };
      // e4m3: this lane's row of the next tile, its slot (-1: no such tile) and exponent.
      int slot_n = -1;
      bool has_n = false;
      uint32_t ex_n = kNoExp, asked = 0;
      auto fetch = [&](int idx) {
        has_n = false;
        if (!kE4M3 || idx >= x.it0 + x.n) return;
        const KeyTile kt = key_tile(x, idx);
        if (kt.chunk) return;
        const int at = kt.tile * kBN + my_row;
        slot_n = slot_of(p, at, page, bad);
        page = peek(idx + 1, my_row, 0);
        ex_n = row_exp(p, p.ke, row_seen(p, x, at) ? slot_n : -1, x.g);
        has_n = true;
        ++asked;
      };
      while (const Segment* px = next_segment()) {
        x = *px;
        const int i0 = x.it0, n = x.n;
        if (n == 0) continue;
        page = peek(i0, my_row, tma_row);
        fetch(i0);
        if (has_n) {
          copy_raw(&p.map_k, 0, slot_n, 0, 0, kRawPiece);
          copy_raw(&p.map_k, 1, slot_n, 16, 0, kRawPiece);
        }
        // Q: this CTA's 128 rows in one box; tokens past the chunk are zeros.  (Warp 9
        // only counts in; nobody waits for Q of a failed run.)
        ok = acquire(&sm.q_empty, nq);
        ++nq;
        if (!ok) continue;
        if (leader && lw == 0 && lane == 0) mbar_arrive_expect_tx(&sm.q_full, 2 * kQBytes);
        __syncwarp();
        if (lane == 0) {
          if (lw == 0)
            tma_load_5d_pair(smem_u32(sQ), &p.map_q, bar_full(&sm.q_full), 0, x.g * p.G,
                             x.tq0 + (((int)rank * kBM) >> p.g_shift), 0, x.b);
          if (!(leader && lw == 0)) mbar_arrive_remote(bar_full(&sm.q_full));
        }
        __syncwarp();
        for (int idx = i0; idx < i0 + n; ++idx) {
          const KeyTile kt = key_tile(x, idx);
          const int s = (int)(uk % kNK);
          const uint32_t item = kring_u + s * kKItem;
          ok = acquire(&sm.k_empty[s], uk / kNK);
          if (!ok) break;
          ++uk;
          const uint32_t full = bar_full(&sm.k_full[s]);
          if (!kE4M3 && p.use_tma && whole_tile(p, x, kt)) {
            tma_item(&p.map_k, &sm.k_full[s], item, 4 * x.g, 4, kt.tile * kBN + 64 * (int)rank, page);
            page = peek(idx + 1, my_row, tma_row);
          } else if (!kE4M3 || kt.chunk) {
            copy_k(kt, item);
            if (!kE4M3) page = peek(idx + 1, my_row, tma_row);
            push(full);
            if (kE4M3 || idx == i0) flush();   // the first tile is waited for
          } else {
            const uint32_t ex = ex_n;
            fetch(idx + 1);
#pragma unroll 1
            for (int h = 0; h < 2 && ok; ++h) {
              ok = rebuild(h, item + (32 * lw + 16 * h) * 128, 2, sub2, piece2, 16 * h, ex);
              if (ok && has_n) copy_raw(&p.map_k, h, slot_n, 16 * h, 0, kRawPiece);
            }
            ++used;
            if (!ok) break;
            signal(full);
          }
        }
        flush();
      }
      land(sm.k_full, kNK, uk);
      land(&sm.q_full, 1, nq);
      land_raw(asked);
    } else {
      const uint32_t vring_u = smem_u32(vring);
      const int my_row = kE4M3 ? 32 * lw + lane : row16;
      const int box_bytes = min(1 << p.page_shift, 32) * 128;      // e4m3: of a raw piece's boxes
      const int tma_row = boxes == 1 ? 0 : min(lane >> 1, boxes - 1) * box;
      uint32_t uv = 0;
      int page0 = kNoRow, page1 = kNoRow;
      auto copy_v = [&](const KeyTile& kt, int h, uint32_t item) {
        const int at = kt.tile * kBN + 64 * h;
        const int mine = kt.chunk ? chunk_row(p, x, codes, at + row16)
                                  : slot_of(p, at + my_row, h ? page1 : page0, bad);
        const int ch = lane & 15;
        const uint8_t* base = static_cast<const uint8_t*>(kt.chunk ? p.v : p.vp) +
                              (x.g * (kD * 2) + (int)rank * 256 + ch * 16);
        copy_rows(mine, base, pitch, item + (ch >> 3) * kKBlk, 16, lw * 2 + (lane >> 4), 4,
                  lane >> 4, 2);
      };
      // e4m3: this lane's rows (one of each half) of the next tile, their exponents.
      uint32_t exn0 = kNoExp, exn1 = kNoExp, asked = 0;
      int slot0 = -1, slot1 = -1;
      bool has_n = false;
      auto fetch = [&](int idx) {
        has_n = false;
        if (!kE4M3 || idx >= x.it0 + x.n) return;
        const KeyTile kt = key_tile(x, idx);
        if (kt.chunk) return;
        const int at = kt.tile * kBN + my_row;
        slot0 = slot_of(p, at, page0, bad);
        slot1 = slot_of(p, at + 64, page1, bad);
        page0 = peek(idx + 1, my_row, 0);
        page1 = peek(idx + 1, 64 + my_row, 0);
        exn0 = row_exp(p, p.ve, row_seen(p, x, at) ? slot0 : -1, x.g);
        exn1 = row_exp(p, p.ve, row_seen(p, x, at + 64) ? slot1 : -1, x.g);
        has_n = true;
        ++asked;
      };
      while (const Segment* px = next_segment()) {
        x = *px;
        const int i0 = x.it0, n = x.n;
        if (n == 0) continue;
        page0 = peek(i0, my_row, tma_row);
        page1 = peek(i0, 64 + my_row, 64 + tma_row);
        fetch(i0);
        if (has_n) {
          copy_raw(&p.map_v, 0, slot0, 0, (int)rank * 128, box_bytes);
          copy_raw(&p.map_v, 1, slot1, 0, (int)rank * 128, box_bytes);
        }
        for (int idx = i0; idx < i0 + n && ok; ++idx) {
          const KeyTile kt = key_tile(x, idx);
          const uint32_t ex0 = exn0, ex1 = exn1;
          if (kE4M3) fetch(idx + 1);
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int s = (int)(uv % kNV);
            const uint32_t item = vring_u + s * kVItem;
            ok = ok && acquire(&sm.v_empty[s], uv / kNV);
            if (!ok) break;
            ++uv;
            const uint32_t full = bar_full(&sm.v_full[s]);
            if (!kE4M3) {
              const bool tma = p.use_tma && whole_tile(p, x, kt);
              if (tma)
                tma_item(&p.map_v, &sm.v_full[s], item, 4 * x.g + 2 * (int)rank, 2,
                         kt.tile * kBN + 64 * h, h ? page1 : page0);
              else
                copy_v(kt, h, item);
              const int next = peek(idx + 1, 64 * h + my_row, 64 * h + tma_row);
              page0 = h ? page0 : next;
              page1 = h ? next : page1;
              if (!tma) push(full);
            } else if (kt.chunk) {
              copy_v(kt, h, item);
              push(full);
            } else {
              ok = rebuild(h, item + 32 * lw * 128, 4, sub4, piece4, 0, h ? ex1 : ex0);
              if (ok && has_n)
                copy_raw(&p.map_v, h, h ? slot1 : slot0, 0, (int)rank * 128, box_bytes);
              used += h;
              if (!ok) break;
              signal(full);
            }
          }
        }
        flush();
      }
      land(sm.v_full, kNV, uv);
      land_raw(asked);
    }
    if (bad) record_status(ctl, kStatusArg);
  } else {
    // ---------------------------------------------- softmax and epilogue
    const int quarter = warp & 3, half = warp >> 2;
    const int r = quarter * 32 + lane;             // row of this thread in the CTA
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t tSr = tS + lane_off + 64 * half, tOr = tO + lane_off + 128 * half;
    const float c = p.scale_log2;
    const uint32_t s_free_l0 = mapa_shared(smem_u32(&sm.s_free[0]), 0);
    const uint32_t s_free_l1 = mapa_shared(smem_u32(&sm.s_free[1]), 0);
    const uint32_t p_full_l = mapa_shared(smem_u32(&sm.p_full), 0);
    const uint32_t o_free_l = mapa_shared(smem_u32(&sm.o_free), 0);
    uint8_t* const p_row = sP + half * kPBlk + r * 128;   // this thread's line of P
    uint8_t* const st = sP + half * kPBlk + quarter * 4096;   // this warp's 32 lines
    uint32_t gt = 0, n_pair = 0;
    bool store_pending = false;                    // this warp's output stores may still read P
    // Meets the quarter's other warp; what either wrote before is visible after.
    auto pair_sync = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.pair[quarter]);
      return warp_wait(&sm.pair[quarter], n_pair++ & 1, sm, ctl);
    };

    while (const Segment* px = next_segment()) {
      const Segment& x = *px;
      const int row = (int)rank * kBM + r;         // row of the query tile
      const int tok_raw = x.tq0 + (row >> p.g_shift);
      const bool row_valid = tok_raw <= x.tq1;
      const int tok = min(tok_raw, x.tq1);
      const long long orow =
          ((long long)x.b * p.Sq + tok) * p.Hq + (long long)x.g * p.G + (row & (p.G - 1));
      float* po = nullptr;
      float* pml = nullptr;
      if (x.slot >= 0) {
        const long long at = (long long)x.slot * kRowsTile + row;
        po = p.ws + at * kD + 128 * half;
        pml = p.ws + (long long)p.n_clusters * 2 * kRowsTile * kD + at * 2;
      }
      if (x.n == 0) {
        if (pml != nullptr) {
          if (row_valid && half == 0) *reinterpret_cast<float2*>(pml) = make_float2(-INFINITY, 0.f);
        } else {                                   // a whole unit without a key: zeros
          for (int rr = 16 * half; rr < 16 * half + 16; ++rr) {
            const long long at = __shfl_sync(0xffffffffu, orow, rr);
            const bool v = __shfl_sync(0xffffffffu, (int)row_valid, rr) != 0;
            if (v)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + at * (kD * 2) + lane * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          if (p.lse && row_valid && half == 0) p.lse[orow] = -INFINITY;
        }
        continue;
      }
      const uint32_t cq = codes[tok];
      const bool row_pad = is_pad(cq);
      const bool any_pad = __any_sync(0xffffffffu, row_pad);
      float m_run = -INFINITY, l_run = 0.f;        // l: this thread's half of the keys

      for (int li = 0; li < x.n; ++li, ++gt) {
        const int bs = (int)(gt & 1);
        const KeyTile kt = key_tile(x, x.it0 + li);
        const int k0 = kt.tile * kBN;
        // Does every row of the unit see every key of the tile?
        bool partial;
        if (kt.chunk) {
          const uint32_t fl = sm.tile_fast[kt.tile];
          partial = k0 + kBN > p.Sq || sm.tile_cs_last[kt.tile] > x.csq0 || (fl & kTilePad) ||
                    (x.any_e && (fl & kTileFast)) ||
                    (p.window > 0 && x.tq1 - k0 >= p.window && x.len + k0 + kBN > p.sinks);
        } else {
          partial = k0 + kBN > x.len || (p.window > 0 && k0 < x.lo1 && k0 + kBN > p.sinks);
        }
        uint2 vis = make_uint2(~0u, ~0u);
        if (partial) vis = row_mask(p, codes, x, kt.chunk, k0 + 64 * half, tok, cq);
        if (row_pad) vis = make_uint2(0u, 0u);
        if (!warp_wait(&sm.s_full[bs], (gt >> 1) & 1, sm, ctl)) { ok = false; break; }
        tc_fence_after();
        float xs[64];
        {
          uint32_t r0[32], r1[32];
          tmem_ld32(tSr + 128 * bs, r0);
          tmem_ld32(tSr + 128 * bs + 32, r1);
          tmem_ld_wait();
          reg_fence(r0);
          reg_fence(r1);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            xs[e] = __uint_as_float(r0[e]);
            xs[32 + e] = __uint_as_float(r1[e]);
          }
        }
        if (partial || any_pad) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            xs[e] = ((vis.x >> e) & 1u) ? xs[e] : -INFINITY;
            xs[32 + e] = ((vis.y >> e) & 1u) ? xs[32 + e] : -INFINITY;
          }
        }
        float m4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float a = xs[k];
#pragma unroll
          for (int i = 1; i < 15; i += 2) a = fmax3(a, xs[k + 4 * i], xs[k + 4 * i + 4]);
          m4[k] = fmaxf(a, xs[k + 60]);
        }
        // The row's maximum over both halves: each thread leaves its own in the
        // first column of its half of S, which only it reads.
        float mx = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * c;
        tmem_st1(tSr + 128 * bs, __float_as_uint(mx));
        tmem_st_wait();
        tc_fence_before();
        if (!pair_sync()) { ok = false; break; }
        tc_fence_after();
        {
          uint32_t o[1];
          tmem_ld1(tS + lane_off + 64 * (1 - half) + 128 * bs, o[0]);
          tmem_ld_wait();
          reg_fence(o);
          mx = fmaxf(mx, __uint_as_float(o[0]));
        }
        // S has been read: the QK after next may overwrite it.
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(bs ? s_free_l1 : s_free_l0);
        // Lazy rescaling.
        const bool upd = mx > m_run + kRescaleThreshold;
        const float m_new = upd ? mx : m_run;
        const float alpha = ex2(m_run - m_new);
        const bool need_o = upd && (m_run != -INFINITY);
        l_run *= (m_run == -INFINITY) ? 0.f : alpha;
        m_run = m_new;
        const float nm = (m_run == -INFINITY) ? 0.f : -m_run;
        const float2 c2 = make_float2(c, c), n2 = make_float2(nm, nm);
        float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 t = ffma2(make_float2(xs[2 * e], xs[2 * e + 1]), c2, n2);
          const float2 pp = make_float2(ex2(t.x), ex2(t.y));
          ls[e & 3] = fadd2(ls[e & 3], pp);
          pk[e] = cvt_bf16x2(pp.x, pp.y);
        }
        const float2 lsum = fadd2(fadd2(ls[0], ls[1]), fadd2(ls[2], ls[3]));
        l_run += lsum.x + lsum.y;

        // The previous PV reads P and accumulates into O.
        if (gt >= 1) {
          if (!warp_wait(&sm.o_done, (gt - 1) & 1, sm, ctl)) { ok = false; break; }
          tc_fence_after();
        }
        if (store_pending) {                       // the last output's stores read P
          if (lane == 0) tma_store_wait_read();
          __syncwarp();
          store_pending = false;
        }
        const bool rescale = __any_sync(0xffffffffu, need_o);
        if (rescale) {
          const float a = need_o ? alpha : 1.f;
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t o[32];
            tmem_ld32(tOr + 32 * cc, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
            tmem_st32(tOr + 32 * cc, o);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(p_row + ((j ^ (r & 7)) << 4)) =
              make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        fence_proxy_async_smem();
        if (rescale) tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(p_full_l);
      }
      if (!ok) continue;

      // ----------------------------------------------------- epilogue
      if (!warp_wait(&sm.o_done, (gt - 1) & 1, sm, ctl)) { ok = false; continue; }
      tc_fence_after();
      // The row's other half of l, through the P line (free: the last PV is done).
      float l_all;
      if (store_pending) {                         // (a segment of one tile before this one)
        if (lane == 0) tma_store_wait_read();
        __syncwarp();
        store_pending = false;
      }
      {
        float* const mine = reinterpret_cast<float*>(p_row);
        const float* const other = reinterpret_cast<const float*>(sP + (1 - half) * kPBlk + r * 128);
        *mine = l_run;
        if (!pair_sync()) { ok = false; continue; }   // both halves have written
        l_all = l_run + *other;
        if (!pair_sync()) { ok = false; continue; }   // and read: the lines are free
      }
      if (po == nullptr) {
        const float inv = l_all > 0.f ? 1.f / l_all : 0.f;
        // Each warp stages 32 rows of 64 columns in its own P lines (another warp may
        // already write the next segment's P) and stores them as one box; tokens past
        // the chunk are clipped.
#pragma unroll 1
        for (int sub = 0; sub < 2; ++sub) {
          uint32_t o0[32], o1[32];
          tmem_ld32(tOr + 64 * sub, o0);
          tmem_ld32(tOr + 64 * sub + 32, o1);
          tmem_ld_wait();
          reg_fence(o0);
          reg_fence(o1);
          if (sub == 1) {                          // this warp's part of O has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_remote(o_free_l);
              tma_store_wait_read();               // the first half's lines
            }
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = 8 * j + 2 * e;
              const uint32_t lo_w = at < 32 ? o0[at & 31] : o1[at & 31];
              const uint32_t hi_w = at < 32 ? o0[(at + 1) & 31] : o1[(at + 1) & 31];
              w[e] = cvt_bf16x2(__uint_as_float(lo_w) * inv, __uint_as_float(hi_w) * inv);
              if (l_all == 0.f) w[e] = 0u;         // O may hold 0 * inf of other rows' keys
            }
            *reinterpret_cast<uint4*>(st + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          const int tok0 = x.tq0 + (((int)rank * kBM + quarter * 32) >> p.g_shift);
          if (lane == 0 && tok0 <= x.tq1) {
            tma_store_5d(&p.map_o, st, 0, x.g * p.G, tok0, 2 * half + sub, x.b);
            tma_store_commit();
          }
          __syncwarp();
        }
        store_pending = true;
        if (p.lse && row_valid && half == 0)
          p.lse[orow] = l_all > 0.f ? (m_run + __log2f(l_all)) * 0.69314718055994531f
                                    : (l_all == l_all ? -INFINITY : l_all);
      } else {
        // Partial: unnormalised O and (m, l).
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t o[32];
          tmem_ld32(tOr + 32 * cc, o);
          tmem_ld_wait();
          reg_fence(o);
          if (row_valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(po + 32 * cc + e) =
                  make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(o_free_l);
        if (row_valid && half == 0) *reinterpret_cast<float2*>(pml) = make_float2(m_run, l_all);
      }
    }
    if (store_pending && lane == 0) tma_store_wait_read();
    __syncwarp();
  }

  // Neither CTA may leave while its partner can still signal its barriers or
  // read its shared memory; then both free their TMEM.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && sm.abort) st_cluster_u32(mapa_shared(smem_u32(&sm.abort), rank ^ 1u), 1u);
  cluster_sync();
  if (sm.abort) settle();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Merges the partials of units that were cut: out = sum_k 2^(m_k - M) O_k /
// sum_k 2^(m_k - M) l_k with M the largest m_k that has l_k > 0.  CTA (u, y):
// every gridDim.y-th eight rows of unit u, a warp each: a lane weighs one partial,
// then takes 8 columns of all of them, four partials in flight.  Bound by that
// latency: the partials lie in L2.
constexpr int kCombineRows = 8;
__global__ void __launch_bounds__(32 * kCombineRows)
    paged_combine_kernel(const __grid_constant__ PagedTcParams p, const DevCtl ctl) {
  __shared__ Plan plan;
  pdl_wait();                  // the partials come from the kernel before
  pdl_launch_dependents();
  if (threadIdx.x < 32) make_plan(p, ctl, plan, threadIdx.x);
  __syncthreads();
  const int per = tiles_per_cluster(p, plan);
  if (per == 0) return;
  const int units = p.Hkv * p.n_tiles;
  const int b = (int)(blockIdx.x / units), u = (int)(blockIdx.x % units);
  const int nom = (plan.cum[b + 1] - plan.cum[b]) / units;
  const int t0 = plan.cum[b] + u * nom;
  const int c0 = t0 / per, c1 = (t0 + nom - 1) / per;
  if (c0 == c1) return;        // ran whole
  const int g = u / p.n_tiles, tile = u % p.n_tiles;
  const int lane = threadIdx.x & 31;
  const float2* ml = reinterpret_cast<const float2*>(
      p.ws + (long long)p.n_clusters * 2 * kRowsTile * kD);
  for (int row = blockIdx.y * kCombineRows + (threadIdx.x >> 5); row < p.G * p.tok_per_tile;
       row += gridDim.y * kCombineRows) {
    const int tok = tile * p.tok_per_tile + (row >> p.g_shift);
    if (tok >= p.Sq) break;
    // the unit's part of cluster c: its last run in c0, else its first
    auto at = [&](int c) { return (long long)(c * 2 + (c == c0 ? 1 : 0)) * kRowsTile + row; };
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) {
      const float2 v = ml[at(c)];
      if (v.y > 0.f) M = fmaxf(M, v.x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    float l = 0.f;
    for (int cb = c0; cb <= c1; cb += 32) {
      const int n = min(c1 - cb + 1, 32);
      float w = 0.f;
      bool live = false;         // false: the part saw no key (a NaN goes on)
      if (lane < n) {
        const float2 v = ml[at(cb + lane)];
        live = !(v.y == 0.f);
        w = live ? ex2(v.x - M) : 0.f;
        if (live) l += w * v.y;
      }
      const uint32_t on = __ballot_sync(0xffffffffu, live);
      for (int j0 = 0; j0 < n; j0 += 4) {
        float4 a[4], d[4];
        float wj[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = j0 + j;
          wj[j] = __shfl_sync(0xffffffffu, w, c & 31);
          a[j] = d[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c < n && ((on >> c) & 1u)) {
            const float4* src = reinterpret_cast<const float4*>(p.ws + at(cb + c) * kD + lane * 8);
            a[j] = src[0];
            d[j] = src[1];
          } else {
            wj[j] = 0.f;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[0] += wj[j] * a[j].x; acc[1] += wj[j] * a[j].y;
          acc[2] += wj[j] * a[j].z; acc[3] += wj[j] * a[j].w;
          acc[4] += wj[j] * d[j].x; acc[5] += wj[j] * d[j].y;
          acc[6] += wj[j] * d[j].z; acc[7] += wj[j] * d[j].w;
        }
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    const long long orow =
        ((long long)(p.b0 + b) * p.Sq + tok) * p.Hq + (long long)g * p.G + (row & (p.G - 1));
    uint4 w;
    w.x = cvt_bf16x2(acc[0] * inv, acc[1] * inv);
    w.y = cvt_bf16x2(acc[2] * inv, acc[3] * inv);
    w.z = cvt_bf16x2(acc[4] * inv, acc[5] * inv);
    w.w = cvt_bf16x2(acc[6] * inv, acc[7] * inv);
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + orow * (kD * 2) + lane * 16) = w;
    if (p.lse && lane == 0)
      p.lse[orow] = l > 0.f ? (M + __log2f(l)) * 0.69314718055994531f : (l == l ? -INFINITY : l);
  }
}

template <bool kE4M3>
cudaError_t launch(PagedTcParams& p, const DevCtl& ctl, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(
      paged_tc_kernel<kE4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e != cudaSuccess) return e;
  p.smem_bytes = kSmemLimit;
  return launch_pdl(paged_tc_kernel<kE4M3>, dim3(2 * p.n_clusters), dim3(kThreads),
                    (size_t)p.smem_bytes, st, p, ctl);
}

// bf16: a pool [slots][Hkv][256] as (64, slots, 4 Hkv column blocks), boxes of a
// page's rows (64 at most) by `blocks` column blocks, or one for small pages.
// e4m3: as (256 bytes, slots, Hkv), boxes of `rows` rows at most by `cols` bytes.
bool encode_pool(CUtensorMap* map, const void* base, const PagedParams& p, uint32_t blocks,
                 uint32_t rows, uint32_t cols) {
  auto fn = encode_fn();
  if (!fn) return false;
  const bool e4 = p.cache_dtype == kCacheE4M3;
  const uint32_t page = 1u << p.page_shift, n = page < rows ? page : rows;
  const cuuint64_t slots = (cuuint64_t)p.num_pages << p.page_shift, row = e4 ? kD : 2 * kD;
  cuuint64_t dims[3] = {e4 ? (cuuint64_t)kD : 64, slots, (e4 ? 1 : 4) * (cuuint64_t)p.Hkv};
  cuuint64_t strides[2] = {row * p.Hkv, e4 ? (cuuint64_t)kD : 128};
  cuuint32_t box[3] = {e4 ? cols : 64, n, e4 || page < 64 ? 1 : blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, e4 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            e4 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query or output rows [B][Sq][Hq][256] as (64, heads, tokens, 4 column blocks,
// B): a box of G heads, n / G tokens and `blocks` blocks is n rows of a tile.
bool encode_rows5(CUtensorMap* map, const void* base, const PagedTcParams& p, uint32_t n,
                  uint32_t blocks) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t row = 2 * kD;
  cuuint64_t dims[5] = {64, (cuuint64_t)p.Hq, (cuuint64_t)p.Sq, 4, (cuuint64_t)p.B};
  cuuint64_t strides[4] = {row, row * p.Hq, 128, row * p.Hq * p.Sq};
  cuuint32_t box[5] = {64, (cuuint32_t)p.G, n / (uint32_t)p.G, blocks, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether n_units units may be cut.  Not with four or more per cluster: the last
// round's idle clusters cost less than partials and a merge.  Nor if the longest
// cache the page table can hold has few tiles and cutting would not pay for a full
// batch: then the merge kernel (6 us of 32 at 32 sequences of 816 + 51 tokens) is
// not launched, and a ragged batch loses at most those few tiles' time.
bool may_cut(const PagedParams& p, long long n_units, int slots) {
  if (n_units >= 4ll * slots) return false;
  const long long nom = (((long long)p.max_pages << p.page_shift) + kBN - 1) / kBN +
                        (p.Sq + kBN - 1) / kBN;
  const long long per = (nom * n_units + slots - 1) / slots;
  const long long rounds = (n_units + slots - 1) / slots;
  return nom > 16 || rounds * nom > (per > 2 ? per : 2) + 5;
}

int slots() { return max(sm_count() / 2, 1); }

}  // namespace

// Sequences per launch: at most kGroup, their tiles below 2^31.
static int group_size(const PagedParams& p) {
  const int G = p.Hq / p.Hkv;
  const long long units = (long long)p.Hkv * ((p.Sq + kRowsTile / G - 1) / (kRowsTile / G));
  const long long tiles = (((long long)p.max_pages << p.page_shift) + kBN - 1) / kBN +
                          (p.Sq + kBN - 1) / kBN;
  const long long n = ((1ll << 31) - 1) / max(units * tiles, 1ll);
  return (int)min(n, (long long)kGroup);
}

bool paged_tc_applies(const PagedParams& p) {
  const int G = p.Hq / p.Hkv;
  return !p.f32 && p.d == kD && (G == 1 || G == 2 || G == 4 || G == 8 || G == 16) &&
         (long long)p.B * p.Sq < (1ll << 31) && group_size(p) >= 1;
}

// e4m3 pages and a chunk of several query tiles: each tile's cluster would rebuild
// the same rows.  From four tiles on, one pass writes the cached rows that the chunk
// sees as bf16 into the workspace and the bf16 form reads those.  Measured, rebuilt
// in every cluster / expanded first, 32 new tokens a tile: four sequences of 15000
// tokens, 2 tiles 71 / 77 us, 3 tiles 86 / 87, 4 tiles 103 / 98, 8 tiles 178 / 147,
// 16 tiles 337 / 247; 32 sequences of 816 tokens, 2 tiles 33 / 36, 4 tiles 57 / 54, 8
// tiles 115 / 103; one of 2000 tokens, 4 tiles 35 / 37.  Not for page tables that
// reach over more than half a GiB of rows.
static size_t expanded_bytes(const PagedParams& p) {
  const int tiles = (p.Sq * (p.Hq / p.Hkv) + kRowsTile - 1) / kRowsTile;
  if (p.cache_dtype != kCacheE4M3 || tiles < 4 || p.num_pages == 0) return 0;
  const unsigned long long n =
      ((unsigned long long)p.max_pages << p.page_shift) * p.B * p.Hkv * (kD * 2);
  return n <= (1ull << 28) ? (size_t)n : 0;
}

size_t paged_tc_workspace_bytes(const PagedParams& p) {
  const int G = p.Hq / p.Hkv, group = group_size(p);
  const long long units = (long long)p.Hkv * ((p.Sq + kRowsTile / G - 1) / (kRowsTile / G));
  // The last group of sequences is the smallest: it decides.
  const int last = p.B % group ? p.B % group : group;
  size_t n = 0;
  if (may_cut(p, last * units, slots())) n += (size_t)slots() * 2 * kRowsTile * (kD + 2) * sizeof(float);
  if (p.Sq > kSmemTokens) n += (size_t)slots() * 2 * pad_tokens(p.Sq) * sizeof(uint16_t);
  return n + 2 * expanded_bytes(p);
}

cudaError_t launch_paged_tc(const PagedParams& given, float* ws, const DevCtl& ctl,
                            cudaStream_t st) {
  PagedParams a = given;
  if (const size_t n = expanded_bytes(a)) {
    CacheParams c{};
    uint8_t* rows = reinterpret_cast<uint8_t*>(ws);
    ws = reinterpret_cast<float*>(rows + 2 * n);
    c.k_out = rows; c.v_out = rows + n;
    c.kp = const_cast<void*>(a.kp); c.vp = const_cast<void*>(a.vp);
    c.ke = const_cast<uint8_t*>(a.ke); c.ve = const_cast<uint8_t*>(a.ve);
    c.table = a.table; c.lens = a.lens;
    c.B = a.B; c.S = a.max_pages << a.page_shift; c.Hkv = a.Hkv; c.d = a.d;
    c.page_shift = a.page_shift; c.num_pages = a.num_pages; c.max_pages = a.max_pages;
    c.seen_only = true; c.window = a.window; c.sinks = a.sinks;
    const cudaError_t e = launch_cache(c, false, false, kCacheE4M3, ctl, st);
    if (e != cudaSuccess) return e;
    a.kp = c.k_out; a.vp = c.v_out;
    a.ke = a.ve = nullptr;
    a.num_pages = a.B * a.max_pages;
    a.cache_dtype = kCacheBF16;
    a.in_order = true;
  }
  PagedTcParams p{};
  static_cast<PagedParams&>(p) = a;
  p.ws = ws;
  p.G = a.Hq / a.Hkv;
  p.g_shift = p.G == 1 ? 0 : p.G == 2 ? 1 : p.G == 4 ? 2 : p.G == 8 ? 3 : 4;
  p.tok_per_tile = kRowsTile / p.G;
  p.n_tiles = (a.Sq + p.tok_per_tile - 1) / p.tok_per_tile;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.spread = {16u, 240u};
  p.use_tma = a.num_pages > 0;
  const bool e4 = a.cache_dtype == kCacheE4M3;
  if (p.use_tma && (!encode_pool(&p.map_k, a.kp, a, 4, e4 ? 16 : 64, 256) ||
                    !encode_pool(&p.map_v, a.vp, a, 2, e4 ? 32 : 64, 128)))
    return cudaErrorUnknown;
  if (!encode_rows5(&p.map_q, a.q, p, kBM, 4) || !encode_rows5(&p.map_o, a.out, p, 32, 1))
    return cudaErrorUnknown;
  const int group = group_size(a);
  const long long unit_tiles = (long long)a.Hkv * p.n_tiles;
  const bool any_cut = may_cut(a, (a.B % group ? a.B % group : group) * unit_tiles, slots());
  p.codes = reinterpret_cast<uint16_t*>(
      ws + (any_cut ? (size_t)slots() * 2 * kRowsTile * (kD + 2) : 0));
  for (int b0 = 0; b0 < a.B; b0 += group) {
    p.b0 = b0;
    p.nb = min(group, a.B - b0);
    const long long n_units = (long long)p.nb * a.Hkv * p.n_tiles;
    p.may_cut = any_cut && may_cut(a, n_units, slots()) ? 1 : 0;
    p.n_clusters = p.may_cut ? slots() : (int)min(n_units, (long long)slots());
    const cudaError_t e = e4 ? launch<true>(p, ctl, st) : launch<false>(p, ctl, st);
    if (e != cudaSuccess) return e;
    if (p.may_cut) {
      // A round of CTAs at most: each derives the schedule, cut unit or not.
      int y = kRowsTile / kCombineRows;
      while (y > 4 && n_units * y > 4ll * sm_count()) y >>= 1;
      const dim3 grid((unsigned)n_units, (unsigned)y);
      const cudaError_t c =
          launch_pdl(paged_combine_kernel, grid, dim3(32 * kCombineRows), 0, st, p, ctl);
      if (c != cudaSuccess) return c;
    }
  }
  return cudaSuccess;
}

}  // namespace piattn
