// paged_tc.cu -- attention of a chunk over the paged cache on tcgen05,
// CTA-pair (2-SM) form: bf16 queries, head_dim 256, pages in bf16 or e4m3.
//
// A cluster of two CTAs computes 256-row query tiles: 256 / G new tokens x the
// G query heads of one key/value head, 128 rows per CTA, against tiles of 128
// keys (cached tiles first, then the chunk's own).  Per key tile
//   S = Q K^T   tcgen05.mma.cta_group::2, M = 256: K split by keys (64 per CTA)
//   P           fp32 online softmax, one thread per row, P rounded to bf16 once
//   O += P V    tcgen05.mma.cta_group::2: V split by columns (128 per CTA)
// as in the dense kernel (tc_pair.cu).  What differs is how keys arrive and how
// the work is shared out.
//
// Loading.  Four loader warps per CTA gather rows by page into the operands'
// 128-byte-swizzled layout: every lane looks up one row's slot, warps copy whole
// rows (16 bytes per lane).  A tensor-map load would need one copy per page and
// 64-column block (32 per tile at 16-token pages), could not hide a row that no
// query sees, and its map costs the host more than the smallest call takes.
// Rows past the length, outside the window or of padding tokens are written as
// zeros, so whatever a stale slot holds (NaN) meets P = 0 as 0.
//   bf16: cp.async, up to three items (K: 32 KB, half V: 16 KB) in flight.
//   e4m3: 16-byte loads held in registers one tile ahead (32 KB raw per CTA in
//   flight), then e4m3 -> fp16 -> fp32 * 2^e -> bf16.  Every step is exact, as
//   the scale is a power of two: no rounding beside the cache's own.
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
// Warp roles per CTA (384 threads, three warpgroups):
//   warps 0..3   softmax, O correction, epilogue (240 registers)
//   warps 4..7   loaders
//   warp 8       TMEM allocation; QK issue (even CTA)
//   warp 9       PV issue (even CTA)
// TMEM per CTA (512 columns): O fp32 [0,256) | S0 [256,384) | S1 [384,512).
// Shared memory per CTA: Q 64 KB | K ring 2 x 32 KB | V ring 2 or 4 x 16 KB |
// P 32 KB (also the output staging area) | control | chunk token codes.
// Every wait is bounded (DevCtl); counters that index barriers and ring slots
// run across segments.
#include <cfloat>

#include "launch.h"
#include "paged.cuh"

namespace piattn {

namespace {

constexpr int kThreads = 384;
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

template <int kNV_, int kMaxTok_>
struct Layout {
  static constexpr int kNV = kNV_;
  static constexpr int kMaxTok = kMaxTok_;
  static constexpr int kTiles = (kMaxTok + kBN - 1) / kBN;
  static constexpr int kOffV = kOffK + kNK * kKItem;
  static constexpr int kOffP = kOffV + kNV * kVItem;
  static constexpr int kOffCtl = kOffP + kPBytes;
};

template <class L>
struct __align__(8) Smem {
  uint64_t q_full, q_empty;
  uint64_t k_full[kNK], k_empty[kNK];
  uint64_t v_full[L::kNV], v_empty[L::kNV];
  uint64_t s_full[2], s_free[2];
  uint64_t p_full, o_done, o_free;
  uint64_t drain_qk, drain_pv;
  uint32_t tmem_base;
  int abort;
  int scan[kThreads / 32];
  long long cum[kGroup + 1];        // nominal tiles before each sequence's units
  int max_nom;
  uint16_t tile_cs_first[L::kTiles];
  uint16_t tile_cs_last[L::kTiles];
  uint8_t tile_fast[L::kTiles];
};

template <class L>
__host__ __device__ constexpr int off_codes() {
  return L::kOffCtl + ((int)sizeof(Smem<L>) + 127) / 128 * 128;
}
__host__ __device__ constexpr int pad_tokens(int n) { return (n + 127) / 128 * 128; }
template <class L>
__host__ __device__ constexpr int layout_bytes(int n_tok) {
  return off_codes<L>() + pad_tokens(n_tok) * 2;
}
using LayoutLong = Layout<2, kMaxTokens>;
using LayoutShort = Layout<4, 512>;         // four V halves beside a short chunk's codes
static_assert(layout_bytes<LayoutLong>(kMaxTokens) <= kSmemLimit, "layout too large");
static_assert(layout_bytes<LayoutShort>(512) <= kSmemLimit, "short layout too large");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, int* abort,
                                              const DevCtl& ctl) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*(volatile int*)abort) return false;
    if ((unsigned long long)(clock64() - t0) > ctl.wait_limit) {
      record_status(ctl, kStatusTimeout);
      *(volatile int*)abort = 1;
      return false;
    }
  }
  return true;
}

template <class SmemT>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, SmemT& sm,
                                          const DevCtl& ctl) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, &sm.abort, ctl));
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

// Block-wide: cum[0 .. nb] (tiles before each sequence) and the largest nominal
// count, from cache_lens.  Every thread of the block calls it.
template <int kT>
__device__ void build_schedule(const PagedTcParams& p, const DevCtl& ctl, long long* cum,
                               int* max_nom) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) *max_nom = 0;
  __syncthreads();
  if (warp == 0) {
    long long carry = 0;
    int top = 0;
    bool bad = false;
    const long long units = (long long)p.Hkv * p.n_tiles;
    for (int base = 0; base < p.nb; base += 32) {
      const int b = base + lane;
      int nom = 0;
      if (b < p.nb)
        nom = nominal_tiles(p, cached_len(p.lens, p.b0 + b, p.max_pages, p.page_shift, bad));
      top = max(top, nom);
      long long x = units * nom;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      if (b < p.nb) cum[b + 1] = carry + x;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) cum[0] = 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) *max_nom = top;
    if (bad && blockIdx.x == 0) record_status(ctl, kStatusArg);
  }
  __syncthreads();
}

// Tiles per cluster when the tiles are cut into equal ranges; 0: units run
// whole, unit u on cluster u % n_clusters.  A cut costs a cluster about five
// tiles' time (partials written and merged: measured against whole units at 32
// sequences of 816 + 51 tokens), so units stay whole unless cutting saves that.
__device__ __forceinline__ long long tiles_per_cluster(const PagedTcParams& p, long long total,
                                                       int max_nom) {
  if (!p.may_cut) return 0;
  const long long n_units = (long long)p.nb * p.Hkv * p.n_tiles;
  const long long per = max((total + p.n_clusters - 1) / p.n_clusters, 2ll);
  const long long rounds = (n_units + p.n_clusters - 1) / p.n_clusters;
  return rounds * max_nom <= per + 5 ? 0 : per;
}

// A run of key tiles of one unit on this cluster.
struct Segment {
  int b, g, tile;            // sequence (absolute), kv head, query tile
  int tq0, tq1;              // its first / last new token
  int len;                   // cached tokens
  int lo0, lo1;              // window start of the first / last token (cached positions)
  int sink_tiles, win_tile;  // cached tiles [0, sink_tiles) and [win_tile, ...)
  int n_cached, c0;          // number of cached tiles; first chunk tile
  int it0, n;                // this run: tiles [it0, it0 + n) of the unit's list
  int slot;                  // partial slot, -1: the unit runs whole here
  uint32_t csq0, csq1;       // block index of the first / last token
  bool any_e;                // an expert among the tokens
};

// Where the walk over this cluster's segments stands.
struct Walk {
  long long pos, end, step;  // cut: tile range; whole: unit index, count, stride
  int seg;
};

template <class SmemT>
__device__ __forceinline__ int find_seq(const SmemT& sm, int nb, long long pos) {
  int lo = 0, hi = nb - 1;                   // largest b with cum[b] <= pos
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sm.cum[mid] <= pos) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Takes the next segment's place in the schedule: b, g, tile and the nominal
// range [s0, s1) of nom tiles.  False when the cluster is done.
template <class SmemT>
__device__ bool next_place(const PagedTcParams& p, const SmemT& sm, long long per, Walk& w,
                           Segment& x, int& s0, int& s1, int& nom) {
  if (w.pos >= w.end) return false;
  const int units = p.Hkv * p.n_tiles;
  long long u;
  int b;
  if (per == 0) {
    b = (int)(w.pos / units);
    u = w.pos % units;
    nom = (int)((sm.cum[b + 1] - sm.cum[b]) / units);
    s0 = 0;
    s1 = nom;
    x.slot = -1;
    w.pos += w.step;
  } else {
    b = find_seq(sm, p.nb, w.pos);
    nom = (int)((sm.cum[b + 1] - sm.cum[b]) / units);
    const long long rem = w.pos - sm.cum[b];
    u = rem / nom;
    s0 = (int)(rem % nom);
    s1 = (int)min((long long)nom, s0 + (w.end - w.pos));
    // A run that begins mid-unit is its cluster's first: slot 0, else slot 1.
    x.slot = s0 == 0 && s1 == nom ? -1 : (int)(w.pos / per) * 2 + (s0 > 0 ? 0 : 1);
    w.pos += s1 - s0;
  }
  x.b = p.b0 + b;
  x.g = (int)(u / p.n_tiles);
  x.tile = (int)(u % p.n_tiles);
  return true;
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
                                          const uint16_t* codes, Segment& x, int s0, int s1,
                                          int nom, int lane) {
  x.tq0 = x.tile * p.tok_per_tile;
  x.tq1 = min(x.tq0 + p.tok_per_tile, p.Sq) - 1;
  bool bad = false;
  x.len = cached_len(p.lens, x.b, p.max_pages, p.page_shift, bad);
  int any_e = 0, any_live = 0;
  for (int t = x.tq0 + lane; t <= x.tq1; t += 32) {
    const uint32_t c = codes[t];
    any_e |= (c >> 1) & 1;
    any_live |= is_pad(c) ? 0 : 1;
  }
  x.any_e = __any_sync(0xffffffffu, any_e);
  const bool live = __any_sync(0xffffffffu, any_live);
  x.csq0 = codes[x.tq0] >> 2;
  x.csq1 = codes[x.tq1] >> 2;
  x.lo0 = window_lo(p, x.len, x.tq0);
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
  x.it0 = (int)((long long)s0 * total / nom);
  x.n = (int)((long long)s1 * total / nom) - x.it0;
}

struct KeyTile {
  int tile;
  bool chunk;
};
__device__ __forceinline__ KeyTile key_tile(const Segment& x, int idx) {
  if (idx >= x.n_cached) return {x.c0 + idx - x.n_cached, true};
  return {idx < x.sink_tiles ? idx : x.win_tile + idx - x.sink_tiles, false};
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

// The cache slot of cached position x, -1 if no query of the segment sees it
// (or its page id is out of range, which is recorded).
__device__ __forceinline__ int cached_slot(const PagedTcParams& p, const Segment& s, int x,
                                           bool& bad) {
  if (x >= s.len || (p.window > 0 && x < s.lo0 && x >= p.sinks)) return -1;
  const int page = p.table[(long long)s.b * p.max_pages + (x >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) {
    bad = true;
    return -1;
  }
  return (page << p.page_shift) + (x & ((1 << p.page_shift) - 1));
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

// Eight raw e4m3 -> four bf16x2 words, times 2^(byte - 127): exact.
__device__ __forceinline__ void dequant8(uint32_t w0, uint32_t w1, float2 sc, uint32_t (&o)[4]) {
  const uint32_t w[2] = {w0, w1};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = fmul2(e4m3x2_to_float2((uint16_t)(w[i >> 1] >> (16 * (i & 1)))), sc);
    o[i] = cvt_bf16x2(v.x, v.y);
  }
}

template <bool kE4M3, class L>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedTcParams p, const DevCtl ctl) {
  using SmemT = Smem<L>;
  constexpr int kNV = L::kNV;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // Both CTAs see the same base offset, so both leave here or neither does.
  if ((int)(smem - smem_raw) + layout_bytes<L>(p.Sq) > p.smem_bytes || p.Sq > L::kMaxTok) {
    pdl_wait();
    if (threadIdx.x == 0) record_status(ctl, kStatusUnsupported);
    return;
  }
  SmemT& sm = *reinterpret_cast<SmemT*>(smem + L::kOffCtl);
  uint16_t* codes = reinterpret_cast<uint16_t*>(smem + off_codes<L>());
  uint8_t* sQ = smem + kOffQ;
  uint8_t* kring = smem + kOffK;
  uint8_t* vring = smem + L::kOffV;
  uint8_t* sP = smem + L::kOffP;

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cluster = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 8);
    mbar_init(&sm.q_empty, 1);
    for (int s = 0; s < kNK; ++s) {
      mbar_init(&sm.k_full[s], 8);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kNV; ++s) {
      mbar_init(&sm.v_full[s], 8);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.s_free[s], 8);
    }
    mbar_init(&sm.p_full, 8);
    mbar_init(&sm.o_done, 1);
    mbar_init(&sm.o_free, 8);
    mbar_init(&sm.drain_qk, 1);
    mbar_init(&sm.drain_pv, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  cluster_sync();                             // both CTAs' barriers exist
  if (warp == 8) {
    tmem_alloc_pair(&sm.tmem_base, 512);
    tmem_relinquish_pair();
  }
  pdl_wait();
  pdl_launch_dependents();
  build_schedule<kThreads>(p, ctl, sm.cum, &sm.max_nom);
  const long long per = tiles_per_cluster(p, sm.cum[p.nb], sm.max_nom);
  Walk walk;
  if (per == 0) {
    walk = {cluster, (long long)p.nb * p.Hkv * p.n_tiles, p.n_clusters, 0};
  } else {
    walk = {min(cluster * per, sm.cum[p.nb]), min((cluster + 1) * per, sm.cum[p.nb]), 0, 0};
  }

  // Block-wide: the codes of sequence b's chunk.
  int codes_b = -1;
  auto scan_codes = [&](int b) {
    const uint8_t* ar = p.ar + (long long)b * p.mask_bs;
    const int32_t* seg = p.seg ? p.seg + (long long)b * p.mask_bs : nullptr;
    const Flags32 f0 = load_flags32(ar, seg, p.Sq, (int)threadIdx.x * 32);
    __syncthreads();                          // nobody reads the old codes any more
    build_codes_x32<kThreads>(ar, seg, p.Sq, pad_tokens(p.Sq), codes, sm.scan, f0,
                              TileSums{sm.tile_cs_first, sm.tile_cs_last, sm.tile_fast});
    codes_b = b;
  };
  if (p.mask_bs == 0) scan_codes(0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Every warp walks the same segments; with a mask per sequence all of them
  // meet to scan the next sequence's (after a failure too, so that no one waits
  // for a warp that gave up).
  auto next_segment = [&](Segment& x) -> bool {
    int s0, s1, nom;
    if (!next_place(p, sm, per, walk, x, s0, s1, nom)) return false;
    if (p.mask_bs != 0 && x.b != codes_b) scan_codes(x.b);
    fill_segment(p, sm, codes, x, s0, s1, nom, lane);
    return true;
  };

  const uint32_t tmem = sm.tmem_base;
  const uint32_t tO = tmem + kColO, tS = tmem + kColS;      // S[b] at +128 b
  bool ok = true;
  Segment x;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    auto commit_both = [&](uint64_t* bar) {
      umma_commit_pair(mapa_shared(smem_u32(bar), 0));
      umma_commit_pair(mapa_shared(smem_u32(bar), 1));
    };
    uint32_t gt = 0, nu = 0;      // key tiles and segments processed
    if (warp == 8) {
      const uint64_t qdesc0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t kdesc0 = sdesc_sw128(smem_u32(kring), 16, 1024);
      while (next_segment(x)) {
        if (!leader || !ok || x.n == 0) continue;
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
#pragma unroll
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
    } else if (warp == 9) {
      const uint64_t pdesc0 = sdesc_sw128(smem_u32(sP), 16, 1024);
      const uint64_t vdesc0 = sdesc_sw128(smem_u32(vring), kKBlk, 1024);
      uint32_t uv = 0;
      while (next_segment(x)) {
        if (!leader || !ok || x.n == 0) continue;
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
    } else {
      while (next_segment(x)) {
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------- loaders
    const int lw = warp - 4;
    bool bad = false;
    uint32_t uk = 0, uv = 0, nq = 0;
    const uint32_t kring_u = smem_u32(kring), vring_u = smem_u32(vring), sQ_u = smem_u32(sQ);
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
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      flush();
      return warp_wait(bar, parity, sm, ctl);
    };
    auto bar_full = [&](uint64_t* bar) { return mapa_shared(smem_u32(bar), 0); };

    // Row lookup: lane l < 16 holds the l-th of the 16 rows this warp copies.
    // K: this CTA's rows l * 4 + lw of the tile; V half h: (l / 2) * 8 + lw * 2
    // + l % 2.  Cached rows are slots, chunk rows are rows of k_new.
    auto lookup = [&](const KeyTile& kt, int row) -> int {
      const int at = kt.tile * kBN + row;
      return kt.chunk ? chunk_row(p, x, codes, at) : cached_slot(p, x, at, bad);
    };
    auto copy_k = [&](const KeyTile& kt, int s) {
      const int mine = lane < 16 ? lookup(kt, 64 * (int)rank + lane * 4 + lw) : -1;
      const uint8_t* base = static_cast<const uint8_t*>(kt.chunk ? p.k : p.kp) + lane * 16;
      const uint32_t dst0 = kring_u + s * kKItem + (lane >> 3) * kKBlk;
#pragma unroll
      for (int it = 0; it < 16; ++it) {
        const int r = __shfl_sync(0xffffffffu, mine, it);
        const int row = it * 4 + lw;
        cp_async16(dst0 + row * 128 + (((lane & 7) ^ (row & 7)) << 4),
                   base + ((long long)max(r, 0) * p.Hkv + x.g) * (kD * 2), r >= 0);
      }
    };
    auto copy_v = [&](const KeyTile& kt, int h, int s) {
      const int mine =
          lane < 16 ? lookup(kt, 64 * h + (lane >> 1) * 8 + lw * 2 + (lane & 1)) : -1;
      const int ch = lane & 15;
      const uint8_t* base =
          static_cast<const uint8_t*>(kt.chunk ? p.v : p.vp) + (int)rank * 256 + ch * 16;
      const uint32_t dst0 = vring_u + s * kVItem + (ch >> 3) * kKBlk;
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int r = __shfl_sync(0xffffffffu, mine, it * 2 + (lane >> 4));
        const int row = it * 8 + lw * 2 + (lane >> 4);
        cp_async16(dst0 + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                   base + ((long long)max(r, 0) * p.Hkv + x.g) * (kD * 2), r >= 0);
      }
    };

    // e4m3: raw rows in registers, a tile ahead of their use.  K: 16 lanes per
    // row, rows it * 8 + lw * 2 + lane / 16; V half: 8 lanes per row, rows
    // it * 16 + lw * 4 + lane / 8.
    uint4 rk[kE4M3 ? 8 : 1], rv[2][kE4M3 ? 4 : 1];
    uint32_t ek[kE4M3 ? 8 : 1], ev[2][kE4M3 ? 4 : 1];
    auto fetch_k = [&](int idx) {
      if constexpr (kE4M3) {
        const KeyTile kt = key_tile(x, idx);
        if (idx >= x.it0 + x.n || kt.chunk) return;
        const int mine =
            lane < 16 ? lookup(kt, 64 * (int)rank + (lane >> 1) * 8 + lw * 2 + (lane & 1)) : -1;
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int r = __shfl_sync(0xffffffffu, mine, it * 2 + (lane >> 4));
          const long long at = (long long)r * p.Hkv + x.g;
          rk[it] = make_uint4(0u, 0u, 0u, 0u);
          ek[it] = 127u;
          if (r >= 0) {
            rk[it] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.kp) + at * kD +
                                                     (lane & 15) * 16);
            ek[it] = p.ke[at];
          }
        }
      }
    };
    auto fetch_v = [&](int idx, int h) {
      if constexpr (kE4M3) {
        const KeyTile kt = key_tile(x, idx);
        if (idx >= x.it0 + x.n || kt.chunk) return;
        const int mine =
            lane < 16 ? lookup(kt, 64 * h + (lane >> 2) * 16 + lw * 4 + (lane & 3)) : -1;
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const int r = __shfl_sync(0xffffffffu, mine, it * 4 + (lane >> 3));
          const long long at = (long long)r * p.Hkv + x.g;
          rv[h][it] = make_uint4(0u, 0u, 0u, 0u);
          ev[h][it] = 127u;
          if (r >= 0) {
            rv[h][it] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.vp) +
                                                        at * kD + (int)rank * 128 + (lane & 7) * 16);
            ev[h][it] = p.ve[at];
          }
        }
      }
    };
    // 16 raw bytes -> two 16-byte chunks; odd column blocks store them in the
    // other order, so that the eight lanes of a store hit eight bank groups.
    auto put16 = [&](uint32_t dst_row, int row, int c16, const uint4& w, uint32_t e) {
      const float sc = exp_scale(e);
      const float2 s2 = make_float2(sc, sc);
      uint32_t a[4], b[4];
      dequant8(w.x, w.y, s2, a);
      dequant8(w.z, w.w, s2, b);
      const bool swap = (c16 >> 2) & 1;
      const int c = (c16 & 3) * 2;
      const uint32_t base = dst_row + (c16 >> 2) * kKBlk;
      const uint32_t d0 = base + (((c + (swap ? 1 : 0)) ^ (row & 7)) << 4);
      const uint32_t d1 = base + (((c + (swap ? 0 : 1)) ^ (row & 7)) << 4);
      st_shared_v4(d0, swap ? make_uint4(b[0], b[1], b[2], b[3]) : make_uint4(a[0], a[1], a[2], a[3]));
      st_shared_v4(d1, swap ? make_uint4(a[0], a[1], a[2], a[3]) : make_uint4(b[0], b[1], b[2], b[3]));
    };

    auto load_k = [&](int idx) -> bool {
      const KeyTile kt = key_tile(x, idx);
      const int s = (int)(uk % kNK);
      if (!acquire(&sm.k_empty[s], uk / kNK)) return false;
      ++uk;
      if (!kE4M3 || kt.chunk) {
        copy_k(kt, s);
        push(bar_full(&sm.k_full[s]));
      } else {
#pragma unroll
        for (int it = 0; it < (kE4M3 ? 8 : 0); ++it) {
          const int row = it * 8 + lw * 2 + (lane >> 4);
          put16(kring_u + s * kKItem + row * 128, row, lane & 15, rk[it], ek[it]);
        }
        signal(bar_full(&sm.k_full[s]));
        if (n_pend > 0) flush();              // Q, or a chunk tile's item
      }
      fetch_k(idx + 1);
      return true;
    };
    auto load_v = [&](int idx, int h) -> bool {
      const KeyTile kt = key_tile(x, idx);
      const int s = (int)(uv % kNV);
      if (!acquire(&sm.v_empty[s], uv / kNV)) return false;
      ++uv;
      if (!kE4M3 || kt.chunk) {
        copy_v(kt, h, s);
        push(bar_full(&sm.v_full[s]));
      } else {
#pragma unroll
        for (int it = 0; it < (kE4M3 ? 4 : 0); ++it) {
          const int row = it * 16 + lw * 4 + (lane >> 3);
          put16(vring_u + s * kVItem + row * 128, row, lane & 7, rv[h][it], ev[h][it]);
        }
        signal(bar_full(&sm.v_full[s]));
      }
      return true;
    };

    while (next_segment(x)) {
      if (!ok || x.n == 0) continue;
      const int i0 = x.it0, n = x.n;
      fetch_k(i0);
      fetch_v(i0, 0);
      fetch_v(i0, 1);
      // Q: rows r of this CTA, 32 lanes per row.
      ok = acquire(&sm.q_empty, nq);
      ++nq;
      if (!ok) continue;
      {
        const uint8_t* qb = static_cast<const uint8_t*>(p.q) + lane * 16;
#pragma unroll 8
        for (int it = 0; it < 32; ++it) {
          const int r = it * 4 + lw;
          const int row = (int)rank * kBM + r;
          const int tok = x.tq0 + row / p.G;
          const long long at = ((long long)x.b * p.Sq + min(tok, x.tq1)) * p.Hq +
                               (long long)x.g * p.G + row % p.G;
          cp_async16(sQ_u + (lane >> 3) * kQBlk + r * 128 + (((lane & 7) ^ (r & 7)) << 4),
                     qb + at * (kD * 2), tok <= x.tq1);
        }
        push(bar_full(&sm.q_full));
      }
      ok = load_k(i0);
      if (ok && n > 1) ok = load_k(i0 + 1);
      for (int j = 0; j < n && ok; ++j) {
        if (j + 2 < n) ok = load_k(i0 + j + 2);
        if (ok) ok = load_v(i0 + j, 0);
        fetch_v(i0 + j + 1, 0);
        if (ok) ok = load_v(i0 + j, 1);
        fetch_v(i0 + j + 1, 1);
      }
      flush();
    }
    flush();
    if (bad) record_status(ctl, kStatusArg);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 240;");
    // ---------------------------------------------- softmax and epilogue
    const int r = warp * 32 + lane;                // row of this thread in the CTA
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const float c = p.scale_log2;
    const uint32_t s_free_l0 = mapa_shared(smem_u32(&sm.s_free[0]), 0);
    const uint32_t s_free_l1 = mapa_shared(smem_u32(&sm.s_free[1]), 0);
    const uint32_t p_full_l = mapa_shared(smem_u32(&sm.p_full), 0);
    const uint32_t o_free_l = mapa_shared(smem_u32(&sm.o_free), 0);
    uint8_t* const p_row0 = sP + r * 128;
    uint8_t* const p_row1 = sP + kPBlk + r * 128;
    uint32_t gt = 0;

    while (next_segment(x)) {
      if (!ok) continue;
      const int row = (int)rank * kBM + r;         // row of the query tile
      const int tok_raw = x.tq0 + row / p.G;
      const bool row_valid = tok_raw <= x.tq1;
      const int tok = min(tok_raw, x.tq1);
      const long long orow =
          ((long long)x.b * p.Sq + tok) * p.Hq + (long long)x.g * p.G + row % p.G;
      float* po = nullptr;
      float* pml = nullptr;
      if (x.slot >= 0) {
        const long long at = (long long)x.slot * kRowsTile + row;
        po = p.ws + at * kD;
        pml = p.ws + (long long)p.n_clusters * 2 * kRowsTile * kD + at * 2;
      }
      if (x.n == 0) {
        if (pml != nullptr) {
          if (row_valid) *reinterpret_cast<float2*>(pml) = make_float2(-INFINITY, 0.f);
        } else {                                   // a whole unit without a key: zeros
          for (int rr = 0; rr < 32; ++rr) {
            const long long at = __shfl_sync(0xffffffffu, orow, rr);
            const bool v = __shfl_sync(0xffffffffu, (int)row_valid, rr) != 0;
            if (v)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + at * (kD * 2) + lane * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          if (p.lse && row_valid) p.lse[orow] = -INFINITY;
        }
        continue;
      }
      const uint32_t cq = codes[tok];
      const uint32_t csq = cq >> 2;
      const bool row_expert = (cq & 2u) != 0;
      const bool row_pad = is_pad(cq);
      const int lo = window_lo(p, x.len, tok);     // cached keys below it: sinks only
      const int sink_end = p.window > 0 ? min(p.sinks, x.len) : 0;
      float m_run = -INFINITY, l_run = 0.f;

      for (int li = 0; li < x.n; ++li, ++gt) {
        const int bs = (int)(gt & 1);
        const KeyTile kt = key_tile(x, x.it0 + li);
        const int k0 = kt.tile * kBN;
        // Does every row of the unit see every key of the tile?
        bool partial;
        uint32_t fl = 0;
        if (kt.chunk) {
          fl = sm.tile_fast[kt.tile];
          partial = k0 + kBN > p.Sq || sm.tile_cs_last[kt.tile] > x.csq0 || (fl & 4u) ||
                    (x.any_e && (fl & 1u)) ||
                    (p.window > 0 && x.tq1 - k0 >= p.window && x.len + k0 + kBN > p.sinks);
        } else {
          partial = k0 + kBN > x.len || (p.window > 0 && k0 < x.lo1 && k0 + kBN > p.sinks);
        }
        if (!warp_wait(&sm.s_full[bs], (gt >> 1) & 1, sm, ctl)) { ok = false; break; }
        tc_fence_after();
        float xs[kBN];
        {
          uint32_t r0[32], r1[32], r2[32], r3[32];
          tmem_ld32(tS + lane_off + 128 * bs, r0);
          tmem_ld32(tS + lane_off + 128 * bs + 32, r1);
          tmem_ld32(tS + lane_off + 128 * bs + 64, r2);
          tmem_ld32(tS + lane_off + 128 * bs + 96, r3);
          tmem_ld_wait();
          reg_fence(r0);
          reg_fence(r1);
          reg_fence(r2);
          reg_fence(r3);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            xs[e] = __uint_as_float(r0[e]);
            xs[32 + e] = __uint_as_float(r1[e]);
            xs[64 + e] = __uint_as_float(r2[e]);
            xs[96 + e] = __uint_as_float(r3[e]);
          }
        }
        // S is in registers: the next QK into this buffer may start.
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(bs ? s_free_l1 : s_free_l0);
        if (partial || __any_sync(0xffffffffu, row_pad)) {
          // One visibility bit per key of the tile.
          uint32_t vm[4] = {~0u, ~0u, ~0u, ~0u};
          if (partial) {
            // Visible keys, as offsets in the tile: [a, e) and [0, s).
            int a, e, s;
            if (kt.chunk) {
              e = 0;                               // keys whose block the row admits: a prefix
#pragma unroll
              for (int step = kBN; step >= 1; step >>= 1) {
                const int probe = e + step;
                if (probe <= kBN && (uint32_t)(codes[k0 + probe - 1] >> 2) <= csq) e = probe;
              }
              e = min(e, p.Sq - k0);
              a = p.window > 0 ? tok - p.window + 1 - k0 : 0;
              s = p.window > 0 ? min(max(p.sinks - x.len, 0) - k0, e) : 0;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                // FAST bit (padding keys carry it too) and padding, per key
                const uint32_t ck = codes[k0 + 32 * w + lane];
                const uint32_t fw = __ballot_sync(0xffffffffu, (ck & 1u) != 0u);
                const uint32_t pw = __ballot_sync(0xffffffffu, is_pad(ck));
                vm[w] = ~(row_expert ? fw : pw);
              }
            } else {
              e = min(kBN, x.len - k0);
              a = lo - k0;
              s = sink_end - k0;
            }
#pragma unroll
            for (int w = 0; w < 4; ++w)
              vm[w] &= (bits_below(e - 32 * w) & ~bits_below(a - 32 * w)) | bits_below(s - 32 * w);
          }
          if (row_pad) vm[0] = vm[1] = vm[2] = vm[3] = 0u;
#pragma unroll
          for (int j = 0; j < kBN; ++j) xs[j] = ((vm[j >> 5] >> (j & 31)) & 1u) ? xs[j] : -INFINITY;
        }
        float m8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float a = fmax3(xs[k], xs[k + 8], xs[k + 16]);
#pragma unroll
          for (int i = 3; i < 15; i += 2) a = fmax3(a, xs[k + 8 * i], xs[k + 8 * i + 8]);
          m8[k] = fmaxf(a, xs[k + 120]);
        }
        const float mx =
            fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], fmax3(m8[4], m8[5], m8[6]), m8[7])) * c;
        // Lazy rescaling (exact: O and l always share the reference maximum).
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
        uint32_t pk[64];
#pragma unroll
        for (int e = 0; e < 64; ++e) {
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
        const bool rescale = __any_sync(0xffffffffu, need_o);
        if (rescale) {
          const float a = need_o ? alpha : 1.f;
#pragma unroll 1
          for (int cc = 0; cc < kD / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + lane_off + 32 * cc, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
            tmem_st32(tO + lane_off + 32 * cc, o);
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int sw = (j ^ (r & 7)) << 4;
          *reinterpret_cast<uint4*>(p_row0 + sw) =
              make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
          *reinterpret_cast<uint4*>(p_row1 + sw) =
              make_uint4(pk[32 + 4 * j], pk[33 + 4 * j], pk[34 + 4 * j], pk[35 + 4 * j]);
        }
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
      if (po == nullptr) {
        const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
        // P is free: each warp stages its 32 rows there, 128 columns (256
        // bytes) at a time, then writes whole half rows.
        // (A warp stays inside its own P rows: another warp may already write
        // the next segment's P.)
        uint8_t* const st = sP + warp * 4096;
        auto staged = [&](int rr, int ch) {        // row rr's 16-byte chunk ch
          return reinterpret_cast<uint4*>(st + (ch >> 3) * kPBlk + rr * 128 +
                                          (((ch & 7) ^ (rr & 7)) << 4));
        };
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int sub = 0; sub < 4; ++sub) {
            uint32_t o[32];
            tmem_ld32(tO + lane_off + 128 * half + 32 * sub, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = cvt_bf16x2(__uint_as_float(o[8 * j + 2 * e]) * inv,
                                  __uint_as_float(o[8 * j + 2 * e + 1]) * inv);
              *staged(lane, 4 * sub + j) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          if (half == 1) {                         // O has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(o_free_l);
          }
          __syncwarp();
#pragma unroll 4
          for (int it = 0; it < 16; ++it) {
            const int rr = it * 2 + (lane >> 4), ch = lane & 15;
            const long long at = __shfl_sync(0xffffffffu, orow, rr);
            const bool v = __shfl_sync(0xffffffffu, (int)row_valid, rr) != 0;
            const uint4 w = *staged(rr, ch);
            if (v)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + at * (kD * 2) + half * 256 +
                                        ch * 16) = w;
          }
          __syncwarp();
        }
        if (p.lse && row_valid)
          p.lse[orow] = l_run > 0.f ? (m_run + __log2f(l_run)) * 0.69314718055994531f
                                    : (l_run == l_run ? -INFINITY : l_run);
      } else {
        // Partial: unnormalised O and (m, l).
#pragma unroll 1
        for (int cc = 0; cc < kD / 32; ++cc) {
          uint32_t o[32];
          tmem_ld32(tO + lane_off + 32 * cc, o);
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
        if (row_valid) *reinterpret_cast<float2*>(pml) = make_float2(m_run, l_run);
      }
    }
  }

  // Neither CTA may leave while its partner can still signal its barriers or
  // read its shared memory; then both free their TMEM.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Merges the partials of units that were cut: out = sum_k 2^(m_k - M) O_k /
// sum_k 2^(m_k - M) l_k with M the largest m_k that has l_k > 0.  CTA (u, y):
// rows [32 y, 32 y + 32) of unit u, one warp per row at a time, 8 columns per
// lane.  HBM-bound: reads the fp32 partials once.
struct CombineSmem {
  long long cum[kGroup + 1];
  int max_nom;
};
__global__ void __launch_bounds__(256)
    paged_combine_kernel(const __grid_constant__ PagedTcParams p, const DevCtl ctl) {
  __shared__ CombineSmem sm;
  pdl_wait();                  // the partials come from the kernel before
  pdl_launch_dependents();
  build_schedule<256>(p, ctl, sm.cum, &sm.max_nom);
  const long long per = tiles_per_cluster(p, sm.cum[p.nb], sm.max_nom);
  if (per == 0) return;
  const int units = p.Hkv * p.n_tiles;
  const int b = (int)(blockIdx.x / units), u = (int)(blockIdx.x % units);
  const int nom = (int)((sm.cum[b + 1] - sm.cum[b]) / units);
  const long long t0 = sm.cum[b] + (long long)u * nom;
  const int c0 = (int)(t0 / per), c1 = (int)((t0 + nom - 1) / per);
  if (c0 == c1) return;        // ran whole
  const int g = u / p.n_tiles, tile = u % p.n_tiles;
  const int lane = threadIdx.x & 31;
  const float2* ml = reinterpret_cast<const float2*>(
      p.ws + (long long)p.n_clusters * 2 * kRowsTile * kD);
  for (int i = threadIdx.x >> 5; i < 32; i += 8) {
    const int row = blockIdx.y * 32 + i;
    const int tok = tile * p.tok_per_tile + row / p.G;
    if (tok >= p.Sq || row >= p.G * p.tok_per_tile) continue;
    float M = -INFINITY;
    for (int c = c0; c <= c1; ++c) {
      const float2 v = ml[(long long)(c * 2 + (c == c0 ? 1 : 0)) * kRowsTile + row];
      if (v.y > 0.f) M = fmaxf(M, v.x);
    }
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    float l = 0.f;
    for (int c = c0; c <= c1; ++c) {
      const long long at = (long long)(c * 2 + (c == c0 ? 1 : 0)) * kRowsTile + row;
      const float2 v = ml[at];
      if (!(v.y > 0.f)) {
        if (v.y == v.y) continue;            // no visible key; NaN goes on
      }
      const float w = ex2(v.x - M);
      l += w * v.y;
      const float4* src = reinterpret_cast<const float4*>(p.ws + at * kD + lane * 8);
      const float4 a = src[0], d = src[1];
      acc[0] += w * a.x; acc[1] += w * a.y; acc[2] += w * a.z; acc[3] += w * a.w;
      acc[4] += w * d.x; acc[5] += w * d.y; acc[6] += w * d.z; acc[7] += w * d.w;
    }
    const float inv = l > 0.f ? 1.f / l : (l == l ? 0.f : l);
    const long long orow = ((long long)(p.b0 + b) * p.Sq + tok) * p.Hq + (long long)g * p.G + row % p.G;
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

template <bool kE4M3, class L>
cudaError_t launch(PagedTcParams& p, const DevCtl& ctl, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(
      paged_tc_kernel<kE4M3, L>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e != cudaSuccess) return e;
  p.smem_bytes = min(layout_bytes<L>(p.Sq) + 1024, kSmemLimit);
  return launch_pdl(paged_tc_kernel<kE4M3, L>, dim3(2 * p.n_clusters), dim3(kThreads),
                    (size_t)p.smem_bytes, st, p, ctl);
}

// Whether a group of nb sequences may be cut: with four units or more per
// cluster the last round's idle clusters cost less than partials and a merge.
bool may_cut(long long n_units, int slots) { return n_units < 4ll * slots; }

int slots() { return max(sm_count() / 2, 1); }

}  // namespace

bool paged_tc_applies(const PagedParams& p) {
  const int G = p.Hq / p.Hkv;
  return !p.f32 && p.d == kD && (G == 1 || G == 2 || G == 4 || G == 8 || G == 16) &&
         (long long)p.B * p.Sq < (1ll << 31);
}

size_t paged_tc_workspace_bytes(const PagedParams& p) {
  const int G = p.Hq / p.Hkv;
  const long long units = (long long)p.Hkv * ((p.Sq + kRowsTile / G - 1) / (kRowsTile / G));
  // The last group of sequences is the smallest: it decides.
  const int last = p.B % kGroup ? p.B % kGroup : kGroup;
  if (!may_cut((p.B < kGroup ? p.B : last) * units, slots())) return 0;
  return (size_t)slots() * 2 * kRowsTile * (kD + 2) * sizeof(float);
}

cudaError_t launch_paged_tc(const PagedParams& a, float* ws, const DevCtl& ctl, cudaStream_t st) {
  PagedTcParams p;
  static_cast<PagedParams&>(p) = a;
  p.ws = ws;
  p.G = a.Hq / a.Hkv;
  p.tok_per_tile = kRowsTile / p.G;
  p.n_tiles = (a.Sq + p.tok_per_tile - 1) / p.tok_per_tile;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  for (int b0 = 0; b0 < a.B; b0 += kGroup) {
    p.b0 = b0;
    p.nb = min(kGroup, a.B - b0);
    const long long n_units = (long long)p.nb * a.Hkv * p.n_tiles;
    p.may_cut = may_cut(n_units, slots()) ? 1 : 0;
    p.n_clusters = p.may_cut ? slots() : (int)min(n_units, (long long)slots());
    const bool e4 = a.cache_dtype == kCacheE4M3;
    const bool short_s = a.Sq <= LayoutShort::kMaxTok;
    const cudaError_t e = e4 ? (short_s ? launch<true, LayoutShort>(p, ctl, st)
                                        : launch<true, LayoutLong>(p, ctl, st))
                             : (short_s ? launch<false, LayoutShort>(p, ctl, st)
                                        : launch<false, LayoutLong>(p, ctl, st));
    if (e != cudaSuccess) return e;
    if (p.may_cut) {
      const dim3 grid((unsigned)n_units, kRowsTile / 32);
      const cudaError_t c = launch_pdl(paged_combine_kernel, grid, dim3(256), 0, st, p, ctl);
      if (c != cudaSuccess) return c;
    }
  }
  return cudaSuccess;
}

}  // namespace piattn
