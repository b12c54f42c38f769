// paged_decode.cu -- attention over the paged cache when a kv head has few
// query rows (Sq * Hq / Hkv <= 8): the single-token decoding step.
//
// The work is reading the cache: every cached row feeds at most eight dot
// products, so the kernel spreads the cache over the whole GPU and keeps the
// arithmetic off the critical path with warp-level tensor instructions.
//
//  * Work is cut into 16-key tiles (never across a page), shared out on the device
//    from cache_lens, so that ragged lengths and few long sequences fill the GPU
//    alike: each sequence's tiles in equal pieces of at most `per`, one CTA a piece,
//    or, with more sequences than half the CTAs, all tiles in a row in equal
//    ranges.  (A CTA whose range crosses into another sequence starts over with its
//    queries: 4 us of 12 at 32 sequences of 880 tokens.)  A CTA's four warps take its
//    tiles in turn, each through its own 16-key stage: one TMA box per tile and
//    operand, K refilled as soon as the scores are done, V as soon as the product is.
//  * Scores transposed, S^T = K Q^T by mma.m16n8k16, so that the 8 query rows
//    fill the n8 side; an fp32 online softmax per query column; O^T += V^T P^T,
//    P^T by an in-register 8x8 transpose.
//  * e4m3 pages: ldmatrix moves pairs of bytes, so the operands' d order is
//    permuted inside groups of 16 (Q is loaded in the same order, O written
//    back in it).  K becomes fp16 by the conversion instructions and meets Q in
//    fp16 (scaled per row to below 2^15: bf16's 8 bits fit, and what falls under
//    fp16's range is 2^-39 of the row's largest); V is rebuilt as bf16 by integer
//    and bf16 instructions (paged.cuh).  Both are exact, and the two kinds of
//    instructions use different units.
//  * The warps' partials merge in shared memory.  A sequence that one CTA read
//    whole is written out; the others leave fp32 partials that a second kernel
//    merges by the log-sum-exp rule.  No atomics: the result does not depend on
//    timing.
//  * When all sequences' clusters fit at once and none is very long (clustered()),
//    a cluster of eight CTAs takes a sequence instead, in equal pieces, and merges
//    their partials over distributed shared memory: no plan, no second launch.
// The chunk's own keys (at most 8) are one more, cheap tile: a short loop of dot
// products while the first copies are in flight, kept as a fifth warp's partial.
// Code is kept short throughout: a small call waits for its instructions more
// than for its data.  Rows that no query sees are zeroed (bf16: in V's tile; e4m3:
// by their scale), so that what a stale slot holds (NaN) does not reach the result.
//
// Measured: one token of 16 sequences of 12000 to 16000 bf16 tokens 44.0 us (5.2
// TB/s, of 6.5 that a copy reaches; 49.3 in two launches), of 32 sequences of 400 to
// 880 e4m3 tokens 11.5 us (15.3), of one of 880 tokens 7.9 us (9.6).  Short calls are
// a chain of waits: launch, length, page, first tiles, merge.
#include <cfloat>
#include <cstddef>

#include "launch.h"
#include "paged.cuh"
#include "stage.h"

namespace piattn {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kRows = 8;
constexpr int kD = 256;
constexpr int kTile = 16;
constexpr int kPartStride = kD + 4;         // fp32 partial rows: 4-bank skew
constexpr int kGroup = kPagedDecodeGroup;
constexpr int kClusterCtas = 8;                // CTAs of a cluster that shares a unit
constexpr int kPerSm = 3;                   // CTAs per SM (164 registers a thread)

template <bool kE4M3>
struct Cfg {
  static constexpr int kRow = kE4M3 ? kD : 2 * kD;        // bytes of a cached row
  static constexpr int kBytes = kTile * kRow;             // one operand's tile
  static constexpr int kRing = kWarps * 2 * kBytes;
  static constexpr int kPart = kWarps * kRows * kPartStride * 4;
  static constexpr int kBody = kRing > kPart ? kRing : kPart;
};

struct Plan {
  int cum[kGroup + 1];                      // tiles, or pieces, before each sequence's units
  int len[kGroup];
  int part[kWarps];
  int per;                                  // tiles per CTA
  bool pieces;                              // units are cut one by one
};
struct Smem {
  Plan plan;
  float m[kWarps + 1][kRows];               // [kWarps]: the chunk's own keys
  float l[kWarps + 1][kRows];
  alignas(16) float o_chunk[kRows][kD];
  float2 own[kRows];                        // this CTA's (m, l) for its cluster
  uint64_t k_full[kWarps], v_full[kWarps];
  int abort;
};

static_assert(offsetof(Smem, o_chunk) % 16 == 0 && offsetof(Smem, own) % 8 == 0 &&
                  Cfg<true>::kBody % 16 == 0 &&
                  Cfg<false>::kBody % 16 == 0 && offsetof(Smem, k_full) % 8 == 0,
              "vector accesses need aligned places");

static_assert(kPerSm * (Cfg<false>::kBody + (int)sizeof(Smem) + 2048) <= 228 * 1024, "per SM");
template <bool kE4M3>
constexpr int smem_bytes() { return Cfg<kE4M3>::kBody + (int)sizeof(Smem) + 1024; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D (16x8 fp32) += A (16x16 bf16) * B (16x8 bf16).
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same in fp16.
__device__ __forceinline__ void mma16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint2 halves(uint32_t w) {   // four e4m3 as fp16
  return make_uint2(e4m3x2_to_half2((uint16_t)w), e4m3x2_to_half2((uint16_t)(w >> 16)));
}
__device__ __forceinline__ uint32_t movm_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// What a sequence's queries see of its cache: tiles [0, sink_tiles) and
// [win_tile, n_ct); lo0: the first token's window start.
struct Seen { int sink_tiles, win_tile, lo0, count; };
__device__ __forceinline__ Seen seen_tiles(const PagedDecodeParams& p, int len) {
  Seen s;
  s.lo0 = p.window > 0 ? min(max(len - p.window + 1, 0), len) : 0;
  const int n_ct = (len + kTile - 1) / kTile;
  s.sink_tiles = p.window > 0 ? (min(p.sinks, s.lo0) + kTile - 1) / kTile : 0;
  s.win_tile = max(s.lo0 / kTile, s.sink_tiles);
  s.count = s.sink_tiles + max(n_ct - s.win_tile, 0);
  return s;
}

// Tiles of a unit: its cached ones and one of the chunk's own keys.
__device__ __forceinline__ int unit_tiles_of(const PagedDecodeParams& p, int len) {
  return seen_tiles(p, len).count + 1;
}

// Block-wide: the plan, from cache_lens.  All kThreads threads call it.
__device__ void make_plan(const PagedDecodeParams& p, const DevCtl& ctl, Plan& plan) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  // cum[b + 1] = sum of count(length) over sequences 0 .. b, times the kv heads;
  // returns the total.
  auto scan = [&](auto count) -> int {
    int carry = 0;
    for (int base = 0; base < p.nb; base += kThreads) {
      const int b = base + t;
      int x = b < p.nb ? count(plan.len[b]) * p.Hkv : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      if (lane == 31) plan.part[warp] = x;
      __syncthreads();
      int before = 0, total = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? plan.part[w] : 0;
        total += plan.part[w];
      }
      if (b < p.nb) plan.cum[b + 1] = carry + before + x;
      carry += total;
      __syncthreads();
    }
    return carry;
  };
  bool bad = false;
  for (int b = t; b < p.nb; b += kThreads)
    plan.len[b] = cached_len(p.lens, p.b0 + b, p.max_pages, p.page_shift, bad);
  if (bad && blockIdx.x == 0) record_status(ctl, kStatusArg);
  __syncthreads();
  const int total = scan([&](int n) { return unit_tiles_of(p, n); });
  const int units = p.nb * p.Hkv;
  const bool pieces = 2 * units <= p.n_ctas;
  // One CTA more per unit than an even share needs: the pieces always fit.
  const int ctas = pieces ? p.n_ctas - units : p.n_ctas;
  const int per = max((total + ctas - 1) / ctas, kWarps);
  if (pieces) (void)scan([&](int n) { return (unit_tiles_of(p, n) + per - 1) / per; });
  if (t == 0) {
    plan.cum[0] = 0;
    plan.per = per;
    plan.pieces = pieces;
  }
  __syncthreads();
}

__device__ __forceinline__ int find_seq(const Plan& plan, int nb, int pos) {
  int lo = 0, hi = nb - 1;                  // largest b with cum[b] <= pos
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (plan.cum[mid] <= pos) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Shared-memory byte offset of the 16-byte chunk at byte c of row j in a tile
// of 128-byte column blocks, 128-byte swizzle.
__device__ __forceinline__ uint32_t chunk_off(int j, int c) {
  return (uint32_t)((c >> 7) * (kTile * 128) + j * 128 + ((((c >> 4) & 7) ^ (j & 7)) << 4));
}

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr)
               : "memory");
  return v;
}

// kCluster: the eight CTAs of a cluster read one unit in equal pieces and merge on
// chip.  Else CTAs follow the plan and leave partials to paged_decode_merge.
template <bool kE4M3, bool kCluster>
__global__ void __launch_bounds__(kThreads, kPerSm)
    paged_decode_kernel(const __grid_constant__ PagedDecodeParams p, const DevCtl ctl) {
  using C = Cfg<kE4M3>;
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  Smem& sm = *reinterpret_cast<Smem*>(ring + C::kBody);
  float* opart = reinterpret_cast<float*>(ring);

  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int g = lane >> 2, t4 = lane & 3;             // mma fragment coordinates
  if (t == 0) {
    for (int w = 0; w < kWarps; ++w) {
      mbar_init(&sm.k_full[w], 1);
      mbar_init(&sm.v_full[w], 1);
    }
    sm.abort = 0;
    fence_barrier_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  const int cta = (int)blockIdx.x;
  int per = 0, pos = 0, end = 1;
  bool pieces = true;
  if constexpr (kCluster) {
    __syncthreads();                                  // the barriers exist
  } else {
    make_plan(p, ctl, sm.plan);
    per = sm.plan.per;
    pieces = sm.plan.pieces;
    const int total = sm.plan.cum[p.nb];
    // Tiles [pos, end) of all, or this CTA's piece.
    pos = pieces ? cta : (int)min((long long)cta * per, (long long)total);
    end = pieces ? min(cta + 1, total) : min(pos + per, total);
  }
  const int R = p.Sq * p.G;
  const float sl2 = p.scale_log2;
  const uint32_t kt = smem_u32(ring + warp * 2 * C::kBytes), vt = kt + C::kBytes;
  uint32_t n_load = 0;                                // tiles this warp has loaded by TMA
  bool bad = false;
  Stuck stuck = Stuck::kNo;

  while (pos < end) {
    // ------------------------------------------------- the segment
    const int b = kCluster ? cta / kClusterCtas / p.Hkv : find_seq(sm.plan, p.nb, pos);
    const int len = kCluster ? cached_len(p.lens, b, p.max_pages, p.page_shift, bad)
                             : sm.plan.len[b];
    const Seen sn = seen_tiles(p, len);
    const int unit_tiles = sn.count + 1;
    const int rem = kCluster ? cta / kClusterCtas % p.Hkv : pos - sm.plan.cum[b];
    int h, i0, i1;
    if constexpr (kCluster) {
      const int c = cta % kClusterCtas;
      h = rem;
      i0 = (int)((long long)c * unit_tiles / kClusterCtas);
      i1 = (int)((long long)(c + 1) * unit_tiles / kClusterCtas);
      ++pos;
    } else if (pieces) {
      const int n = (unit_tiles + per - 1) / per;
      h = rem / n;
      i0 = (int)((long long)(rem - h * n) * unit_tiles / n);
      i1 = (int)((long long)(rem - h * n + 1) * unit_tiles / n);
      ++pos;
    } else {
      h = rem / unit_tiles;
      i0 = rem - h * unit_tiles;
      i1 = min(unit_tiles, i0 + (end - pos));
      pos += i1 - i0;
    }
    const int bb = p.b0 + b;
    const int32_t* table = p.table + (long long)bb * p.max_pages;

    auto tile_at = [&](int i) {                       // the unit's i-th cached tile
      return i < sn.sink_tiles ? i : sn.win_tile + i - sn.sink_tiles;
    };
    // First row (slot) of cached tile i; past the pool (TMA fills zeros) for a
    // page id out of range.
    auto slot_at = [&](int i) -> int {
      const int x = tile_at(i) * kTile;
      const int page = table[x >> p.page_shift];
      if (page >= 0 && page < p.num_pages)
        return (page << p.page_shift) + (x & ((1 << p.page_shift) - 1));
      bad = true;
      return p.num_pages << p.page_shift;
    };
    auto load_tile = [&](const CUtensorMap* map, uint64_t* bar, uint32_t dst, int slot) {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, C::kBytes);
        tma_load_3d_at(dst, map, bar, 0, slot, h * (C::kRow / 128));
      }
    };
    // e4m3: lane l has the exponents of rows l (K) and l - 16 (V) of a tile.
    auto exp_at = [&](int slot) -> uint32_t {
      if (!kE4M3 || slot >= p.num_pages << p.page_shift) return kNoExp;
      const uint8_t* e = lane < 16 ? p.ke : p.ve;
      return (uint32_t)e[((long long)slot + (lane & 15)) * p.Hkv + h];
    };

    // First loads: this warp's tile i0 + warp, if it is a cached one.
    int i = i0 + warp;
    int slot = 0;
    uint32_t ex = kNoExp;
    if (i < i1 && i < sn.count) {
      slot = slot_at(i);
      load_tile(&p.map_k, &sm.k_full[warp], kt, slot);
      load_tile(&p.map_v, &sm.v_full[warp], vt, slot);
      ex = exp_at(slot);
    }
    // The chunk's codes, in lanes 0 .. Sq - 1.
    uint32_t code = 3u;                               // no such token: acts as padding
    {
      const long long at = (long long)bb * p.mask_bs + lane;
      const bool in = lane < p.Sq;
      const uint32_t on = __ballot_sync(0xffffffffu, in && p.ar[at] != 0);
      if (in) code = make_code(__popc(on & (0xffffffffu >> (31 - lane))), p.seg ? p.seg[at] : 0);
    }
    const long long q0 = ((long long)bb * p.Sq * p.Hq + (long long)h * p.G) * kD;
    auto q_row = [&](int r) {                         // row r of the unit's queries
      return static_cast<const __nv_bfloat16*>(p.q) + q0 +
             ((long long)(r >> p.g_shift) * p.Hq + (r & (p.G - 1))) * kD;
    };
    // The chunk's own keys fall to the CTA that has the unit's last tile: warp w has
    // rows w and w + 4, a lane 8 columns.  Their loads go out now.
    const bool chunk = i1 == unit_tiles;
    const int rw[2] = {min(warp, R - 1), min(warp + kWarps, R - 1)};
    const __nv_bfloat16* kn = static_cast<const __nv_bfloat16*>(p.k);
    const __nv_bfloat16* vn = static_cast<const __nv_bfloat16*>(p.v);
    const long long n0 = ((long long)bb * p.Sq * p.Hkv + h) * kD + lane * 8;
    const long long n_step = (long long)p.Hkv * kD;
    uint4 cq[2], ck, cv;
    if (chunk) {
      cq[0] = *reinterpret_cast<const uint4*>(q_row(rw[0]) + lane * 8);
      cq[1] = *reinterpret_cast<const uint4*>(q_row(rw[1]) + lane * 8);
      ck = *reinterpret_cast<const uint4*>(kn + n0);
      cv = *reinterpret_cast<const uint4*>(vn + n0);
    }
    // Q^T as the B operand, straight from global memory: bf16: lane (g, t4)
    // holds Q[g][16 kk + 2 t4 ..] and Q[g][16 kk + 8 + 2 t4 ..]; e4m3: Q[g][16 kk
    // + 4 t4 ..] and the two after, as fp16 times a power of two.
    uint32_t qb[16][2];
    float qf0 = sl2, qf1 = sl2;                       // what a score of this lane's rows lacks
    {
      const uint32_t* qg = reinterpret_cast<const uint32_t*>(q_row(g < R ? g : 0));
#pragma unroll
      for (int kk = 0; kk < 16; ++kk) {
        if constexpr (kE4M3) {
          const uint2 v = *reinterpret_cast<const uint2*>(qg + 8 * kk + 2 * t4);
          qb[kk][0] = v.x;
          qb[kk][1] = v.y;
        } else {
          qb[kk][0] = qg[8 * kk + t4];
          qb[kk][1] = qg[8 * kk + 4 + t4];
        }
      }
      if constexpr (kE4M3) {
        uint32_t top = 0;                             // the row's largest exponent
#pragma unroll
        for (int kk = 0; kk < 16; ++kk)
          top = max(max(top, max(qb[kk][0] & 0x7F80u, (qb[kk][0] >> 16) & 0x7F80u)),
                    max(qb[kk][1] & 0x7F80u, (qb[kk][1] >> 16) & 0x7F80u));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // times 2^(14 - e): the largest element falls in [2^14, 2^15)
        const int e = max((int)(top >> 7), 15) - 127;
        const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
#pragma unroll
        for (int kk = 0; kk < 16; ++kk) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t w = qb[kk][x];
            asm("cvt.rn.f16x2.f32 %0, %1, %2;"
                : "=r"(qb[kk][x])
                : "f"(__uint_as_float(w & 0xFFFF0000u) * up), "f"(__uint_as_float(w << 16) * up));
          }
        }
        const float down = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
        qf0 *= __shfl_sync(0xffffffffu, down, 8 * t4);          // rows 2 t4 and 2 t4 + 1
        qf1 *= __shfl_sync(0xffffffffu, down, 8 * t4 + 4);
      }
    }
    if (chunk) {
      float acc[2][8], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[u][c] = 0.f;
#pragma unroll 1
      for (int j = 0; j < p.Sq; ++j) {
        float k[8], v[8];
        unpack8(ck, k);
        unpack8(cv, v);
        if (j + 1 < p.Sq) {
          ck = *reinterpret_cast<const uint4*>(kn + n0 + (j + 1) * n_step);
          cv = *reinterpret_cast<const uint4*>(vn + n0 + (j + 1) * n_step);
        }
        const uint32_t code_j = __shfl_sync(0xffffffffu, code, j);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int tq = rw[u] >> p.g_shift;
          const uint32_t code_q = __shfl_sync(0xffffffffu, code, tq);
          if (!visible(code_q, code_j) || !in_window(len, tq, j, p.window, p.sinks)) continue;
          float q[8], sc = 0.f;
          unpack8(cq[u], q);
#pragma unroll
          for (int c = 0; c < 8; ++c) sc = fmaf(q[c], k[c], sc);
#pragma unroll
          for (int sh = 16; sh >= 1; sh >>= 1) sc += __shfl_xor_sync(0xffffffffu, sc, sh);
          sc *= sl2;
          const float mn = fmaxf(m[u], sc), f = m[u] == -INFINITY ? 0.f : ex2(m[u] - mn);
          const float w = sc == -INFINITY ? 0.f : ex2(sc - mn);     // (mn may be -inf too)
          l[u] = l[u] * f + w;
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[u][c] = fmaf(acc[u][c], f, w * v[c]);
          m[u] = mn;
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = warp + u * kWarps;
        if (r < R) {
          float4* dst = reinterpret_cast<float4*>(&sm.o_chunk[r][lane * 8]);
          dst[0] = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
          dst[1] = make_float4(acc[u][4], acc[u][5], acc[u][6], acc[u][7]);
          if (lane == 0) {
            sm.m[kWarps][r] = m[u];
            sm.l[kWarps][r] = l[u];
          }
        }
      }
    }
    const int qr0 = 2 * t4, qr1 = 2 * t4 + 1;         // this lane's query rows
    const int tk0 = qr0 >> p.g_shift, tk1 = qr1 >> p.g_shift;
    const uint32_t code0 = __shfl_sync(0xffffffffu, code, tk0);
    const uint32_t code1 = __shfl_sync(0xffffffffu, code, tk1);
    const bool row0_ok = qr0 < R && !is_pad(code0), row1_ok = qr1 < R && !is_pad(code1);
    // No query sees a cached position before lo_live: padding in front sees nothing.
    const uint32_t real = __ballot_sync(0xffffffffu, !is_pad(code));
    const int lo_live =
        p.window > 0 ? min(max(len + max(__ffs(real) - 1, 0) - p.window + 1, 0), len) : 0;
    const int lo_a = p.window > 0 ? min(max(len + tk0 - p.window + 1, 0), len) : 0;
    const int lo_b = p.window > 0 ? min(max(len + tk1 - p.window + 1, 0), len) : 0;
    // O^T [256 x 8 rows]: 16 column blocks of m16n8k16.
    float o[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

#pragma unroll 1
    for (; i < min(i1, sn.count); i += kWarps) {
      const int k0 = tile_at(i) * kTile;
      const int nx = i + kWarps;
      const bool more = nx < i1 && nx < sn.count;
      const int next_slot = more ? slot_at(nx) : 0;
      // Keys that some query sees; all of them in most tiles.
      uint32_t live = 0xFFFFu;
      const bool whole = __all_sync(0xffffffffu, k0 + kTile <= len && (p.window <= 0 || k0 >= lo_b ||
                                                                       k0 + kTile <= p.sinks));
      if (!whole) {
        const int x = k0 + (lane & 15);
        live = __ballot_sync(0xffffffffu, x < len && (p.window <= 0 || x >= lo_live || x < p.sinks)) &
               0xFFFFu;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.k_full[warp], n_load & 1, ctl))) {
        sm.abort = 1;
        stuck = Stuck::kAtK;
        break;
      }
      // sc[0]: key g, row qr0; [1]: g, qr1; [2], [3]: key g + 8.
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
      const int lrow = 8 * ((lane >> 3) & 1) + (lane & 7);       // ldmatrix row
      const uint32_t kl = kt + lrow * 128, ks = lrow & 7;
      if constexpr (kE4M3) {
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          // two 16-byte chunks of the 16 rows: 4 bytes of d per lane and row
          uint32_t r[4];
          ldsm_x4(kl + (c >> 3) * (kTile * 128) + ((((c & 7) + (lane >> 4)) ^ ks) << 4), r);
          const uint2 a = halves(r[0]), e = halves(r[1]), f = halves(r[2]), w = halves(r[3]);
          mma16816_f16(sa, a.x, e.x, a.y, e.y, qb[c][0], qb[c][1]);
          mma16816_f16(sb, f.x, w.x, f.y, w.y, qb[c + 1][0], qb[c + 1][1]);
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < 16; ++kk) {
          uint32_t r[4];
          ldsm_x4(kl + (kk >> 2) * (kTile * 128) + (((2 * (kk & 3) + (lane >> 4)) ^ ks) << 4), r);
          if (kk & 1) mma16816(sb, r[0], r[1], r[2], r[3], qb[kk][0], qb[kk][1]);
          else mma16816(sa, r[0], r[1], r[2], r[3], qb[kk][0], qb[kk][1]);
        }
      }
      __syncwarp();                                   // K has been read
      if (more) load_tile(&p.map_k, &sm.k_full[warp], kt, next_slot);
      float fg = 1.f, fh = 1.f;                       // e4m3: the keys' scales
      if constexpr (kE4M3) {
        const float f = ex == kNoExp ? 0.f : exp_scale(ex);
        fg = __shfl_sync(0xffffffffu, f, g);
        fh = __shfl_sync(0xffffffffu, f, g + 8);
      }
      float sc[4] = {(sa[0] + sb[0]) * qf0 * fg, (sa[1] + sb[1]) * qf1 * fg,
                     (sa[2] + sb[2]) * qf0 * fh, (sa[3] + sb[3]) * qf1 * fh};
      if (!whole) {
        auto sees = [&](int x, int lo) {
          return x < len && (p.window <= 0 || x >= lo || x < p.sinks);
        };
        sc[0] = sees(k0 + g, lo_a) ? sc[0] : -INFINITY;
        sc[1] = sees(k0 + g, lo_b) ? sc[1] : -INFINITY;
        sc[2] = sees(k0 + g + 8, lo_a) ? sc[2] : -INFINITY;
        sc[3] = sees(k0 + g + 8, lo_b) ? sc[3] : -INFINITY;
      }
      if (!row0_ok) sc[0] = sc[2] = -INFINITY;
      if (!row1_ok) sc[1] = sc[3] = -INFINITY;
      // Column maxima over the 16 keys: the 8 lanes of equal t4.
      float x0 = fmaxf(sc[0], sc[2]), x1 = fmaxf(sc[1], sc[3]);
#pragma unroll
      for (int sh = 4; sh <= 16; sh <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, sh));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, sh));
      }
      // Lazy rescaling: the references move only when a maximum grows by more
      // than 8 (log2 units), so p stays <= 256.
      const bool up0 = x0 > m0 + 8.f, up1 = x1 > m1 + 8.f;
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float n0 = up0 ? x0 : m0, n1 = up1 ? x1 : m1;
        const float a0 = m0 == -INFINITY ? 0.f : ex2(m0 - n0), a1 = m1 == -INFINITY ? 0.f : ex2(m1 - n1);
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          o[n][0] *= a0;
          o[n][1] *= a1;
          o[n][2] *= a0;
          o[n][3] *= a1;
        }
        m0 = n0;
        m1 = n1;
      }
      const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
      float pa0 = ex2(sc[0] - r0), pa1 = ex2(sc[1] - r1);
      float pb0 = ex2(sc[2] - r0), pb1 = ex2(sc[3] - r1);
      l0 += pa0 + pb0;
      l1 += pa1 + pb1;
      uint32_t m_lo = 0, m_hi = 0;                    // e4m3: V's scales, two keys each
      if constexpr (kE4M3) {
        // lane l: exponent of V row l; rows that nobody sees get scale 0
        const uint32_t ev = __shfl_sync(0xffffffffu, ex, 16 + (lane & 15));
        const uint32_t mv = (live >> (lane & 15)) & 1u ? main_scale(ev) : 0u;
        m_lo = __byte_perm(__shfl_sync(0xffffffffu, mv, 2 * t4),
                           __shfl_sync(0xffffffffu, mv, 2 * t4 + 1), 0x5410);
        m_hi = __byte_perm(__shfl_sync(0xffffffffu, mv, 2 * t4 + 8),
                           __shfl_sync(0xffffffffu, mv, 2 * t4 + 9), 0x5410);
        // what a scale above 2^7 lacks goes to the probabilities (<= 2^8 * 2^113)
        const bool big = ev > 134u && ev < 255u;
        if (__any_sync(0xffffffffu, big)) {
          const float f = big ? exp_scale(ev - 7u) : 1.f;
          const float vg = __shfl_sync(0xffffffffu, f, g), vh = __shfl_sync(0xffffffffu, f, g + 8);
          pa0 *= vg;
          pa1 *= vg;
          pb0 *= vh;
          pb1 *= vh;
        }
      }
      // P^T as the B operand of O^T += V^T P^T: lane (g, t4) needs P[row g][keys 2 t4,
      // + 1] (and + 8) and holds P[keys g, g + 8][rows 2 t4, + 1].
      const uint32_t pb_lo = movm_trans(cvt_bf16x2(pa0, pa1));
      const uint32_t pb_hi = movm_trans(cvt_bf16x2(pb0, pb1));
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.v_full[warp], n_load & 1, ctl))) {
        sm.abort = 1;
        stuck = more ? Stuck::kAtVAhead : Stuck::kAtV;
        break;
      }
      if constexpr (kE4M3) {
        const uint32_t vl = vt + lrow * 128;
#pragma unroll
        for (int n = 0; n < 16; n += 2) {
          // keys 0-7 and 8-15 of two 16-byte chunks, transposed: per lane a pair of
          // d of two keys; row g of the product is d = 16 n + 2 g, row g + 8 the one
          // after
          uint32_t r[4];
          ldsm_x4_t(vl + (n >> 3) * (kTile * 128) + ((((n & 7) + (lane >> 4)) ^ ks) << 4), r);
          const uint2 a = dequant4_t(r[0], m_lo, p.spread), e = dequant4_t(r[1], m_hi, p.spread);
          const uint2 f = dequant4_t(r[2], m_lo, p.spread), w = dequant4_t(r[3], m_hi, p.spread);
          mma16816(o[n], a.x, a.y, e.x, e.y, pb_lo, pb_hi);
          mma16816(o[n + 1], f.x, f.y, w.x, w.y, pb_lo, pb_hi);
        }
      } else {
        if (!whole) {                                 // zero the rows nobody sees
#pragma unroll 1
          for (int j = 0; j < kTile; ++j)
            if (!((live >> j) & 1u))
              st_shared_v4(vt + chunk_off(j, lane * 16), make_uint4(0u, 0u, 0u, 0u));
          __syncwarp();
        }
        const int vrow = 8 * (lane >> 4) + (lane & 7);
        const uint32_t vl = vt + vrow * 128, vs = vrow & 7;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          uint32_t r[4];
          ldsm_x4_t(vl + (n >> 2) * (kTile * 128) + (((2 * (n & 3) + ((lane >> 3) & 1)) ^ vs) << 4), r);
          mma16816(o[n], r[0], r[1], r[2], r[3], pb_lo, pb_hi);
        }
        if (!whole) fence_proxy_async_smem();         // TMA may write the rows next
      }
      __syncwarp();                                   // V has been read
      ++n_load;
      if (more) {
        load_tile(&p.map_v, &sm.v_full[warp], vt, next_slot);
        ex = exp_at(next_slot);
      }
    }
    // ------------------------------------ warp partials -> the segment's
#pragma unroll
    for (int sh = 4; sh <= 16; sh <<= 1) {            // row sums over equal t4
      l0 += __shfl_xor_sync(0xffffffffu, l0, sh);
      l1 += __shfl_xor_sync(0xffffffffu, l1, sh);
    }
    __syncthreads();                                  // every warp's ring is idle
    if (sm.abort) break;                              // (a timeout: nothing more is loaded)
    {
      float* ow = opart + warp * kRows * kPartStride;
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const int da = 16 * n + (kE4M3 ? 2 * g : g), db = kE4M3 ? da + 1 : da + 8;
        ow[qr0 * kPartStride + da] = o[n][0];
        ow[qr1 * kPartStride + da] = o[n][1];
        ow[qr0 * kPartStride + db] = o[n][2];
        ow[qr1 * kPartStride + db] = o[n][3];
      }
      if (g == 0) {
        sm.m[warp][qr0] = m0;
        sm.m[warp][qr1] = m1;
        sm.l[warp][qr0] = l0;
        sm.l[warp][qr1] = l1;
      }
    }
    __syncthreads();
    {
      // Thread t: row t / 16, columns 4 (t % 16) + 64 k (k < 4): consecutive
      // 16-byte pieces across the lanes.
      const int r = t >> 4, c0 = (t & 15) * 4;
      const int parts = chunk && r < R ? kWarps + 1 : kWarps;
      float mw[kWarps + 1], lw[kWarps + 1], M = -INFINITY;
#pragma unroll
      for (int w = 0; w <= kWarps; ++w) {
        mw[w] = w < parts ? sm.m[w][r] : -INFINITY;
        lw[w] = w < parts ? sm.l[w][r] : 0.f;
        M = fmaxf(M, mw[w]);
      }
      float4 acc[4];
      float L = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w <= kWarps; ++w) {
        if (lw[w] == 0.f) continue;                   // no visible key (O may hold 0 * inf)
        const float f = lw[w] > 0.f ? ex2(mw[w] - M) : 1.f;      // NaN goes on
        L += f * lw[w];
        const float* src = w < kWarps ? opart + (w * kRows + r) * kPartStride + c0 : &sm.o_chunk[r][c0];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 x = *reinterpret_cast<const float4*>(src + 64 * k);
          acc[k].x += f * x.x;
          acc[k].y += f * x.y;
          acc[k].z += f * x.z;
          acc[k].w += f * x.w;
        }
      }
      if constexpr (kCluster) {
        __syncthreads();                              // the warps' partials have been read
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float4*>(opart + r * kD + c0 + 64 * k) = acc[k];
        if (c0 == 0) sm.own[r] = make_float2(M, L);
      } else if (r < R) {
        if (i0 == 0 && i1 == unit_tiles) {
          const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);
          const long long row = ((long long)bb * p.Sq + (r >> p.g_shift)) * p.Hq +
                                (long long)h * p.G + (r & (p.G - 1));
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + row * kD + c0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint2*>(dst + 64 * k) =
                make_uint2(cvt_bf16x2(acc[k].x * inv, acc[k].y * inv),
                           cvt_bf16x2(acc[k].z * inv, acc[k].w * inv));
          if (p.lse && c0 == 0)
            p.lse[row] = L > 0.f ? (M + __log2f(L)) * 0.69314718055994531f : (L == L ? -INFINITY : L);
        } else {
          // A piece: slot 0.  A range that begins mid-unit is its CTA's first: slot 0,
          // else slot 1.
          const long long at = ((long long)cta * 2 + (pieces || i0 > 0 ? 0 : 1)) * kRows + r;
          float* dst = p.ws + at * kD + c0;
#pragma unroll
          for (int k = 0; k < 4; ++k) *reinterpret_cast<float4*>(dst + 64 * k) = acc[k];
          if (c0 == 0)
            *reinterpret_cast<float2*>(p.ws + (long long)p.n_ctas * 2 * kRows * kD + at * 2) =
                make_float2(M, L);
        }
      }
    }
    fence_proxy_async_smem();                         // TMA writes the ring next
    __syncthreads();
  }
  if (bad) record_status(ctl, kStatusArg);
  if constexpr (kCluster) {
    // CTA c merges columns [32 c, 32 c + 32) of the eight partials: thread t row
    // t / 16, two columns.
    if (sm.abort && t < kRows) sm.own[t] = make_float2(-INFINITY, 0.f);
    __syncwarp();
    cluster_sync();
    const int r = t >> 4, c = cta % kClusterCtas, col = 32 * c + (t & 15) * 2;
    const int b = cta / kClusterCtas / p.Hkv, h = cta / kClusterCtas % p.Hkv;
    const uint32_t src = smem_u32(opart + r * kD + col), own = smem_u32(&sm.own[r]);
    float2 ml[kClusterCtas], x[kClusterCtas];
#pragma unroll
    for (int k = 0; k < kClusterCtas; ++k) {
      ml[k] = ld_cluster_f32x2(mapa_shared(own, (uint32_t)k));
      x[k] = ld_cluster_f32x2(mapa_shared(src, (uint32_t)k));
    }
    float M = -INFINITY, L = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
    for (int k = 0; k < kClusterCtas; ++k) M = fmaxf(M, ml[k].y > 0.f ? ml[k].x : -INFINITY);
#pragma unroll
    for (int k = 0; k < kClusterCtas; ++k) {
      if (ml[k].y == 0.f) continue;                   // no visible key
      const float w = ml[k].y > 0.f ? ex2(ml[k].x - M) : 1.f;    // NaN goes on
      L += w * ml[k].y;
      a0 += w * x[k].x;
      a1 += w * x[k].y;
    }
    if (r < R) {
      const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);
      const long long row = ((long long)b * p.Sq + (r >> p.g_shift)) * p.Hq + (long long)h * p.G +
                            (r & (p.G - 1));
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + row * kD + col) =
          cvt_bf16x2(a0 * inv, a1 * inv);
      if (p.lse && col == 0)
        p.lse[row] =
            L > 0.f ? (M + __log2f(L)) * 0.69314718055994531f : (L == L ? -INFINITY : L);
    }
    __syncwarp();
    cluster_sync();                                   // the others may still read this CTA's
  }
  // After a timeout: a bounded wait for this warp's copies in flight.
  if (stuck != Stuck::kNo && lane == 0) {
    const StagePhases last = last_phases(n_load, stuck);
    (void)mbar_wait(&sm.k_full[warp], last.k, ctl);
    (void)mbar_wait(&sm.v_full[warp], last.v, ctl);
  }
}

// Merges the partials of the units that several CTAs read: CTA (unit, row), two
// groups of 64 threads (4 columns each) that share out the pieces; a thread has
// eight pieces' loads in flight.
constexpr int kMergeFlight = 8;
__global__ void __launch_bounds__(kThreads)
    paged_decode_merge(const __grid_constant__ PagedDecodeParams p, const DevCtl ctl) {
  __shared__ Plan plan;
  __shared__ alignas(16) float s_acc[64][4];
  __shared__ float s_l;
  pdl_wait();                  // the partials come from the kernel before
  pdl_launch_dependents();
  make_plan(p, ctl, plan);
  const int per = plan.per;
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  const int n = (plan.cum[b + 1] - plan.cum[b]) / p.Hkv;    // the unit's pieces or tiles
  const int t0 = plan.cum[b] + h * n;
  const int c0 = plan.pieces ? t0 : t0 / per, c1 = plan.pieces ? t0 + n - 1 : (t0 + n - 1) / per;
  if (c0 == c1) return;        // read whole
  const int first = plan.pieces ? 0 : 1;       // slot of the unit's first range
  const int r = blockIdx.y;
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 6, col = (threadIdx.x & 63) * 4;
  const float2* ml = reinterpret_cast<const float2*>(p.ws + (long long)p.n_ctas * 2 * kRows * kD);
  auto slot = [&](int c) { return ((long long)c * 2 + (c == c0 ? first : 0)) * kRows + r; };
  float2 v[kMergeFlight];
  float4 x[kMergeFlight];
  auto fetch = [&](int cb) {
#pragma unroll
    for (int i = 0; i < kMergeFlight; ++i) {
      const int c = min(cb + 2 * i, c1);
      v[i] = ml[slot(c)];
      x[i] = *reinterpret_cast<const float4*>(p.ws + slot(c) * kD + col);
    }
  };
  fetch(c0 + grp);             // under way while the maximum is found
  float M = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32) {
    const float2 w = ml[slot(c)];
    if (w.y > 0.f) M = fmaxf(M, w.x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, L = 0.f;
  for (int cb = c0 + grp; cb <= c1; cb += 2 * kMergeFlight) {
    if (cb != c0 + grp) fetch(cb);
#pragma unroll
    for (int i = 0; i < kMergeFlight; ++i) {
      // none left, or no visible key (O may hold 0 * inf); NaN goes on
      if (cb + 2 * i > c1 || v[i].y == 0.f) continue;
      const float w = v[i].y > 0.f ? ex2(v[i].x - M) : 1.f;
      L += w * v[i].y;
      acc[0] += w * x[i].x;
      acc[1] += w * x[i].y;
      acc[2] += w * x[i].z;
      acc[3] += w * x[i].w;
    }
  }
  if (grp == 1) {
    *reinterpret_cast<float4*>(s_acc[threadIdx.x & 63]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if (col == 0) s_l = L;
  }
  __syncthreads();
  if (grp == 1) return;
  const float4 o = *reinterpret_cast<const float4*>(s_acc[threadIdx.x]);
  L += s_l;
  const float inv = L > 0.f ? 1.f / L : (L == L ? 0.f : L);
  const long long row = ((long long)(p.b0 + b) * p.Sq + (r >> p.g_shift)) * p.Hq +
                        (long long)h * p.G + (r & (p.G - 1));
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * kD + col) =
      make_uint2(cvt_bf16x2((acc[0] + o.x) * inv, (acc[1] + o.y) * inv),
                 cvt_bf16x2((acc[2] + o.z) * inv, (acc[3] + o.w) * inv));
  if (p.lse && col == 0)
    p.lse[row] = L > 0.f ? (M + __log2f(L)) * 0.69314718055994531f : (L == L ? -INFINITY : L);
}

bool encode_pool(CUtensorMap* map, const void* base, const PagedParams& p, bool e4m3) {
  auto fn = encode_fn();
  if (!fn) return false;
  // [slots][Hkv][row] as (128 bytes, slots, column blocks), 16 rows of one head a box
  const cuuint64_t row = e4m3 ? kD : 2 * kD, blocks = row / 128;
  cuuint64_t dims[3] = {e4m3 ? 128ull : 64ull, (cuuint64_t)p.num_pages << p.page_shift,
                        blocks * (cuuint64_t)p.Hkv};
  cuuint64_t strides[2] = {row * (cuuint64_t)p.Hkv, 128};
  cuuint32_t box[3] = {e4m3 ? 128u : 64u, (cuuint32_t)kTile, (cuuint32_t)blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sequences per launch: at most kGroup, their tiles below 2^31.
int group_size(const PagedParams& p) {
  const long long tiles = (((long long)p.max_pages << p.page_shift) / kTile + 2) * p.Hkv;
  const long long n = ((1ll << 31) - 1) / tiles;
  return (int)min(n, (long long)kGroup);
}

template <bool kE4M3, bool kCluster>
cudaError_t launch(const PagedDecodeParams& p, const DevCtl& ctl, cudaStream_t st) {
  auto* kernel = paged_decode_kernel<kE4M3, kCluster>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             smem_bytes<kE4M3>());
  if (e != cudaSuccess) return e;
  // Three CTAs an SM need the whole carve-out.
  const cudaError_t c = cudaFuncSetAttribute(
      kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (c != cudaSuccess) return c;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n_ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem_bytes<kE4M3>();
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {kClusterCtas, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, ctl);
}

// Whether a cluster takes each unit: all clusters are resident at once, and the
// longest cache that the page table can hold is neither too long for eight CTAs nor,
// with few units, worth spreading over more.  An e4m3 tile is half the bytes of a bf16
// one and more instructions, so that eight CTAs are the limit sooner.  Measured, split
// in two launches / a cluster each, us, lengths from half to all of the stated one:
//   bf16, 1 sequence of 880 10.4 / 8.3, 4000 12.3 / 11.7, 8000 16.4 / 17.8; 2 of 12000
//   24.5 / 22.3; 4 of 8000 23.6 / 18.9, 12000 25.5 / 23.5, 14000 24.5 / 27.4; 8 of 12000
//   28.5 / 28.0, 16000 33.1 / 35.5; 12 of 16000 39.4 / 37.6; 16 of 880 13.0 / 9.5, 16000
//   45.3 / 42.0, 32000 72.8 / 75.7; 32 of 880 14.7 / 11.5, 16000 71.4 / 70.5; 55 of 2000
//   26.0 / 27.6; 64 of 880 19.7 / 22.7, 128 of 880 27 / 34.
//   e4m3, 1 of 880 10.5 / 8.6, 2000 11.3 / 11.0, 3000 12.3 / 12.6; 2 of 3000 13.6 / 13.4,
//   6000 17.0 / 19.6; 4 of 5000 20.4 / 18.2, 8000 23.6 / 24.8; 16 of 3000 19.2 / 15.4, 5000
//   21.9 / 22.4, 16000 36.6 / 56.4; 32 of 880 15.3 / 11.5, 5000 27.0 / 26.7, 16000 52.5 /
//   68.2; 44 of 4000 28.1 / 24.2; 55 of 1500 20.2 / 22.9.
bool clustered(const PagedParams& p) {
  const long long units = (long long)p.B * p.Hkv;
  long long n = (long long)p.max_pages << p.page_shift;
  if (p.window > 0) n = min(n, (long long)p.window + p.sinks);
  const long long longest = p.cache_dtype == kCacheE4M3
                                ? min(2000 * units, 5120ll)
                                : min(5000 * units, units < 12 ? 12288ll : 16384ll);
  return units * kClusterCtas <= (long long)sm_count() * kPerSm && n <= longest;
}

}  // namespace

// (A pool without pages has no tensor map; the tensor-core kernel takes it.)
bool paged_decode_applies(const PagedParams& p) {
  const int G = p.Hq / p.Hkv;
  return !p.f32 && p.d == kD && (G == 1 || G == 2 || G == 4 || G == 8) && p.Sq * G <= kRows &&
         p.num_pages > 0 && group_size(p) >= 1;
}

size_t paged_decode_workspace_bytes(const PagedParams& p) {
  if (clustered(p)) return 0;
  return (size_t)sm_count() * kPerSm * 2 * kRows * (kD + 2) * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedParams& a, float* ws, const DevCtl& ctl,
                                cudaStream_t st) {
  PagedDecodeParams p{};
  static_cast<PagedParams&>(p) = a;
  p.ws = ws;
  p.G = a.Hq / a.Hkv;
  p.g_shift = p.G == 1 ? 0 : p.G == 2 ? 1 : p.G == 4 ? 2 : 3;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.spread = {16u, 240u};
  const bool e4 = a.cache_dtype == kCacheE4M3;
  if (!encode_pool(&p.map_k, a.kp, a, e4) || !encode_pool(&p.map_v, a.vp, a, e4))
    return cudaErrorUnknown;
  if (clustered(a)) {
    p.nb = a.B;
    p.n_ctas = a.B * a.Hkv * kClusterCtas;
    return e4 ? launch<true, true>(p, ctl, st) : launch<false, true>(p, ctl, st);
  }
  const int group = group_size(a);
  for (int b0 = 0; b0 < a.B; b0 += group) {
    p.b0 = b0;
    p.nb = min(group, a.B - b0);
    p.n_ctas = sm_count() * kPerSm;
    const cudaError_t e = e4 ? launch<true, false>(p, ctl, st) : launch<false, false>(p, ctl, st);
    if (e != cudaSuccess) return e;
    const cudaError_t m = launch_pdl(paged_decode_merge,
                                     dim3((unsigned)(p.nb * a.Hkv), (unsigned)(a.Sq * p.G)),
                                     dim3(kThreads), 0, st, p, ctl);
    if (m != cudaSuccess) return m;
  }
  return cudaSuccess;
}

}  // namespace piattn
