// paged.cuh -- what the paged-cache kernels share: parameters, the e4m3
// conversions, and the rules that turn cached lengths, the page table and the
// sliding window into slots and visible key ranges.
#pragma once
#include <cstdint>

#include "common.cuh"
#include "mask.cuh"

namespace piattn {

constexpr int kStatusArg = 1;        // device-side: a bad length or page id

constexpr int kCacheBF16 = 0, kCacheF32 = 1, kCacheE4M3 = 2;   // enum pi_dtype

struct E4M3 { uint8_t bits; };

// Two e4m3 values (low byte first) as floats; every e4m3 value is exact in fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return h;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {
  const uint32_t h = e4m3x2_to_half2(v);
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// lo, hi rounded to nearest e4m3 (ties to even, saturating at 448, NaN kept).
__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 2^(byte - 127): exact; byte 0 is 2^-127 (subnormal), byte 255 NaN.
__device__ __forceinline__ float exp_scale(uint32_t byte) {
  return byte == 0 ? __uint_as_float(0x00400000u)
                   : byte == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

// e4m3 -> bf16, exact.  A byte's exponent and mantissa moved to bf16's places
// read as the value times 2^-120 (subnormals too); a multiplication by 2^(byte - 7)
// undoes that and applies the vector's scale.  The move: bytes spread to the low
// half of each 16 bits, x; then 16 x + 240 (x & 0x80) has the sign at bit 15 and the
// rest from bit 4 on.  The factors come as kernel parameters, so that they stay
// multiply-adds: those, the byte permutes and the multiplication spread over
// different pipes, whereas the conversion instructions run at a quarter of their
// rate on the units that the softmax's exponentials need.
struct Spread { uint32_t k16, k240; };
__device__ __forceinline__ uint32_t spread_bf16(uint32_t x, uint32_t m, const Spread& k) {
  const uint32_t y = x * k.k16 + (x & 0x00800080u) * k.k240;
  uint32_t o;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(y), "r"(m));
  return o;
}
// Four bytes -> two bf16x2 words in order, times m.
__device__ __forceinline__ uint2 dequant4(uint32_t w, uint32_t m, const Spread& k) {
  return make_uint2(spread_bf16(__byte_perm(w, 0u, 0x4140), m, k),
                    spread_bf16(__byte_perm(w, 0u, 0x4342), m, k));
}
// bf16x2 of 2^(byte - 7) twice (at most 2^127: rest_scale has what is missing);
// NaN for byte 255, 0 where there is no row.
constexpr uint32_t kNoExp = 256u;
__device__ __forceinline__ uint32_t main_scale(uint32_t byte) {
  const uint32_t f = byte == kNoExp ? 0u : byte == 255u ? 0x7FC0u : min(byte + 120u, 254u) << 7;
  return f * 0x10001u;
}
// Scales above 2^7 (values above 448 * 2^7): bf16x2 of 2^(byte - 134).
__device__ __forceinline__ uint32_t rest_scale(uint32_t byte) {
  return ((byte >= 255u || byte <= 134u ? 127u : byte - 7u) << 7) * 0x10001u;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t o;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
  return o;
}

// A transposed pair: bytes (key 0: d 0, d 1; key 1: d 0, d 1) -> words (key 0, key 1)
// of d 0 and of d 1, times m's halves for the two keys.
__device__ __forceinline__ uint2 dequant4_t(uint32_t w, uint32_t m, const Spread& k) {
  return make_uint2(spread_bf16(__byte_perm(w, 0u, 0x4240), m, k),
                    spread_bf16(__byte_perm(w, 0u, 0x4341), m, k));
}

// Writing to and reading from the pages (cache.cu).
constexpr int kCacheMaxTok = 128;    // tokens per CTA at most
struct CacheParams {
  const void* k_in;                  // write: new tokens [B, S, Hkv, d]
  const void* v_in;
  void* k_out;                       // read: rows [B, S, Hkv, d]
  void* v_out;
  void* kp;                          // pools [num_pages, page, Hkv, d]
  void* vp;
  uint8_t* ke;                       // e4m3 pools: exponent bytes [num_pages, page, Hkv]
  uint8_t* ve;
  const int32_t* table;              // [B, max_pages]
  const int32_t* lens;               // [B]
  const uint8_t* tmask;              // write: [B or 1, S], null = all valid
  long long tmask_bs;
  int32_t* lens_out;                 // write: [B], may be null
  uint8_t* valid_out;                // read: [B, S], may be null
  int B, S, Hkv, d;
  int page_shift, num_pages, max_pages;
  bool seen_only;                    // read: only rows that a chunk sees (window, sinks)
  int window, sinks;
};
cudaError_t launch_cache(const CacheParams& p, bool write, bool f32, int cache_dtype,
                         const DevCtl& ctl, cudaStream_t st);

// Attention of a chunk of new tokens over the pages.
struct PagedParams {
  const void* q;                     // [B, Sq, Hq, d]
  const void* k;                     // the chunk's keys and values [B, Sq, Hkv, d]
  const void* v;
  const void* kp;                    // pools and exponents as in CacheParams
  const void* vp;
  const uint8_t* ke;
  const uint8_t* ve;
  const int32_t* table;
  const int32_t* lens;
  const uint8_t* ar;                 // chunk mask rows, segment ids (may be null)
  const int32_t* seg;
  long long mask_bs;
  void* out;
  float* lse;                        // [B, Sq, Hq], may be null
  int B, Sq, Hq, Hkv, d;
  int page_shift, num_pages, max_pages;
  int window, sinks;                 // window 0: none
  int cache_dtype;
  bool f32;                          // q, k, v, out
  float scale;
  bool in_order;                     // bf16 pages [B * max_pages] in order, no table
};

// A sequence's cached length, clamped to what its page-table row can hold.
// `bad` is set when it had to be.
__device__ __forceinline__ int cached_len(const int32_t* lens, int b, int max_pages,
                                          int page_shift, bool& bad) {
  const long long cap = (long long)max_pages << page_shift;
  const int n = lens[b];
  bad = bad || n < 0 || n > cap;
  return (int)min((long long)max(n, 0), cap);
}

// Query i of a chunk stands at position len + i.  Cached keys it sees are
// [0, sink_end) and [lo, len): everything without a window; with one, keys
// less than `window` positions back plus the first `sinks`.
struct CachedRange { int sink_end, lo; };
__device__ __forceinline__ CachedRange cached_range(int len, int i, int window, int sinks) {
  if (window <= 0) return {0, 0};
  const int lo = min(max(len + i - window + 1, 0), len);
  return {min(sinks, lo), lo};
}

// The n low bits set (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n >= 32 ? ~0u : (n <= 0 ? 0u : (1u << n) - 1u);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// Whether the window lets query i see the chunk's key j.
__device__ __forceinline__ bool in_window(int len, int i, int j, int window, int sinks) {
  return window <= 0 || i - j < window || len + j < sinks;
}

// bf16 queries, d = 256, G = Hq / Hkv in {1, 2, 4, 8, 16} on tcgen05
// (paged_tc.cu).  Sequences are scheduled in groups of kPagedTcGroup.
constexpr int kPagedTcGroup = 64;
struct PagedTcParams : PagedParams {
  CUtensorMap map_q, map_o;  // query and output rows
  CUtensorMap map_k, map_v;  // the pools, if use_tma (there is a page)
  int use_tma;
  float* ws;                 // partials [n_clusters * 2][256 rows][256], then (m, l)
  uint16_t* codes;           // chunks over 512 tokens: the CTAs' codes
  int G, g_shift;            // heads per kv head (a power of two), its logarithm
  int tok_per_tile;          // new tokens per 256-row tile
  int n_tiles;               // query tiles per (sequence, kv head)
  int b0, nb;                // this launch's sequences
  int n_clusters;
  int may_cut;               // units may be cut (ws is given)
  int smem_bytes;
  float scale_log2;
  Spread spread;             // {16, 240}
};
bool paged_tc_applies(const PagedParams& p);
size_t paged_tc_workspace_bytes(const PagedParams& p);
cudaError_t launch_paged_tc(const PagedParams& p, float* ws, const DevCtl& ctl, cudaStream_t st);

// At most 8 query rows per kv head: bf16 queries, d = 256, G in {1, 2, 4, 8}
// (paged_decode.cu).
constexpr int kPagedDecodeGroup = 128;
struct PagedDecodeParams : PagedParams {
  CUtensorMap map_k, map_v;  // the pools, boxes of 16 rows
  float* ws;                 // partials [n_ctas * 2][8 rows][256], then (m, l)
  int G, g_shift;
  int b0, nb;                // this launch's sequences
  int n_ctas;
  float scale_log2;
  Spread spread;             // {16, 240}
};
bool paged_decode_applies(const PagedParams& p);
size_t paged_decode_workspace_bytes(const PagedParams& p);
cudaError_t launch_paged_decode(const PagedParams& p, float* ws, const DevCtl& ctl,
                                cudaStream_t st);

cudaError_t launch_paged_simt(const PagedParams& p, const DevCtl& ctl, cudaStream_t st);

}  // namespace piattn
