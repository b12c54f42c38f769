// cache.cu -- the paged key/value cache: appending new tokens (optionally
// quantised to e4m3) and reading sequences back as dense tensors.
//
// Format.  A pool is [pages][page_size][Hkv][d]; sequence b's token at
// position x lives in slot table[b][x / page_size] * page_size + x % page_size.
// An e4m3 pool carries one exponent byte per (slot, head): a vector x is held
// as y = rn_e4m3(x * 2^-e) with e the smallest integer for which amax(|x|) <=
// 448 * 2^e (e >= -126), byte = e + 127.  A power of two costs nothing: e4m3
// keeps its 3 mantissa bits over 2^-6 .. 448 wherever amax falls in (224, 448],
// so every element down to amax * 2^-13 is rounded once, by at most half a
// step (2^-4 of it; 2^-10 of the scale where e4m3 is subnormal, also for larger
// elements if e stops at -126), and undoing the scale is exact in bf16 and fp32, which
// lets the attention kernels rebuild bf16 operands without a second rounding.
// Non-finite input: a NaN makes the whole vector NaN (byte 255, so that no
// reader has to look for NaN bytes); an infinity reads back infinite (448 *
// 2^120 overflows) and flushes the finite rest of its vector, up to 2^110.
// Finite input reads back finite (cap_top()).
//
// Both kernels move each byte once and are bound by HBM (long calls) or by
// launch latency (a token per sequence).  d / 8 lanes own one vector, 8
// elements each (16 bytes of bf16), so a warp access is a contiguous run; the
// amax is one warp reduction (d / 8 lanes of shuffles below d = 256); a thread
// keeps the loads of several vectors of keys and of values in flight.  Measured: 32
// prefixes of 824 tokens to e4m3 in 11.5 us (3.5 TB/s; 20 us with the loads behind
// the slot lookups and the scaling in fp32), four bf16 sequences of up to 16000
// tokens read back in 17.2 us (6.7 TB/s), a token for each of 32 sequences 2.2 us.
#include <algorithm>

#include "launch.h"
#include "paged.cuh"

namespace piattn {

namespace {

constexpr int kCacheThreads = 128;
// Vectors per thread and tensor.  Writing, 32 prefixes of 824 tokens to e4m3 / 8 of
// 611 in bf16: 1 vector 13.8 / 3.1 us, 2 11.5 / 2.8, 3 11.5 / 2.7, 4 11.8 / 2.9, 8 14.6
// / 3.1 (more copies in flight against more CTAs).
constexpr int kWriteRows = 3, kReadRows = 4;

// Eight elements as they lie in memory, and as floats.
struct F8 { float x[8]; };
template <typename T> struct Raw;
template <> struct Raw<float> { uint4 a, b; };
template <> struct Raw<__nv_bfloat16> { uint4 a; };
template <> struct Raw<E4M3> { uint2 a; };

__device__ __forceinline__ void zero(Raw<float>& r) { r.a = r.b = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void zero(Raw<__nv_bfloat16>& r) { r.a = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void zero(Raw<E4M3>& r) { r.a = make_uint2(0u, 0u); }

__device__ __forceinline__ void load(const float* p, Raw<float>& r) {
  r.a = *reinterpret_cast<const uint4*>(p);
  r.b = *reinterpret_cast<const uint4*>(p + 4);
}
__device__ __forceinline__ void load(const __nv_bfloat16* p, Raw<__nv_bfloat16>& r) {
  r.a = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void load(const E4M3* p, Raw<E4M3>& r) {
  r.a = *reinterpret_cast<const uint2*>(p);
}
__device__ __forceinline__ void store(float* p, const Raw<float>& r) {
  *reinterpret_cast<uint4*>(p) = r.a;
  *reinterpret_cast<uint4*>(p + 4) = r.b;
}
__device__ __forceinline__ void store(__nv_bfloat16* p, const Raw<__nv_bfloat16>& r) {
  *reinterpret_cast<uint4*>(p) = r.a;
}
__device__ __forceinline__ F8 floats(const Raw<float>& r) {
  return F8{{__uint_as_float(r.a.x), __uint_as_float(r.a.y), __uint_as_float(r.a.z),
             __uint_as_float(r.a.w), __uint_as_float(r.b.x), __uint_as_float(r.b.y),
             __uint_as_float(r.b.z), __uint_as_float(r.b.w)}};
}
__device__ __forceinline__ F8 floats(const Raw<__nv_bfloat16>& r) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.x[2 * i] = __uint_as_float(w[i] << 16);
    f.x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return f;
}
__device__ __forceinline__ F8 floats(const Raw<E4M3>& r) {
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? r.a.x : r.a.y;
    const float2 v = e4m3x2_to_float2((uint16_t)(w >> (16 * (i & 1))));
    f.x[2 * i] = v.x;
    f.x[2 * i + 1] = v.y;
  }
  return f;
}
__device__ __forceinline__ void store8(float* p, const F8& f) {
  *reinterpret_cast<float4*>(p) = make_float4(f.x[0], f.x[1], f.x[2], f.x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f.x[4], f.x[5], f.x[6], f.x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const F8& f) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(cvt_bf16x2(f.x[0], f.x[1]), cvt_bf16x2(f.x[2], f.x[3]),
                 cvt_bf16x2(f.x[4], f.x[5]), cvt_bf16x2(f.x[6], f.x[7]));
}
__device__ __forceinline__ void store8(E4M3* p, const F8& f) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = (uint32_t)float2_to_e4m3x2(f.x[4 * i], f.x[4 * i + 1]) |
           ((uint32_t)float2_to_e4m3x2(f.x[4 * i + 2], f.x[4 * i + 3]) << 16);
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

template <typename T> constexpr bool kIsE4M3 = false;
template <> constexpr bool kIsE4M3<E4M3> = true;

// The byte of e = 120, the largest that finite input takes (an infinity's too).
constexpr uint32_t kTopByte = 247u;

// The exponent byte of a vector whose largest magnitude has the bits u (above
// infinity's: a NaN): 448 = 1.75 * 2^8, so 1.M * 2^(E - 127) needs e = E - 135, one
// more if 1.M > 1.75.  Zero vectors take scale 1.
__device__ __forceinline__ uint32_t exp_byte(uint32_t u) {
  if (u == 0) return 127u;
  if (u > 0x7F800000u) return 255u;
  const int byte = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(byte, 1);
}

// The largest magnitude of eight elements, as the bits of a float: magnitudes
// compare as integers, and a NaN's is the largest.  bf16: two at a time.
__device__ __forceinline__ uint32_t magnitude(const Raw<float>& r) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ uint32_t magnitude(const Raw<__nv_bfloat16>& r) {
  const uint32_t k = 0x7FFF7FFFu;
  const uint32_t m = __vmaxu2(__vmaxu2(r.a.x & k, r.a.y & k), __vmaxu2(r.a.z & k, r.a.w & k));
  return max(m & 0xFFFF0000u, m << 16);
}
// The elements times 2^(biased - 127), exact (what would fall under the type's
// range is far under e4m3's).
__device__ __forceinline__ F8 scaled(const Raw<float>& r, uint32_t biased) {
  F8 f = floats(r);
  const float s = __uint_as_float(biased << 23);
#pragma unroll
  for (int e = 0; e < 8; ++e) f.x[e] *= s;
  return f;
}
__device__ __forceinline__ F8 scaled(const Raw<__nv_bfloat16>& r, uint32_t biased) {
  const uint32_t s = (biased << 7) * 0x10001u;
  Raw<__nv_bfloat16> x;
  x.a = make_uint4(mul_bf16x2(r.a.x, s), mul_bf16x2(r.a.y, s), mul_bf16x2(r.a.z, s),
                   mul_bf16x2(r.a.w, s));
  return floats(x);
}

// Valid tokens among mask[0 .. n): the thread's share, 16 bytes at a time where
// the row is aligned.
__device__ __forceinline__ int count_valid(const uint8_t* mask, int n) {
  int cnt = 0, t = 0;
  if ((reinterpret_cast<uintptr_t>(mask) & 15u) == 0) {
    t = n & ~15;
    for (int i = threadIdx.x * 16; i < t; i += kCacheThreads * 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(mask + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        cnt += __popc((w[k] | ((w[k] & 0x7F7F7F7Fu) + 0x7F7F7F7Fu)) & 0x80808080u);
    }
  }
  for (t += threadIdx.x; t < n; t += kCacheThreads) cnt += mask[t] != 0 ? 1 : 0;
  return cnt;
}

// Eight elements just stored with exponent byte `byte`.  At the largest scale, 2^120,
// the e4m3 value 256 (0x78; finite elements reach it, from 248 on, and none above)
// would stand for 2^128 and read back infinite: the one below, 240, is within 2^-4
// of them.  Apart from the loop, which such vectors never enter in earnest: in it,
// the test cost a prefix 0.8 us of 11.5.
__device__ __forceinline__ void cap_top(E4M3* p, uint32_t byte) {
  if (byte != kTopByte) return;
  uint2 w = *reinterpret_cast<const uint2*>(p);
  w.x -= __vcmpeq4(w.x & 0x7F7F7F7Fu, 0x78787878u) & 0x01010101u;
  w.y -= __vcmpeq4(w.y & 0x7F7F7F7Fu, 0x78787878u) & 0x01010101u;
  *reinterpret_cast<uint2*>(p) = w;
}

// One CTA takes `tok` consecutive new tokens of one sequence, one pass of its
// threads.  The vectors are loaded first: where they go takes three dependent
// lookups (length and mask, page, slot), which the loads cover.  A token's
// position is the sequence's cached length plus the valid tokens before it: the
// CTA counts the mask bytes before its run, and one ballot per 32 tokens ranks
// its own.
template <typename TIn, typename TC>
__global__ void __launch_bounds__(kCacheThreads)
    cache_write_kernel(const __grid_constant__ CacheParams p, const DevCtl ctl, int tok) {
  __shared__ int s_count[kCacheThreads / 32];
  __shared__ int s_slot[kCacheMaxTok];       // slot of each token, -1: not stored
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, t0 = blockIdx.x * tok;
  const int nt = min(tok, p.S - t0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lpv = p.d >> 3;                  // lanes per vector
  const int n_vec = nt * p.Hkv;              // vectors of each tensor in the run
  const int vpb = kCacheThreads / lpv;       // vectors per row of the pass
  const int vi = threadIdx.x / lpv, e0 = (threadIdx.x % lpv) * 8;
  const long long src0 = ((long long)b * p.S + t0) * p.Hkv;
  const TIn* kin = static_cast<const TIn*>(p.k_in);
  const TIn* vin = static_cast<const TIn*>(p.v_in);
  Raw<TIn> kr[kWriteRows], vr[kWriteRows];
  auto fetch = [&](int v0) {
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
      const int v = v0 + i * vpb + vi;
      if (v < n_vec) {
        load(kin + (src0 + v) * p.d + e0, kr[i]);
        load(vin + (src0 + v) * p.d + e0, vr[i]);
      } else {
        zero(kr[i]);
        zero(vr[i]);
      }
    }
  };
  fetch(0);

  const uint8_t* tm = p.tmask ? p.tmask + (long long)b * p.tmask_bs : nullptr;
  const long long cap = (long long)p.max_pages << p.page_shift;
  bool bad = false;
  const int len = cached_len(p.lens, b, p.max_pages, p.page_shift, bad);
  int before = t0;                           // valid tokens before the run
  if (tm) {
    int cnt = count_valid(tm, t0);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, off);
    if (lane == 0) s_count[warp] = cnt;
    __syncthreads();
    before = 0;
#pragma unroll
    for (int w = 0; w < kCacheThreads / 32; ++w) before += s_count[w];
  }
  if (warp == 0) {
    int n = before;
    for (int base = 0; base < nt; base += 32) {
      const int t = base + lane;
      const bool on = t < nt && (!tm || tm[t0 + t] != 0);
      const uint32_t bits = __ballot_sync(0xffffffffu, on);
      if (t < nt) {
        int slot = -1;
        const long long x = (long long)len + n + __popc(bits & ((1u << lane) - 1u));
        if (on) {
          if (x < cap) {
            const int page = p.table[(long long)b * p.max_pages + (x >> p.page_shift)];
            if (page >= 0 && page < p.num_pages)
              slot = (page << p.page_shift) + (int)(x & ((1 << p.page_shift) - 1));
            else
              bad = true;
          } else {
            bad = true;
          }
        }
        s_slot[t] = slot;
      }
      n += __popc(bits);
    }
    if (p.lens_out && t0 + nt == p.S && lane == 0)
      p.lens_out[b] = (int)min((long long)len + n, cap);
    if (bad) record_status(ctl, kStatusArg);
  }
  __syncthreads();

  TC* kp = static_cast<TC*>(p.kp);
  TC* vp = static_cast<TC*>(p.vp);
  bool top = false;                          // (e4m3) some vector has the largest scale
  for (int v0 = 0; v0 < n_vec; v0 += vpb * kWriteRows) {
    if (v0 > 0) fetch(v0);
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
      const int v = v0 + i * vpb + vi;
      const int t = p.Hkv == 1 ? v : v / p.Hkv;
      const int slot = v < n_vec ? s_slot[t] : -1;
      const long long dst = (long long)(slot - t) * p.Hkv + v;   // slot * Hkv + v % Hkv
      if constexpr (kIsE4M3<TC>) {
        uint32_t ka = magnitude(kr[i]), va = magnitude(vr[i]);
        if (lpv == 32) {
          ka = __reduce_max_sync(0xffffffffu, ka);
          va = __reduce_max_sync(0xffffffffu, va);
        } else {
          for (int off = lpv >> 1; off > 0; off >>= 1) {
            ka = max(ka, __shfl_xor_sync(0xffffffffu, ka, off));
            va = max(va, __shfl_xor_sync(0xffffffffu, va, off));
          }
        }
        const uint32_t kb = exp_byte(ka), vb = exp_byte(va);
        // 2^-e = 2^(127 - byte): biased exponent 254 - byte, in [7, 253] (a NaN
        // vector: 0, what it holds does not matter)
        const F8 kx = scaled(kr[i], 254u - min(kb, 254u)), vx = scaled(vr[i], 254u - min(vb, 254u));
        top = top || kb == kTopByte || vb == kTopByte;
        if (slot >= 0) {
          store8(kp + dst * p.d + e0, kx);
          store8(vp + dst * p.d + e0, vx);
          if (e0 == 0) {
            p.ke[dst] = (uint8_t)kb;
            p.ve[dst] = (uint8_t)vb;
          }
        }
      } else if (slot >= 0) {
        store(kp + dst * p.d + e0, kr[i]);
        store(vp + dst * p.d + e0, vr[i]);
      }
    }
  }
  if constexpr (kIsE4M3<TC>) {
    if (__any_sync(0xffffffffu, top)) {
      __syncwarp();                          // the exponents that this warp's lanes wrote
#pragma unroll 1
      for (int v = vi; v < n_vec; v += vpb) {
        const int t = v / p.Hkv;
        if (s_slot[t] < 0) continue;
        const long long dst = (long long)(s_slot[t] - t) * p.Hkv + v;
        cap_top(kp + dst * p.d + e0, p.ke[dst]);
        cap_top(vp + dst * p.d + e0, p.ve[dst]);
      }
    }
  }
}

// One CTA brings `tok` consecutive rows of one sequence; rows past its length
// are written as zeros (a dense pass over the result multiplies them by 0).  With
// seen_only, rows that the chunk's first query does not see (no later one sees
// more of the cache) are neither read nor written.
template <typename TOut, typename TC>
__global__ void __launch_bounds__(kCacheThreads)
    cache_read_kernel(const __grid_constant__ CacheParams p, const DevCtl ctl, int tok) {
  __shared__ int s_slot[kCacheMaxTok];
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y, t0 = blockIdx.x * tok;
  const int nt = min(tok, p.S - t0);
  bool bad = false;
  const int len = cached_len(p.lens, b, p.max_pages, p.page_shift, bad);
  const int lo = p.window > 0 ? min(max(len - p.window + 1, 0), len) : 0;
  for (int t = threadIdx.x; t < nt; t += kCacheThreads) {
    const int x = t0 + t;
    int slot = -1;                           // -1: zeros, -2: left alone
    if (p.seen_only && (x >= len || (x < lo && x >= p.sinks))) {
      slot = -2;
    } else if (x < len) {
      const int page = p.table[(long long)b * p.max_pages + (x >> p.page_shift)];
      if (page >= 0 && page < p.num_pages)
        slot = (page << p.page_shift) + (x & ((1 << p.page_shift) - 1));
      else
        bad = true;
    }
    s_slot[t] = slot;
    if (p.valid_out) p.valid_out[(long long)b * p.S + x] = x < len ? 1 : 0;
  }
  if (bad) record_status(ctl, kStatusArg);
  __syncthreads();

  const int lpv = p.d >> 3;
  const int n_vec = nt * p.Hkv;
  const int vpb = kCacheThreads / lpv;
  const int vi = threadIdx.x / lpv, e0 = (threadIdx.x % lpv) * 8;
  const long long dst0 = ((long long)b * p.S + t0) * p.Hkv;
  const TC* kp = static_cast<const TC*>(p.kp);
  const TC* vp = static_cast<const TC*>(p.vp);
  TOut* ko = static_cast<TOut*>(p.k_out);
  TOut* vo = static_cast<TOut*>(p.v_out);
  for (int v0 = 0; v0 < n_vec; v0 += vpb * kReadRows) {
    Raw<TC> kr[kReadRows], vr[kReadRows];
    uint8_t kb[kReadRows], vb[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      const int v = v0 + i * vpb + vi;
      const int t = p.Hkv == 1 ? v : v / p.Hkv;
      const int slot = v < n_vec ? s_slot[t] : -1;
      kb[i] = vb[i] = 127;
      zero(kr[i]);
      zero(vr[i]);
      if (slot >= 0) {
        const long long src = (long long)(slot - t) * p.Hkv + v;   // slot * Hkv + v % Hkv
        load(kp + src * p.d + e0, kr[i]);
        load(vp + src * p.d + e0, vr[i]);
        if constexpr (kIsE4M3<TC>) {
          kb[i] = p.ke[src];
          vb[i] = p.ve[src];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      const int v = v0 + i * vpb + vi;
      if (v >= n_vec || s_slot[p.Hkv == 1 ? v : v / p.Hkv] == -2) continue;
      const long long at = (dst0 + v) * p.d + e0;
      if constexpr (kIsE4M3<TC>) {
        F8 kx = floats(kr[i]), vx = floats(vr[i]);
        const float ks = exp_scale(kb[i]), vs = exp_scale(vb[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          kx.x[e] *= ks;
          vx.x[e] *= vs;
        }
        store8(ko + at, kx);
        store8(vo + at, vx);
      } else {
        store(ko + at, kr[i]);
        store(vo + at, vr[i]);
      }
    }
  }
}

// Tokens per CTA: enough vectors that every thread has `rows` of each tensor,
// fewer when the grid would leave SMs idle.
int tokens_per_cta(const CacheParams& p, int rows) {
  const int vpb = kCacheThreads / (p.d >> 3);
  int tok = (vpb * rows + p.Hkv - 1) / p.Hkv;
  tok = std::min(std::max(tok, 1), kCacheMaxTok);
  while (tok > 1 && (long long)p.B * ((p.S + tok - 1) / tok) < 2 * sm_count()) tok = (tok + 1) / 2;
  return tok;
}

// (Pools and dense tensors share a type unless the pool is e4m3.)
template <typename T, typename TC>
cudaError_t launch(const CacheParams& p, bool write, const DevCtl& ctl, cudaStream_t st) {
  const int tok = tokens_per_cta(p, write ? kWriteRows : kReadRows);
  // (Without tokens one CTA a sequence still writes its length.)
  dim3 grid((unsigned)std::max((p.S + tok - 1) / tok, 1), (unsigned)p.B);
  return write ? launch_pdl(cache_write_kernel<T, TC>, grid, dim3(kCacheThreads), 0, st, p, ctl, tok)
               : launch_pdl(cache_read_kernel<T, TC>, grid, dim3(kCacheThreads), 0, st, p, ctl, tok);
}

}  // namespace

cudaError_t launch_cache(const CacheParams& p, bool write, bool f32, int cache_dtype,
                         const DevCtl& ctl, cudaStream_t st) {
  if (cache_dtype == kCacheE4M3)
    return f32 ? launch<float, E4M3>(p, write, ctl, st)
               : launch<__nv_bfloat16, E4M3>(p, write, ctl, st);
  return f32 ? launch<float, float>(p, write, ctl, st)
             : launch<__nv_bfloat16, __nv_bfloat16>(p, write, ctl, st);
}

}  // namespace piattn
