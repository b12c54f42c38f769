// cache.cu -- the paged key/value cache: appending new tokens (optionally
// quantised to e4m3) and reading sequences back as dense tensors.
//
// Format.  A pool is [pages][page_size][Hkv][d]; sequence b's token at
// position x lives in slot table[b][x / page_size] * page_size + x % page_size.
// An e4m3 pool carries one exponent byte per (slot, head): a vector x is held
// as y = rn_e4m3(x * 2^-e) with e the smallest integer for which amax(|x|) <=
// 448 * 2^e (e >= -126), byte = e + 127.  A power of two costs nothing: e4m3
// keeps its 3 mantissa bits over 2^-6 .. 448 wherever amax falls in (224, 448],
// so every element down to amax * 2^-14 is rounded once, by at most half a
// step (2^-4 of it), and undoing the scale is exact in bf16 and fp32, which
// lets the attention kernels rebuild bf16 operands without a second rounding.
// Non-finite input: a NaN makes the whole vector NaN (byte 255, so that no
// reader has to look for NaN bytes); an infinity reads back infinite (448 *
// 2^120 overflows) and flushes the finite rest of its vector.
//
// Both kernels move each byte once and are bound by HBM (long calls) or by
// launch latency (a token per sequence).  d / 8 lanes own one vector, 8
// elements each (16 bytes of bf16), so a warp access is a contiguous run; the
// amax is d / 8 lanes of shuffles; a thread keeps the loads of kRows tokens'
// keys and values in flight.
#include <algorithm>

#include "launch.h"
#include "paged.cuh"

namespace piattn {

namespace {

constexpr int kCacheThreads = 128;
constexpr int kRows = 4;                    // vectors per thread and tensor

struct F8 { float x[8]; };

__device__ __forceinline__ F8 load8(const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ F8 load8(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.x[2 * i] = __uint_as_float(w[i] << 16);
    f.x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return f;
}
__device__ __forceinline__ F8 load8(const E4M3* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  F8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? u.x : u.y;
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

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The exponent byte of a vector with largest magnitude amax (NaN if it holds
// one): 448 = 1.75 * 2^8, so amax = 1.M * 2^(E - 127) needs e = E - 135, one more
// if 1.M > 1.75.  Zero vectors take scale 1.
__device__ __forceinline__ uint32_t exp_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return 127u;
  if (u > 0x7F800000u) return 255u;
  const int byte = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(byte, 1);
}

// One CTA takes `tok` consecutive new tokens of one sequence.  A token's
// position is the sequence's cached length plus the valid tokens before it:
// the CTA counts the mask bytes before its run, and one ballot per 32 tokens
// ranks its own.
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
  const uint8_t* tm = p.tmask ? p.tmask + (long long)b * p.tmask_bs : nullptr;
  const long long cap = (long long)p.max_pages << p.page_shift;
  bool bad = false;
  const int len = cached_len(p.lens, b, p.max_pages, p.page_shift, bad);

  int before = t0;                           // valid tokens before the run
  if (tm) {
    int cnt = 0;
    for (int t = threadIdx.x; t < t0; t += kCacheThreads) cnt += tm[t] != 0 ? 1 : 0;
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

  const int lpv = p.d >> 3;                  // lanes per vector
  const int n_vec = nt * p.Hkv;              // vectors of each tensor in the run
  const int vpb = kCacheThreads / lpv;       // vectors per pass of the CTA
  const int vi = threadIdx.x / lpv, e0 = (threadIdx.x % lpv) * 8;
  const long long src0 = ((long long)b * p.S + t0) * p.Hkv;
  const TIn* kin = static_cast<const TIn*>(p.k_in);
  const TIn* vin = static_cast<const TIn*>(p.v_in);
  TC* kp = static_cast<TC*>(p.kp);
  TC* vp = static_cast<TC*>(p.vp);
  for (int v0 = 0; v0 < n_vec; v0 += vpb * kRows) {
    F8 kx[kRows], vx[kRows];
    long long dst[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int v = v0 + i * vpb + vi;
      dst[i] = -1;
      if (v < n_vec) {
        const int slot = s_slot[v / p.Hkv];
        if (slot >= 0) {
          dst[i] = (long long)slot * p.Hkv + v % p.Hkv;
          kx[i] = load8(kin + (src0 + v) * p.d + e0);
          vx[i] = load8(vin + (src0 + v) * p.d + e0);
        }
      }
      if (dst[i] < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) kx[i].x[e] = vx[i].x[e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if constexpr (kIsE4M3<TC>) {
        float ka = 0.f, va = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ka = max_nan(ka, fabsf(kx[i].x[e]));
          va = max_nan(va, fabsf(vx[i].x[e]));
        }
        for (int off = lpv >> 1; off > 0; off >>= 1) {
          ka = max_nan(ka, __shfl_xor_sync(0xffffffffu, ka, off));
          va = max_nan(va, __shfl_xor_sync(0xffffffffu, va, off));
        }
        const uint32_t kb = exp_byte(ka), vb = exp_byte(va);
        // 2^-e = 2^(127 - byte): biased exponent 254 - byte, in [7, 253] (a NaN
        // vector: 0, what it holds does not matter)
        const float ks = __uint_as_float((254u - min(kb, 254u)) << 23);
        const float vs = __uint_as_float((254u - min(vb, 254u)) << 23);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          kx[i].x[e] *= ks;
          vx[i].x[e] *= vs;
        }
        if (dst[i] >= 0 && e0 == 0) {
          p.ke[dst[i]] = (uint8_t)kb;
          p.ve[dst[i]] = (uint8_t)vb;
        }
      }
      if (dst[i] >= 0) {
        store8(kp + dst[i] * p.d + e0, kx[i]);
        store8(vp + dst[i] * p.d + e0, vx[i]);
      }
    }
  }
}

// One CTA brings `tok` consecutive rows of one sequence; rows past its length
// are written as zeros (a dense pass over the result multiplies them by 0).
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
  for (int t = threadIdx.x; t < nt; t += kCacheThreads) {
    const int x = t0 + t;
    int slot = -1;
    if (x < len) {
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
  for (int v0 = 0; v0 < n_vec; v0 += vpb * kRows) {
    F8 kx[kRows], vx[kRows];
    float ks[kRows], vs[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int v = v0 + i * vpb + vi;
      const int slot = v < n_vec ? s_slot[v / p.Hkv] : -1;
      ks[i] = vs[i] = 1.f;
      if (slot >= 0) {
        const long long src = (long long)slot * p.Hkv + v % p.Hkv;
        kx[i] = load8(kp + src * p.d + e0);
        vx[i] = load8(vp + src * p.d + e0);
        if constexpr (kIsE4M3<TC>) {
          ks[i] = exp_scale(p.ke[src]);
          vs[i] = exp_scale(p.ve[src]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) kx[i].x[e] = vx[i].x[e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int v = v0 + i * vpb + vi;
      if (v >= n_vec) continue;
      if constexpr (kIsE4M3<TC>) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          kx[i].x[e] *= ks[i];
          vx[i].x[e] *= vs[i];
        }
      }
      store8(ko + (dst0 + v) * p.d + e0, kx[i]);
      store8(vo + (dst0 + v) * p.d + e0, vx[i]);
    }
  }
}

// Tokens per CTA: enough vectors that every thread has kRows of each tensor,
// fewer when the grid would leave SMs idle.
int tokens_per_cta(const CacheParams& p) {
  const int vpb = kCacheThreads / (p.d >> 3);
  int tok = (vpb * kRows + p.Hkv - 1) / p.Hkv;
  tok = std::min(std::max(tok, 1), kCacheMaxTok);
  while (tok > 1 && (long long)p.B * ((p.S + tok - 1) / tok) < 2 * sm_count()) tok = (tok + 1) / 2;
  return tok;
}

template <typename T, typename TC>
cudaError_t launch(const CacheParams& p, bool write, const DevCtl& ctl, cudaStream_t st) {
  const int tok = tokens_per_cta(p);
  dim3 grid((unsigned)((p.S + tok - 1) / tok), (unsigned)p.B);
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
