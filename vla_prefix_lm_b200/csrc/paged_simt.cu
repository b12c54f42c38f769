// paged_simt.cu -- attention of a chunk over the paged cache on CUDA cores:
// the fp32 form (1e-4 tolerances rule out reduced-precision tensor cores) and
// every bf16 head geometry that the tensor-core kernels leave out.
//
// One warp per (batch, new token, query head) row, q and the running output
// in registers (d / 32 consecutive elements per lane).  Keys are visited four
// at a time: four dot products reduce through interleaved shuffles and share
// one running-maximum update, so the chain of dependent shuffles is paid once
// per four keys; four consecutive cached positions never cross a page.
// Masked keys are never loaded, so nothing they hold (NaN in a stale slot)
// reaches the result.
//
// Bound by that chain of dependent steps.  So the eight warps of a CTA share one row,
// every eighth group of four keys each, and merge their states through shared
// memory; only many rows of few keys are left whole to a warp each, which saves that
// merge (split_rows).
#include <cfloat>

#include "launch.h"
#include "paged.cuh"

namespace piattn {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 4;                   // new tokens per CTA (whole rows per warp)

template <int C>
__device__ __forceinline__ void load_row(const float* p, float (&x)[C]) {
  if constexpr (C % 4 == 0) {
#pragma unroll
    for (int c = 0; c < C; c += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + c);
      x[c] = v.x; x[c + 1] = v.y; x[c + 2] = v.z; x[c + 3] = v.w;
    }
  } else if constexpr (C == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x; x[1] = v.y;
  } else {
    x[0] = *p;
  }
}
template <int C>
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, float (&x)[C]) {
  if constexpr (C == 1) {
    x[0] = __bfloat162float(*p);
  } else {
#pragma unroll
    for (int c = 0; c < C; c += 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p + c);
      x[c] = __uint_as_float(w << 16);
      x[c + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
  }
}
template <int C>
__device__ __forceinline__ void load_row(const E4M3* p, float (&x)[C]) {
  if constexpr (C == 1) {
    x[0] = e4m3x2_to_float2((uint16_t)p->bits).x;
  } else {
#pragma unroll
    for (int c = 0; c < C; c += 2) {
      const float2 v = e4m3x2_to_float2(*reinterpret_cast<const uint16_t*>(p + c));
      x[c] = v.x;
      x[c + 1] = v.y;
    }
  }
}
template <int C>
__device__ __forceinline__ void store_row(float* p, const float (&x)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) p[c] = x[c];
}
template <int C>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&x)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) p[c] = __float2bfloat16_rn(x[c]);
}

// The state of one row's online softmax over groups of four keys.
template <int C>
struct Row {
  float q[C], acc[C];
  float m = -FLT_MAX, l = 0.f;

  // s[u]: this lane's part of key u's score; on[u]: key u is visible (its
  // value row is in v[u], else zeros).
  __device__ __forceinline__ void add4(float (&s)[4], const bool (&on)[4], const float (&v)[4][C]) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], off);
    }
    float mx = m;
#pragma unroll
    for (int u = 0; u < 4; ++u) mx = on[u] ? fmaxf(mx, s[u]) : mx;
    const float corr = expf(m - mx);
    m = mx;
    float e[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) e[u] = on[u] ? expf(s[u] - mx) : 0.f;
    l = l * corr + ((e[0] + e[1]) + (e[2] + e[3]));
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float a = acc[c] * corr;
#pragma unroll
      for (int u = 0; u < 4; ++u) a = fmaf(e[u], v[u][c], a);
      acc[c] = a;
    }
  }
};

// kSplit: a CTA's warps share one row (blockIdx.x), else each takes rows of its own
// among the CTA's kTokens tokens.
template <int D, typename T, typename TC, bool kSplit>
__global__ void __launch_bounds__(kThreads)
    paged_simt_kernel(const __grid_constant__ PagedParams p, const DevCtl ctl) {
  extern __shared__ uint32_t s_codes[];      // [Sq] codes of the new tokens
  __shared__ int s_scan[33];
  __shared__ float s_acc[kSplit ? kWarps : 1][kSplit ? D : 1];
  __shared__ float2 s_ml[kWarps];
  constexpr int C = D / 32;
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  build_codes<uint32_t>(p.ar + (long long)b * p.mask_bs,
                        p.seg ? p.seg + (long long)b * p.mask_bs : nullptr, p.Sq, s_codes, s_scan);
  bool bad = false;
  const int len = cached_len(p.lens, b, p.max_pages, p.page_shift, bad);
  const int32_t* table = p.table + (long long)b * p.max_pages;
  const int group = p.Hq / p.Hkv;
  const int e0 = lane * C;
  const T* kn = static_cast<const T*>(p.k);
  const T* vn = static_cast<const T*>(p.v);
  const TC* kp = static_cast<const TC*>(p.kp);
  const TC* vp = static_cast<const TC*>(p.vp);

  const int r_first = kSplit ? blockIdx.x : blockIdx.x * kTokens * p.Hq + warp;
  const int r_end = kSplit ? blockIdx.x + 1 : min((int)(blockIdx.x + 1) * kTokens, p.Sq) * p.Hq;
  const int part = kSplit ? warp : 0, parts = kSplit ? kWarps : 1;
  for (int r = r_first; r < r_end; r += kWarps) {
    const int i = r / p.Hq, h = r % p.Hq, g = h / group;
    const long long row = (long long)b * p.Sq * p.Hq + r;
    Row<C> x;
    load_row<C>(static_cast<const T*>(p.q) + row * D + e0, x.q);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      x.q[c] *= p.scale;
      x.acc[c] = 0.f;
    }
    const uint32_t cq = s_codes[i];
    if (!is_pad(cq)) {
      // Groups of four cached positions: those with sinks, then from the window on.
      const CachedRange cr = cached_range(len, i, p.window, p.sinks);
      const int n_sink = (cr.sink_end + 3) >> 2, from = max(cr.lo >> 2, n_sink);
      const int n_groups = n_sink + max(((len + 3) >> 2) - from, 0);
      for (int gi = part; gi < n_groups; gi += parts) {
        const int j0 = (gi < n_sink ? gi : from + gi - n_sink) * 4;
        const int page = table[j0 >> p.page_shift];
        const bool ok = page >= 0 && page < p.num_pages;
        float s[4], v[4][C];
        bool on[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j = j0 + u;
          s[u] = 0.f;
#pragma unroll
          for (int c = 0; c < C; ++c) v[u][c] = 0.f;
          on[u] = j < len && (j < cr.sink_end || j >= cr.lo);
          bad = bad || (on[u] && !ok);
          if (on[u] && ok) {
            const long long slot = ((long long)page << p.page_shift) + (j & ((1 << p.page_shift) - 1));
            const long long at = slot * p.Hkv + g;
            float k[C];
            load_row<C>(kp + at * D + e0, k);
            load_row<C>(vp + at * D + e0, v[u]);
#pragma unroll
            for (int c = 0; c < C; ++c) s[u] = fmaf(x.q[c], k[c], s[u]);
            if constexpr (sizeof(TC) == 1) {
              s[u] *= exp_scale(p.ke[at]);
              const float vs = exp_scale(p.ve[at]);
#pragma unroll
              for (int c = 0; c < C; ++c) v[u][c] *= vs;
            }
          }
        }
        x.add4(s, on, v);
      }
      for (int j0 = 4 * part; j0 < p.Sq; j0 += 4 * parts) {
        float s[4], v[4][C];
        bool on[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int j = j0 + u;
          on[u] = j < p.Sq && visible(cq, s_codes[j]) && in_window(len, i, j, p.window, p.sinks);
        }
        if (!(on[0] || on[1] || on[2] || on[3])) continue;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          s[u] = 0.f;
#pragma unroll
          for (int c = 0; c < C; ++c) v[u][c] = 0.f;
          if (on[u]) {
            const long long at = ((long long)b * p.Sq + j0 + u) * p.Hkv + g;
            float k[C];
            load_row<C>(kn + at * D + e0, k);
            load_row<C>(vn + at * D + e0, v[u]);
#pragma unroll
            for (int c = 0; c < C; ++c) s[u] = fmaf(x.q[c], k[c], s[u]);
          }
        }
        x.add4(s, on, v);
      }
    }
    if constexpr (kSplit) {
#pragma unroll
      for (int c = 0; c < C; ++c) s_acc[warp][e0 + c] = x.acc[c];
      if (lane == 0) s_ml[warp] = make_float2(x.m, x.l);
      __syncthreads();
      if (warp > 0) break;
      float m = -FLT_MAX;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_ml[w].x);   // (-FLT_MAX: saw no key)
      x.l = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) x.acc[c] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = expf(s_ml[w].x - m);
        x.l += f * s_ml[w].y;
#pragma unroll
        for (int c = 0; c < C; ++c) x.acc[c] = fmaf(f, s_acc[w][e0 + c], x.acc[c]);
      }
      x.m = m;
    }
    const float inv = x.l > 0.f ? 1.f / x.l : 0.f;   // no visible key (padding): 0
#pragma unroll
    for (int c = 0; c < C; ++c) x.acc[c] *= inv;
    store_row<C>(static_cast<T*>(p.out) + row * D + e0, x.acc);
    if (p.lse && lane == 0)
      p.lse[row] = x.l > 0.f ? x.m + logf(x.l) : (x.l == x.l ? -INFINITY : x.l);
  }
  if (bad) record_status(ctl, kStatusArg);
}

template <int D, typename T, typename TC, bool kSplit>
cudaError_t launch_as(const PagedParams& p, const DevCtl& ctl, cudaStream_t st) {
  const size_t smem = sizeof(uint32_t) * (size_t)p.Sq;
  if (smem > 32 * 1024) {                    // (what else the kernel has is under 16 KB)
    // The bound of every call, not this one's size: another thread's shorter chunk
    // would lower it before this launch.
    const cudaError_t e = cudaFuncSetAttribute(paged_simt_kernel<D, T, TC, kSplit>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(uint32_t) * kMaxTokens);
    if (e != cudaSuccess) return e;
  }
  const int n = kSplit ? p.Sq * p.Hq : (p.Sq + kTokens - 1) / kTokens;
  return launch_pdl(paged_simt_kernel<D, T, TC, kSplit>, dim3((unsigned)n, (unsigned)p.B),
                    dim3(kThreads), smem, st, p, ctl);
}
// Measured (fp32, d = 64, 4 heads), rows whole / split: 36 rows of 49 keys 27 / 5.6 us,
// of 809 keys 495 / 33; 4096 rows of 816 keys 618 / 358; 32768 rows of 864 keys 3011
// / 2462; 4096 rows of 56 keys 36 / 42; 32768 of 56 keys 181 / 343; 8192 of 104 keys 97
// / 103, 32768 of 612 keys 1831 / 1746.
bool split_rows(const PagedParams& p) {
  return (long long)p.B * p.Sq * p.Hq < 4000 ||
         ((long long)p.max_pages << p.page_shift) + p.Sq >= 128;
}
template <int D, typename T, typename TC>
cudaError_t launch(const PagedParams& p, const DevCtl& ctl, cudaStream_t st) {
  return split_rows(p) ? launch_as<D, T, TC, true>(p, ctl, st)
                       : launch_as<D, T, TC, false>(p, ctl, st);
}

template <int D>
cudaError_t launch_d(const PagedParams& p, const DevCtl& ctl, cudaStream_t st) {
  if (p.f32)
    return p.cache_dtype == kCacheE4M3 ? launch<D, float, E4M3>(p, ctl, st)
                                       : launch<D, float, float>(p, ctl, st);
  return p.cache_dtype == kCacheE4M3 ? launch<D, __nv_bfloat16, E4M3>(p, ctl, st)
                                     : launch<D, __nv_bfloat16, __nv_bfloat16>(p, ctl, st);
}

}  // namespace

cudaError_t launch_paged_simt(const PagedParams& p, const DevCtl& ctl, cudaStream_t st) {
  switch (p.d) {
    case 32: return launch_d<32>(p, ctl, st);
    case 64: return launch_d<64>(p, ctl, st);
    case 128: return launch_d<128>(p, ctl, st);
    case 256: return launch_d<256>(p, ctl, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace piattn
