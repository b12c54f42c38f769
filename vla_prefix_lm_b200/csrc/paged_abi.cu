// paged_abi.cu -- the extern "C" entry points of the paged cache (declared in
// include/pi_attn.h): argument validation on the host, before anything is
// enqueued, and dispatch to the kernels.
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <cstring>

#include "../../include/pi_attn.h"
#include "launch.h"
#include "paged.cuh"

namespace {

using namespace piattn;

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int launched(cudaError_t e) { return e == cudaSuccess ? PI_OK : PI_ERR_CUDA; }

int page_shift(const pi_paged_desc* d) {
  int s = 4;
  while ((1 << s) < d->page_size) ++s;
  return s;
}

// What the three calls have in common.
int check_desc(const pi_paged_desc* d) {
  if (!d) return PI_ERR_ARG;
  if (d->B < 0 || d->Sq < 0 || d->Hkv <= 0 || d->d <= 0 || d->num_pages < 0 || d->max_pages < 0 ||
      d->reserved != 0)
    return PI_ERR_ARG;
  if (d->page_size <= 0) return PI_ERR_ARG;
  if (d->dtype != PI_BF16 && d->dtype != PI_F32) return PI_ERR_UNSUPPORTED;
  if (d->cache_dtype != d->dtype && d->cache_dtype != PI_E4M3) return PI_ERR_UNSUPPORTED;
  if (!(d->d == 32 || d->d == 64 || d->d == 128 || d->d == 256)) return PI_ERR_UNSUPPORTED;
  if (!(d->page_size == 16 || d->page_size == 32 || d->page_size == 64 || d->page_size == 128 ||
        d->page_size == 256))
    return PI_ERR_UNSUPPORTED;
  constexpr long long kMaxSlots = (1ll << 31) - (1ll << 15);
  if ((long long)d->num_pages * d->page_size >= kMaxSlots ||
      (long long)d->max_pages * d->page_size >= kMaxSlots || d->Sq >= kMaxSlots)
    return PI_ERR_UNSUPPORTED;
  if (d->B > 65535 || d->Hkv > 65535) return PI_ERR_UNSUPPORTED;
  return PI_OK;
}

int check_mask_stride(const pi_paged_desc* d) {
  if (d->mask_batch_stride < 0 || (d->mask_batch_stride != 0 && d->mask_batch_stride < d->Sq))
    return PI_ERR_ARG;
  if (d->Sq > kMaxTokens) return PI_ERR_UNSUPPORTED;
  return PI_OK;
}

// The pools, exponents, table and lengths.
int check_cache(const pi_paged_desc* d, const void* kp, const void* vp, const uint8_t* ke,
                const uint8_t* ve, const int32_t* table, const int32_t* lens) {
  if (!lens) return PI_ERR_ARG;
  if (d->max_pages > 0 && !table) return PI_ERR_ARG;
  const bool pool = d->num_pages > 0;
  if (pool && (!kp || !vp)) return PI_ERR_ARG;
  if (pool && d->cache_dtype == PI_E4M3 && (!ke || !ve)) return PI_ERR_ARG;
  if (d->cache_dtype != PI_E4M3 && (ke || ve)) return PI_ERR_ARG;
  if (!aligned(kp, 16) || !aligned(vp, 16) || !aligned(table, 4) || !aligned(lens, 4))
    return PI_ERR_ALIGN;
  return PI_OK;
}

int check_attn(const pi_paged_desc* d) {
  const int rc = check_desc(d);
  if (rc != PI_OK) return rc;
  if (d->Hq <= 0 || d->Hq % d->Hkv != 0 || d->window < 0 || d->sinks < 0) return PI_ERR_ARG;
  if (!std::isfinite(d->softmax_scale) || !(d->softmax_scale > 0.f)) return PI_ERR_ARG;
  // (Kernels step a 32-bit row index past a sequence's last row.)
  if ((long long)d->Sq * d->Hq >= (1ll << 31) - (1ll << 15)) return PI_ERR_UNSUPPORTED;
  return check_mask_stride(d);
}

CacheParams cache_params(const pi_paged_desc* d) {
  CacheParams p;
  std::memset(&p, 0, sizeof(p));
  p.B = d->B; p.S = d->Sq; p.Hkv = d->Hkv; p.d = d->d;
  p.page_shift = page_shift(d);
  p.num_pages = d->num_pages;
  p.max_pages = d->max_pages;
  return p;
}

PagedParams paged_params(const pi_paged_desc* d) {
  PagedParams p;
  std::memset(&p, 0, sizeof(p));
  p.mask_bs = d->mask_batch_stride;
  p.B = d->B; p.Sq = d->Sq; p.Hq = d->Hq; p.Hkv = d->Hkv; p.d = d->d;
  p.page_shift = page_shift(d);
  p.num_pages = d->num_pages;
  p.max_pages = d->max_pages;
  // A window that reaches back over any sequence hides nothing.  (What is
  // left keeps every position difference inside 32 bits.)
  p.window = (long long)d->window >= (long long)d->max_pages * d->page_size + d->Sq ? 0 : d->window;
  p.sinks = p.window > 0 ? d->sinks : 0;
  p.cache_dtype = d->cache_dtype;
  p.f32 = d->dtype == PI_F32;
  p.scale = d->softmax_scale;
  return p;
}

}  // namespace

extern "C" {

int pi_attn_cache_write(const pi_paged_desc* d, const void* k_new, const void* v_new,
                        const uint8_t* token_mask, const int32_t* page_table,
                        const int32_t* cache_lens, void* k_pages, void* v_pages, uint8_t* k_exp,
                        uint8_t* v_exp, int32_t* lens_out, pi_stream_t stream) {
  NvtxRange range("pi_attn_cache_write");
  int rc = check_desc(d);
  if (rc == PI_OK) rc = check_mask_stride(d);
  if (rc != PI_OK) return rc;
  if (d->B == 0) return PI_OK;
  if (d->Sq > 0 && (!k_new || !v_new)) return PI_ERR_ARG;
  if (lens_out && cache_lens) {              // every CTA reads its sequence's length
    const uintptr_t x = reinterpret_cast<uintptr_t>(lens_out), n = sizeof(int32_t) * (size_t)d->B;
    const uintptr_t y = reinterpret_cast<uintptr_t>(cache_lens);
    if (x < y + n && y < x + n) return PI_ERR_ARG;
  }
  rc = check_cache(d, k_pages, v_pages, k_exp, v_exp, page_table, cache_lens);
  if (rc != PI_OK) return rc;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(lens_out, 4)) return PI_ERR_ALIGN;
  if (d->Sq == 0 && !lens_out) return PI_OK;
  DevCtl ctl;
  if (!make_ctl(&ctl)) return PI_ERR_CUDA;
  CacheParams p = cache_params(d);
  p.k_in = k_new; p.v_in = v_new;
  p.kp = k_pages; p.vp = v_pages; p.ke = k_exp; p.ve = v_exp;
  p.table = page_table; p.lens = cache_lens;
  p.tmask = token_mask; p.tmask_bs = d->mask_batch_stride;
  p.lens_out = lens_out;
  return launched(launch_cache(p, true, d->dtype == PI_F32, d->cache_dtype, ctl,
                               static_cast<cudaStream_t>(stream)));
}

int pi_attn_cache_read(const pi_paged_desc* d, const void* k_pages, const void* v_pages,
                       const uint8_t* k_exp, const uint8_t* v_exp, const int32_t* page_table,
                       const int32_t* cache_lens, void* k_out, void* v_out, uint8_t* valid_out,
                       pi_stream_t stream) {
  NvtxRange range("pi_attn_cache_read");
  int rc = check_desc(d);
  if (rc != PI_OK) return rc;
  if (d->B == 0 || d->Sq == 0) return PI_OK;
  if (!k_out || !v_out) return PI_ERR_ARG;
  rc = check_cache(d, k_pages, v_pages, k_exp, v_exp, page_table, cache_lens);
  if (rc != PI_OK) return rc;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return PI_ERR_ALIGN;
  DevCtl ctl;
  if (!make_ctl(&ctl)) return PI_ERR_CUDA;
  CacheParams p = cache_params(d);
  p.k_out = k_out; p.v_out = v_out;
  p.kp = const_cast<void*>(k_pages); p.vp = const_cast<void*>(v_pages);
  p.ke = const_cast<uint8_t*>(k_exp); p.ve = const_cast<uint8_t*>(v_exp);
  p.table = page_table; p.lens = cache_lens;
  p.valid_out = valid_out;
  return launched(launch_cache(p, false, d->dtype == PI_F32, d->cache_dtype, ctl,
                               static_cast<cudaStream_t>(stream)));
}

size_t pi_attn_paged_workspace_bytes(const pi_paged_desc* d) {
  if (check_attn(d) != PI_OK || d->B == 0 || d->Sq == 0) return 0;
  const PagedParams p = paged_params(d);
  if (paged_decode_applies(p)) return paged_decode_workspace_bytes(p);
  return paged_tc_applies(p) ? paged_tc_workspace_bytes(p) : 0;
}

int pi_attn_paged(const pi_paged_desc* d, const void* q, const void* k_new, const void* v_new,
                  const uint8_t* ar_mask, const int32_t* segment_ids, const void* k_pages,
                  const void* v_pages, const uint8_t* k_exp, const uint8_t* v_exp,
                  const int32_t* page_table, const int32_t* cache_lens, void* out, float* lse,
                  void* workspace, size_t ws_bytes, pi_stream_t stream) {
  NvtxRange range("pi_attn_paged");
  int rc = check_attn(d);
  if (rc != PI_OK) return rc;
  if (d->B == 0 || d->Sq == 0) return PI_OK;
  if (!q || !k_new || !v_new || !ar_mask || !out) return PI_ERR_ARG;
  rc = check_cache(d, k_pages, v_pages, k_exp, v_exp, page_table, cache_lens);
  if (rc != PI_OK) return rc;
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(segment_ids, 4))
    return PI_ERR_ALIGN;
  const size_t need = pi_attn_paged_workspace_bytes(d);
  if (need > 0) {
    if (!workspace || ws_bytes < need) return PI_ERR_ARG;
    if (!aligned(workspace, 16)) return PI_ERR_ALIGN;
  }
  DevCtl ctl;
  if (!make_ctl(&ctl)) return PI_ERR_CUDA;
  PagedParams p = paged_params(d);
  p.q = q; p.k = k_new; p.v = v_new;
  p.kp = k_pages; p.vp = v_pages; p.ke = k_exp; p.ve = v_exp;
  p.table = page_table; p.lens = cache_lens;
  p.ar = ar_mask; p.seg = segment_ids;
  p.out = out; p.lse = lse;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* ws = need > 0 ? static_cast<float*>(workspace) : nullptr;
  if (paged_decode_applies(p)) return launched(launch_paged_decode(p, ws, ctl, st));
  if (paged_tc_applies(p)) return launched(launch_paged_tc(p, ws, ctl, st));
  return launched(launch_paged_simt(p, ctl, st));
}

}  // extern "C"
