/* A plain C11 client of the paged-cache calls: the descriptor's layout, which
 * bindings in other languages repeat, and calls that are settled on the host
 * (refusals and no-ops; no GPU is touched). */
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "pi_attn.h"

static int failures;
#define CHECK(x)                                                     \
  do {                                                               \
    if (!(x)) {                                                      \
      fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #x);        \
      ++failures;                                                    \
    }                                                                \
  } while (0)

int main(void) {
  pi_paged_desc d;
  int32_t lens[2] = {0, 0}, after[2], table[2] = {0, 1};
  static _Alignas(16) char buf[64];

#define FIELD(f) printf("%s %zu %zu\n", #f, offsetof(pi_paged_desc, f), sizeof(d.f))
  FIELD(B); FIELD(Sq); FIELD(Hq); FIELD(Hkv); FIELD(d); FIELD(dtype); FIELD(cache_dtype);
  FIELD(page_size); FIELD(num_pages); FIELD(max_pages); FIELD(window); FIELD(sinks);
  FIELD(softmax_scale); FIELD(reserved); FIELD(mask_batch_stride);
  printf("size %zu\n", sizeof(pi_paged_desc));
  CHECK(PI_BF16 == 0 && PI_F32 == 1 && PI_E4M3 == 2);

  memset(&d, 0, sizeof(d));
  d.B = 2; d.Sq = 1; d.Hq = 8; d.Hkv = 1; d.d = 256; d.dtype = PI_BF16; d.cache_dtype = PI_E4M3;
  d.page_size = 16; d.num_pages = 2; d.max_pages = 1; d.softmax_scale = 1.f;

  CHECK(pi_attn_cache_write(NULL, buf, buf, NULL, table, lens, buf, buf, NULL, NULL, after, NULL) ==
        PI_ERR_ARG);
  /* the exponents of an e4m3 pool are missing */
  CHECK(pi_attn_cache_write(&d, buf, buf, NULL, table, lens, buf, buf, NULL, NULL, after, NULL) ==
        PI_ERR_ARG);
  CHECK(pi_attn_cache_read(&d, buf, buf, NULL, NULL, table, lens, buf, buf, NULL, NULL) ==
        PI_ERR_ARG);
  CHECK(pi_attn_paged(&d, buf, buf, buf, (const uint8_t*)buf, NULL, buf, buf, NULL, NULL, table,
                      lens, buf, NULL, NULL, 0, NULL) == PI_ERR_ARG);
  d.cache_dtype = PI_F32;                       /* not the tensors' type, nor e4m3 */
  CHECK(pi_attn_cache_read(&d, buf, buf, NULL, NULL, table, lens, buf, buf, NULL, NULL) ==
        PI_ERR_UNSUPPORTED);
  d.cache_dtype = PI_BF16;
  CHECK(pi_attn_cache_write(&d, buf, buf, NULL, table, lens, buf, buf, NULL, NULL, lens, NULL) ==
        PI_ERR_ARG);                            /* lens_out is cache_lens */
  (void)pi_attn_paged_workspace_bytes(&d);
  CHECK(pi_attn_paged_workspace_bytes(NULL) == 0);
  d.B = 0;
  CHECK(pi_attn_cache_write(&d, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL) ==
        PI_OK);
  CHECK(pi_attn_cache_read(&d, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL) == PI_OK);
  CHECK(pi_attn_paged(&d, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL,
                      NULL, NULL, 0, NULL) == PI_OK);

  if (failures) return 1;
  printf("c abi ok\n");
  return 0;
}
