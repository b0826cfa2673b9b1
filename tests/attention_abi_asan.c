/* Drives the argument checks of include/ipttt_attention.h with host pointers: every call is
 * refused or has nothing to do, so none reaches the device. Built with AddressSanitizer and
 * UndefinedBehaviorSanitizer by tests/test_attention_abi.py. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "ipttt_attention.h"

static int failures;
#define EXPECT(call, status)                                                            \
  do {                                                                                  \
    ipttt_status got = (call);                                                          \
    if (got != (status)) {                                                              \
      printf("line %d: %s, expected %s (%s)\n", __LINE__, ipttt_status_str(got),        \
             ipttt_status_str(status), ipttt_last_error());                             \
      ++failures;                                                                       \
    } else if (got != IPTTT_OK &&                                                       \
               strncmp(ipttt_last_error(), ipttt_status_str(got), strlen(ipttt_status_str(got)))) { \
      printf("line %d: message %s\n", __LINE__, ipttt_last_error());                    \
      ++failures;                                                                       \
    }                                                                                   \
  } while (0)

int main(void) {
  char *raw = (char *)malloc(4096 + 256);
  if (!raw) return 1;
  char *p = (char *)(((uintptr_t)raw + 255) & ~(uintptr_t)255);
  float *f = (float *)p;
  int32_t *i32 = (int32_t *)p;
  ipttt_heads x = {p, 128, 64}, far = {p, INT64_MAX, 64}, low = {p, INT64_MIN, INT64_MIN}, odd = {p + 1, 128, 64};
  ipttt_heads none = {NULL, 0, 0};

  ipttt_headnorm_desc hd = {2, 1, 64, 64, 0, IPTTT_BF16, 1e-6f, p, p, (const double *)p};
  EXPECT(ipttt_headnorm_forward(NULL, &x, &x, i32, 2, &x, &x, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_forward(&hd, NULL, &x, i32, 2, &x, &x, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_forward(&hd, &far, &x, i32, 2, &x, &x, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_forward(&hd, &low, &x, i32, 2, &x, &x, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_forward(&hd, &odd, &x, i32, 2, &x, &x, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_forward(&hd, &x, &x, NULL, 2, &x, &x, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_forward(&hd, &x, &x, i32, INT64_MAX, &x, &x, NULL), IPTTT_E_UNSUPPORTED);
  EXPECT(ipttt_headnorm_forward(&hd, &x, &x, i32, INT64_MIN, &x, &x, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_forward(&hd, &none, &none, NULL, 0, &none, &none, NULL), IPTTT_OK);
  EXPECT(ipttt_headnorm_backward(&hd, &x, &x, i32, &x, &x, 2, &x, &x, f, f, p, 1, NULL), IPTTT_E_WORKSPACE);
  EXPECT(ipttt_headnorm_backward(&hd, &x, &x, i32, &x, &x, 2, &x, &x, f, f, p + 8, 1 << 20, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_backward(&hd, &x, &x, i32, &x, NULL, 2, &x, &x, f, f, p, 1 << 20, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_backward(&hd, NULL, NULL, NULL, NULL, NULL, 0, NULL, NULL, NULL, NULL, NULL, 0, NULL),
         IPTTT_OK);

  ipttt_kv_cache cache = {p, p, 4, 16, 1, 64, IPTTT_BF16};
  ipttt_page_table table = {i32, 4, 2, 4};
  EXPECT(ipttt_headnorm_append(&hd, &x, &x, &x, i32, NULL, 2, &x, NULL, &table, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_append(&hd, &x, &x, &x, i32, NULL, 2, &x, &cache, NULL, NULL), IPTTT_E_INVALID);
  ipttt_page_table huge = {i32, INT64_MAX, 65535, INT32_MAX};
  EXPECT(ipttt_headnorm_append(&hd, &x, &x, &x, i32, NULL, 2, &x, &cache, &huge, NULL), IPTTT_E_UNSUPPORTED);
  huge.width = 8;
  EXPECT(ipttt_headnorm_append(&hd, &x, &x, &x, i32, NULL, 2, &x, &cache, &huge, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_headnorm_append(&hd, &none, &none, &none, NULL, NULL, 0, &none, &cache, &table, NULL), IPTTT_OK);

  ipttt_attention ad = {2, 1, 64, 1, 1, 0, IPTTT_BF16, 0.125f, 2, 2, i32, i32};
  EXPECT(ipttt_attention_forward(NULL, &x, &x, &x, &x, f, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_attention_forward(&ad, &x, &far, &x, &x, f, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_attention_forward(&ad, &x, &x, &low, &x, f, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_attention_forward(&ad, &x, &x, &x, &x, f, p, 0, NULL), IPTTT_E_WORKSPACE);
  EXPECT(ipttt_attention_forward(&ad, &x, &x, &x, &x, f, NULL, 4096, NULL), IPTTT_E_INVALID);
  ipttt_attention big = ad;
  big.n_q = INT64_MAX;
  EXPECT(ipttt_attention_forward(&big, &x, &x, &x, &x, f, p, 4096, NULL), IPTTT_E_UNSUPPORTED);
  if (ipttt_attention_forward_workspace_bytes(&big) || ipttt_attention_backward_workspace_bytes(&big) ||
      ipttt_attention_backward_workspace_bytes(NULL))
    ++failures;
  big.n_q = big.n_k = (int64_t)1 << 30;
  big.q_heads = 1024;
  EXPECT(ipttt_attention_forward(&big, &x, &x, &x, &x, f, p, 4096, NULL), IPTTT_E_UNSUPPORTED);
  big = ad;
  big.n_q = big.n_k = 0;
  EXPECT(ipttt_attention_forward(&big, &none, &none, &none, &none, NULL, NULL, 0, NULL), IPTTT_OK);
  EXPECT(ipttt_attention_backward(&big, &none, &none, &none, &none, NULL, &none, &none, &none, &none, NULL, 0, NULL),
         IPTTT_OK);
  EXPECT(ipttt_attention_backward(&ad, &x, &x, &x, &x, NULL, &x, &x, &x, &x, p, 1 << 20, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_attention_backward(&ad, &x, &x, &x, &x, f, &x, &x, &x, &x, p, 16, NULL), IPTTT_E_WORKSPACE);

  ipttt_step_desc sd = {2, 0, 0.125f};
  EXPECT(ipttt_attention_step(NULL, &x, &cache, &table, i32, &x, f, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_attention_step(&sd, &x, NULL, &table, i32, &x, f, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_attention_step(&sd, &x, &cache, NULL, i32, &x, f, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_attention_step(&sd, &x, &cache, &table, NULL, &x, f, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_attention_step(&sd, &far, &cache, &table, i32, &x, f, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_attention_step(&sd, &x, &cache, &table, i32, &x, f, p, 0, NULL), IPTTT_E_WORKSPACE);
  sd.scale = NAN;
  EXPECT(ipttt_attention_step(&sd, &x, &cache, &table, i32, &x, f, p, 4096, NULL), IPTTT_E_INVALID);
  sd.scale = 1.f;
  ipttt_page_table empty = {NULL, 0, 0, 0};
  EXPECT(ipttt_attention_step(&sd, &none, &cache, &empty, NULL, &none, NULL, NULL, 0, NULL), IPTTT_OK);
  free(raw);
  printf(failures ? "%d failures\n" : "all checks passed\n", failures);
  return failures != 0;
}
