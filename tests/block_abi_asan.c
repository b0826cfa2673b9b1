/* Drives the argument checks of include/ipttt_block.h with host pointers: every call
 * is refused or has nothing to do, so none reaches the device. Built with
 * AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_block_abi.py. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "ipttt_block.h"

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

  ipttt_norm_desc nd = {64, IPTTT_F32, 1e-5f, p, p};
  EXPECT(ipttt_norm_forward(NULL, p, 64, NULL, 0, 1, NULL, p, f, f, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_norm_forward(&nd, NULL, 64, NULL, 0, 1, NULL, p, f, f, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_norm_forward(&nd, p, 64, p, 64, 1, NULL, p, f, f, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_norm_forward(&nd, p, 64, NULL, 0, INT64_MAX, NULL, p, f, f, NULL), IPTTT_E_UNSUPPORTED);
  EXPECT(ipttt_norm_forward(&nd, p, INT64_MAX, NULL, 0, 1000, NULL, p, f, f, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_norm_forward(&nd, p, INT64_MIN, NULL, 0, 1000, NULL, p, f, f, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_norm_forward(&nd, NULL, 0, NULL, 0, 0, NULL, NULL, NULL, NULL, NULL), IPTTT_OK);
  EXPECT(ipttt_norm_backward(&nd, p, 64, f, f, p, 64, p, 64, 3, p, f, f, p, 1, NULL), IPTTT_E_WORKSPACE);
  EXPECT(ipttt_norm_backward(&nd, NULL, 0, NULL, NULL, NULL, 0, NULL, 0, 0, NULL, NULL, NULL, NULL, 0, NULL),
         IPTTT_OK);
  if (ipttt_norm_backward_workspace_bytes(NULL, 1) != 0) ++failures;
  nd.d = -1;
  if (ipttt_norm_backward_workspace_bytes(&nd, 1) != 0) ++failures;
  EXPECT(ipttt_norm_forward(&nd, p, 64, NULL, 0, 1, NULL, p, f, f, NULL), IPTTT_E_INVALID);

  ipttt_view v = {p, 640, 64};
  ipttt_recurrence r;
  memset(&r, 0, sizeof r);
  r.batch = 2;
  r.d = 64;
  r.seq_len = 10;
  r.dtype = IPTTT_BF16;
  r.g = r.v = r.h = v;
  EXPECT(ipttt_recurrence_forward(NULL, f, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_recurrence_forward(&r, f, p, 0, NULL), IPTTT_E_WORKSPACE);
  EXPECT(ipttt_recurrence_step(&r, f, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_recurrence_backward(&r, NULL, f, &v, &v, NULL, p, 4096, NULL), IPTTT_E_INVALID);
  r.batch = INT32_MAX;
  EXPECT(ipttt_recurrence_forward(&r, f, p, 4096, NULL), IPTTT_E_UNSUPPORTED);
  r.batch = 65535;
  r.d = 65536;
  r.seq_len = (int64_t)1 << 30;
  EXPECT(ipttt_recurrence_forward(&r, f, p, 4096, NULL), IPTTT_E_UNSUPPORTED);
  if (ipttt_recurrence_workspace_bytes(&r) != 0) ++failures;
  r.batch = 1;
  r.d = 1;
  if (ipttt_recurrence_workspace_bytes(&r) == 0) ++failures;
  r.g.tok_stride = INT64_MAX;
  EXPECT(ipttt_recurrence_forward(&r, f, p, 4096, NULL), IPTTT_E_INVALID);
  r.g = v;
  r.seq_len = INT64_MAX;
  EXPECT(ipttt_recurrence_forward(&r, f, p, 4096, NULL), IPTTT_E_UNSUPPORTED);
  r.batch = 0;
  r.seq_len = 4;
  EXPECT(ipttt_recurrence_forward(&r, f, NULL, 0, NULL), IPTTT_OK);

  ipttt_ff_desc fd = {64, 128, IPTTT_BF16, p, p, p};
  ipttt_ff_grads g = {p, 64, p, p, p};
  EXPECT(ipttt_ff_forward(NULL, p, 64, 1, p, 64, NULL, NULL, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_ff_forward(&fd, p, 64, 100, p, 64, NULL, NULL, p, 16, NULL), IPTTT_E_WORKSPACE);
  EXPECT(ipttt_ff_forward(&fd, p, 64, 100, p, 64, f, NULL, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_ff_forward(&fd, p, 64, INT64_MAX, p, 64, NULL, NULL, p, 4096, NULL), IPTTT_E_UNSUPPORTED);
  EXPECT(ipttt_ff_forward(&fd, NULL, 0, 0, NULL, 0, NULL, NULL, NULL, 0, NULL), IPTTT_OK);
  EXPECT(ipttt_ff_backward(&fd, p, 64, f, f, p, 64, 100, NULL, p, 4096, NULL), IPTTT_E_INVALID);
  EXPECT(ipttt_ff_backward(&fd, p, 64, f, f, p, 64, 100, &g, p, 4096, NULL), IPTTT_E_WORKSPACE);
  /* the largest sizes: workspace arithmetic stays within 64 bits */
  fd.d = 1 << 16;
  fd.d_ff = 1 << 18;
  fd.dtype = IPTTT_F32;
  if (ipttt_ff_workspace_bytes(&fd, 1 << 24) == 0) ++failures;
  if (ipttt_ff_backward_workspace_bytes(&fd, 1 << 24) < ipttt_ff_workspace_bytes(&fd, 1 << 24)) ++failures;
  if (ipttt_ff_workspace_bytes(NULL, 1) != 0) ++failures;

  free(raw);
  if (failures) {
    printf("%d failures\n", failures);
    return 1;
  }
  printf("all checks passed\n");
  return 0;
}
