/* Calls every entry point of qlora_mx.h with invalid arguments and with valid
 * ones against host-only stand-ins of the launchers: every invalid call must
 * fail with a message before a launcher is reached, every valid one must reach
 * exactly one. Prints "reject_mx: ok" and exits 0 on success. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/qlora_mx.h"

extern int qlora_stub_launches;

static int failures = 0;

static void check(const char *what, int got, int before, int valid) {
  const int reached = qlora_stub_launches - before;
  const int good = valid ? got == QLORA_ERR_HIP && reached == 1
                         : got < 0 && got != QLORA_ERR_HIP && reached == 0 && qlora_last_error()[0] != '\0';
  if (!good) {
    printf("FAIL %s: got %d, launches %d (%s)\n", what, got, reached, qlora_last_error());
    ++failures;
  }
}

#define REJ(call)                       \
  do {                                  \
    const int n0 = qlora_stub_launches; \
    check(#call, (call), n0, 0);        \
  } while (0)
#define REACH(call)                     \
  do {                                  \
    const int n0 = qlora_stub_launches; \
    check(#call, (call), n0, 1);        \
  } while (0)

static char *p;   /* never dereferenced by the layer */

static qlora_mx_matrix mat(int64_t rows, int64_t cols, int type) {
  qlora_mx_matrix m;
  memset(&m, 0, sizeof(m));
  m.rows = rows;
  m.cols = cols;
  m.codes = (uint8_t *)p;
  m.scales = (uint8_t *)p + 4096;
  m.type = type;
  return m;
}

int main(void) {
  p = (char *)aligned_alloc(256, 1 << 16);
  qlora_mx_matrix a = mat(8, 64, QLORA_MX_FP8), w = mat(16, 64, QLORA_MX_FP4), bad;
  void *q = p + 8192;
  const int64_t huge = INT64_MAX;

  REACH(qlora_mx_quantize(q, QLORA_F32, 8, 64, &a, NULL));
  REACH(qlora_mx_quantize(q, QLORA_BF16, 16, 64, &w, NULL));
  REJ(qlora_mx_quantize(NULL, QLORA_F32, 8, 64, &a, NULL));
  REJ(qlora_mx_quantize(q, 7, 8, 64, &a, NULL));
  REJ(qlora_mx_quantize(q, QLORA_F32, 8, 64, NULL, NULL));
  REJ(qlora_mx_quantize(q, QLORA_F32, 9, 64, &a, NULL));
  REJ(qlora_mx_quantize(p + 1, QLORA_F32, 8, 64, &a, NULL));
  for (int i = 0; i < 9; ++i) {
    bad = a;
    if (i == 0) bad.rows = 0;
    if (i == 1) bad.rows = huge;
    if (i == 2) bad.cols = 0;
    if (i == 3) bad.cols = 65;
    if (i == 4) bad.cols = huge - 31;
    if (i == 5) bad.codes = NULL;
    if (i == 6) bad.scales = NULL;
    if (i == 7) bad.scales += 3;
    if (i == 8) bad.type = 2;
    REJ(qlora_mx_quantize(q, QLORA_F32, bad.rows, bad.cols, &bad, NULL));
    REJ(qlora_mx_dequantize(&bad, q, QLORA_F32, NULL));
    REJ(qlora_mx_linear(&bad, &w, q, NULL));
    REJ(qlora_mx_linear(&a, &bad, q, NULL));
    REJ(qlora_mx_linear_grouped(&bad, &w, (int32_t *)p, 2, q, NULL));
    REJ(qlora_rmsnorm_mx(q, NULL, q, QLORA_F32, bad.rows, bad.cols, 1e-6, &bad, NULL, NULL));
  }
  REACH(qlora_mx_dequantize(&a, q, QLORA_BF16, NULL));
  REJ(qlora_mx_dequantize(&a, NULL, QLORA_BF16, NULL));
  REJ(qlora_mx_dequantize(&a, q, -1, NULL));
  REJ(qlora_mx_dequantize(&a, p + 8, QLORA_BF16, NULL));

  REACH(qlora_mx_linear(&a, &w, q, NULL));
  REACH(qlora_mx_linear(&w, &w, q, NULL));
  REJ(qlora_mx_linear(&a, &a, q, NULL));
  REJ(qlora_mx_linear(&a, &w, NULL, NULL));
  REJ(qlora_mx_linear(&a, &w, p + 2, NULL));
  bad = mat(16, 96, QLORA_MX_FP4);
  REJ(qlora_mx_linear(&a, &bad, q, NULL));
  bad = mat((int64_t)1 << 25, 64, QLORA_MX_FP4);
  REJ(qlora_mx_linear(&a, &bad, q, NULL));
  REACH(qlora_mx_linear_grouped(&a, &w, (int32_t *)(p + 4), 16, q, NULL));
  REJ(qlora_mx_linear_grouped(&a, &w, NULL, 2, q, NULL));
  REJ(qlora_mx_linear_grouped(&a, &w, (int32_t *)(p + 2), 2, q, NULL));
  REJ(qlora_mx_linear_grouped(&a, &w, (int32_t *)p, 0, q, NULL));
  REJ(qlora_mx_linear_grouped(&a, &w, (int32_t *)p, 3, q, NULL));
  REJ(qlora_mx_linear_grouped(&a, &w, (int32_t *)p, INT32_MAX, q, NULL));

  REACH(qlora_rmsnorm_fwd(p, NULL, p, QLORA_F32, 8, 64, 0.0, q, NULL, NULL, NULL));
  REACH(qlora_rmsnorm_fwd(p, p, p, QLORA_BF16, 8, 64, 1e-6, q, p, (float *)p, NULL));
  REACH(qlora_rmsnorm_mx(q, q, q, QLORA_F32, 8, 64, 1e-6, &a, q, NULL));
  REJ(qlora_rmsnorm_fwd(p, p, p, QLORA_BF16, 8, 64, 1e-6, q, NULL, NULL, NULL));
  REJ(qlora_rmsnorm_fwd(p, NULL, p, QLORA_BF16, 8, 64, 1e-6, q, p, NULL, NULL));
  REJ(qlora_rmsnorm_fwd(p, p, p, QLORA_BF16, 8, 64, 1e-6, q, q, NULL, NULL));
  REJ(qlora_rmsnorm_fwd(p, p, p, QLORA_BF16, 8, 32800, 1e-6, q, p, NULL, NULL));
  REJ(qlora_rmsnorm_fwd(p, p, p, QLORA_BF16, huge, 64, 1e-6, q, p, NULL, NULL));
  REJ(qlora_rmsnorm_fwd(p, p, p, QLORA_BF16, 8, 64, NAN, q, p, NULL, NULL));
  REJ(qlora_rmsnorm_fwd(p, p, p, QLORA_BF16, 8, 64, -1.0, q, p, NULL, NULL));
  REJ(qlora_rmsnorm_fwd(p, p, p, 3, 8, 64, 1e-6, q, p, NULL, NULL));
  REJ(qlora_rmsnorm_mx(q, q, q, QLORA_F32, 9, 64, 1e-6, &a, q, NULL));

  const size_t need = qlora_rmsnorm_bwd_workspace_bytes(8, 64);
  REACH(qlora_rmsnorm_bwd(p, q, p, QLORA_F32, (float *)p, NULL, 8, 64, p, (float *)p, p, need, NULL));
  REACH(qlora_rmsnorm_bwd(p, q, p, QLORA_F32, (float *)p, p, 2, 64, p, (float *)p, NULL, 0, NULL));
  REJ(qlora_rmsnorm_bwd(p, q, p, QLORA_F32, (float *)p, p, 8, 64, p, (float *)p, NULL, 0, NULL));
  REJ(qlora_rmsnorm_bwd(p, q, p, QLORA_F32, (float *)p, p, 8, 64, p, (float *)p, p, need - 1, NULL));
  REJ(qlora_rmsnorm_bwd(p, q, p, QLORA_F32, (float *)p, p, 8, 64, p, (float *)p, p + 8, need, NULL));
  REJ(qlora_rmsnorm_bwd(p, q, p, QLORA_F32, (float *)p, p, 8, 64, q, (float *)p, p, need, NULL));
  REJ(qlora_rmsnorm_bwd(p, q, p, QLORA_F32, NULL, p, 8, 64, p, (float *)p, p, need, NULL));
  if (qlora_rmsnorm_bwd_workspace_bytes(huge, 64) || qlora_mx_storage_bytes(huge, 64, 0) || qlora_mx_scale_pitch(huge - 31)) ++failures;
  free(p);
  if (failures) return 1;
  printf("reject_mx: ok\n");
  return 0;
}
