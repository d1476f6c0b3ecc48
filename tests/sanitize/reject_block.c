/* Calls every entry point of qlora_block.h with invalid arguments and with
 * valid ones against host-only stand-ins of the launchers. Every invalid call
 * must fail with a message before a launcher is reached, every valid one must
 * reach it (and then fail with QLORA_ERR_HIP, as the stand-ins do). Buffers
 * are host memory: the layer never dereferences a device pointer. Prints
 * "reject_block: ok" and exits 0 on success. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/qlora_block.h"

extern int qlora_stub_launches;

static int failures = 0;

static void check(const char *what, int got, int before, int invalid) {
  const int ok = invalid ? got < 0 && got != QLORA_ERR_HIP && qlora_stub_launches == before && qlora_last_error()[0] != '\0'
                         : got == QLORA_ERR_HIP && qlora_stub_launches == before + 1;
  if (!ok) {
    printf("FAIL %s: got %d, launches %d -> %d (%s)\n", what, got, before, qlora_stub_launches, qlora_last_error());
    ++failures;
  }
}

#define REJ(call)                       \
  do {                                  \
    const int n0 = qlora_stub_launches; \
    check(#call, (call), n0, 1);        \
  } while (0)
#define REACH(call)                     \
  do {                                  \
    const int n0 = qlora_stub_launches; \
    check(#call, (call), n0, 0);        \
  } while (0)
#define WITH(type, name, from, change, line) \
  do {                                       \
    type name = from;                        \
    change;                                  \
    line;                                    \
  } while (0)

static char *pool;

static qlora_mx_matrix matrix(int64_t rows, int64_t cols, int type) {
  qlora_mx_matrix m = {rows, cols, (uint8_t *)pool, (uint8_t *)(pool + 65536), type};
  return m;
}

static qlora_nf4_weight weight(int64_t rows, int64_t cols, int format) {
  qlora_nf4_weight w;
  memset(&w, 0, sizeof w);
  w.rows = rows;
  w.cols = cols;
  w.codes = (uint8_t *)pool;
  w.absmax_q = (int8_t *)(pool + 65536);
  w.dq_scale = (float *)(pool + 66560);
  w.dq_mean = (float *)(pool + 67584);
  w.absmax = (float *)(pool + 68608);
  w.format = format;
  return w;
}

static void microscaled(void) {
  const qlora_mx_matrix g = matrix(64, 64, QLORA_MX_FP4), pair = matrix(128, 64, QLORA_MX_FP4);
  REJ(qlora_mx_pair(NULL, &g, &pair, NULL));
  REJ(qlora_mx_pair(&g, NULL, &pair, NULL));
  REJ(qlora_mx_pair(&g, &g, NULL, NULL));
  REJ(qlora_mx_pair(&g, &g, &g, NULL));
  WITH(qlora_mx_matrix, m, g, m.rows = INT64_MAX, REJ(qlora_mx_pair(&m, &m, &pair, NULL)));
  WITH(qlora_mx_matrix, m, g, m.type = QLORA_MX_FP8, REJ(qlora_mx_pair(&m, &g, &pair, NULL)));
  REACH(qlora_mx_pair(&g, &g, &pair, NULL));
  const qlora_mx_matrix x = matrix(5, 64, QLORA_MX_FP8), h = matrix(5, 64, QLORA_MX_FP8);
  REJ(qlora_mx_gated(NULL, &pair, pool, NULL, NULL));
  REJ(qlora_mx_gated(&x, NULL, pool, NULL, NULL));
  REJ(qlora_mx_gated(&x, &pair, NULL, NULL, NULL));
  REJ(qlora_mx_gated(&x, &pair, pool, &h, NULL));
  REJ(qlora_mx_gated(&x, &pair, pool + 8, NULL, NULL));
  WITH(qlora_mx_matrix, m, pair, m.rows = 96, REJ(qlora_mx_gated(&x, &m, pool, NULL, NULL)));
  WITH(qlora_mx_matrix, m, pair, m.rows = INT64_MAX - 63, REJ(qlora_mx_gated(&x, &m, pool, NULL, NULL)));
  WITH(qlora_mx_matrix, m, x, m.rows = INT64_MAX, REJ(qlora_mx_gated(&m, &pair, pool, NULL, NULL)));
  WITH(qlora_mx_matrix, m, h, m.cols = 32, REJ(qlora_mx_gated(&x, &pair, NULL, &m, NULL)));
  WITH(qlora_mx_matrix, m, h, m.scales = NULL, REJ(qlora_mx_gated(&x, &pair, NULL, &m, NULL)));
  REACH(qlora_mx_gated(&x, &pair, pool, NULL, NULL));
  REACH(qlora_mx_gated(&x, &pair, NULL, &h, NULL));
  const int32_t *off = (const int32_t *)pool;
  REJ(qlora_mx_gated_grouped(&x, &pair, off, 0, pool, NULL, 0, NULL));
  REJ(qlora_mx_gated_grouped(&x, &pair, off, INT32_MIN, pool, NULL, 0, NULL));
  REJ(qlora_mx_gated_grouped(&x, &pair, off, INT32_MAX, pool, NULL, 0, NULL));
  REJ(qlora_mx_gated_grouped(&x, &pair, NULL, 2, pool, NULL, 0, NULL));
  REJ(qlora_mx_gated_grouped(&x, &pair, off, 4, pool, NULL, 0, NULL));
  REACH(qlora_mx_gated_grouped(&x, &pair, off, 2, pool, NULL, 0, NULL));
}

static void block(int format) {
  const qlora_nf4_weight g = weight(128, 192, format), u = g;
  const qlora_gated_adapters ad = {pool, pool, pool, pool, 8, QLORA_BF16, 2.0f};
  const qlora_gated_grads grads = {pool, pool, pool, pool};
  const int64_t M = 40;
  const size_t fws = qlora_gated_workspace_bytes(M, 128, 192, 8, 0), bws = qlora_gated_workspace_bytes(M, 128, 192, 8, 1);
  char *ws = pool + 131072, *p = pool;
#define FWD(g, u, ad, G, U, Hs, ws, n) qlora_gated_fwd(p, M, g, u, ad, p, G, U, Hs, ws, n, NULL)
  REACH(FWD(&g, &u, &ad, NULL, NULL, NULL, ws, fws));
  REACH(FWD(&g, &u, &ad, p, p, p, ws, fws));
  REACH(FWD(&g, &u, NULL, p, p, NULL, ws, fws));
  REJ(FWD(NULL, &u, &ad, NULL, NULL, NULL, ws, fws));
  REJ(FWD(&g, NULL, &ad, NULL, NULL, NULL, ws, fws));
  REJ(FWD(&g, &u, &ad, p, NULL, NULL, ws, fws));
  REJ(FWD(&g, &u, &ad, p, p, NULL, ws, fws));
  REJ(FWD(&g, &u, &ad, NULL, NULL, p, ws, fws));
  REJ(FWD(&g, &u, NULL, p, p, p, ws, fws));
  REJ(FWD(&g, &u, &ad, p, p, p + 8, ws, fws));
  REJ(FWD(&g, &u, &ad, p + 2, p, p, ws, fws));
  REJ(FWD(&g, &u, &ad, p, p, p, NULL, fws));
  REJ(FWD(&g, &u, &ad, p, p, p, ws, fws - 1));
  REJ(FWD(&g, &u, &ad, p, p, p, ws + 8, fws));
  REJ(qlora_gated_fwd(NULL, M, &g, &u, &ad, p, NULL, NULL, NULL, ws, fws, NULL));
  REJ(qlora_gated_fwd(p, M, &g, &u, &ad, NULL, NULL, NULL, NULL, ws, fws, NULL));
  REJ(qlora_gated_fwd(p + 4, M, &g, &u, &ad, p, NULL, NULL, NULL, ws, fws, NULL));
  const int64_t rows[] = {0, -1, INT64_MIN, INT64_MAX, (1 << 24) + 1};
  for (size_t i = 0; i < sizeof rows / sizeof *rows; ++i) REJ(qlora_gated_fwd(p, rows[i], &g, &u, &ad, p, NULL, NULL, NULL, ws, 1u << 20, NULL));
  WITH(qlora_nf4_weight, w, g, w.rows = 64, REJ(FWD(&g, &w, &ad, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_nf4_weight, w, g, w.cols = 96, REJ(FWD(&w, &w, &ad, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_nf4_weight, w, g, w.rows = 100, REJ(FWD(&w, &w, &ad, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_nf4_weight, w, g, w.rows = INT64_MAX - 63, REJ(FWD(&w, &w, &ad, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_nf4_weight, w, g, w.rows = w.cols = (int64_t)1 << 23, REJ(FWD(&w, &w, &ad, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_nf4_weight, w, g, w.codes = NULL, REJ(FWD(&g, &w, &ad, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_nf4_weight, w, g, w.format = 42, REJ(FWD(&w, &w, &ad, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_nf4_weight, w, g, w.format = format == QLORA_FMT_NF4 ? QLORA_FMT_NF4_DQ : QLORA_FMT_NF4,
       REJ(FWD(&g, &w, &ad, NULL, NULL, NULL, ws, fws)));
  const int32_t ranks[] = {0, -1, 257, INT32_MIN, INT32_MAX};
  for (size_t i = 0; i < sizeof ranks / sizeof *ranks; ++i)
    WITH(qlora_gated_adapters, a, ad, a.r = ranks[i], REJ(FWD(&g, &u, &a, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_gated_adapters, a, ad, a.dtype = 7, REJ(FWD(&g, &u, &a, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_gated_adapters, a, ad, a.up_B = NULL, REJ(FWD(&g, &u, &a, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_gated_adapters, a, ad, a.gate_A = p + 8, REJ(FWD(&g, &u, &a, NULL, NULL, NULL, ws, fws)));
  WITH(qlora_gated_adapters, a, ad, a.scale = NAN, REJ(FWD(&g, &u, &a, NULL, NULL, NULL, ws, fws)));
#define BWD(Hs, ad, grads, ws, n) qlora_gated_bwd(p, p, p, p, Hs, M, &g, &u, ad, p, grads, ws, n, NULL)
  REACH(BWD(p, &ad, &grads, ws, bws));
  REACH(BWD(NULL, NULL, NULL, ws, bws));
  REJ(BWD(NULL, &ad, &grads, ws, bws));
  REJ(BWD(p, &ad, NULL, ws, bws));
  REJ(BWD(p, NULL, NULL, ws, bws));
  REJ(BWD(NULL, NULL, &grads, ws, bws));
  REJ(BWD(p, &ad, &grads, NULL, bws));
  REJ(BWD(p, &ad, &grads, ws, bws - 1));
  WITH(qlora_gated_grads, q, grads, q.up_A = NULL, REJ(BWD(p, &ad, &q, ws, bws)));
  WITH(qlora_gated_grads, q, grads, q.gate_B = p + 4, REJ(BWD(p, &ad, &q, ws, bws)));
  for (int i = 0; i < 5; ++i) {   /* each tensor missing, or out of line */
    const void *t[5] = {p, p, p, p, p};
    t[i] = NULL;
    REJ(qlora_gated_bwd(t[0], t[1], t[2], t[3], p, M, &g, &u, &ad, (void *)t[4], &grads, ws, bws, NULL));
    t[i] = p + 2;
    REJ(qlora_gated_bwd(t[0], t[1], t[2], t[3], p, M, &g, &u, &ad, (void *)t[4], &grads, ws, bws, NULL));
  }
}

static void rope(void) {
  double f[64], amplitude;
  const double bad[] = {0.0, -1.0, INFINITY, NAN};
  for (size_t i = 0; i < sizeof bad / sizeof *bad; ++i) {
    REJ(qlora_rope_freqs(128, bad[i], QLORA_ROPE_PLAIN, 1.0, 1, 1.0, 2.0, f, &amplitude));
    REJ(qlora_rope_freqs(128, 1e4, QLORA_ROPE_LINEAR, bad[i], 1, 1.0, 2.0, f, &amplitude));
    REJ(qlora_rope_freqs(128, 1e4, QLORA_ROPE_PARTS, 2.0, 4096, 2.0, bad[i], f, &amplitude));
  }
  const int32_t rots[] = {0, 1, 3, -2, 1026, INT32_MIN, INT32_MAX};
  for (size_t i = 0; i < sizeof rots / sizeof *rots; ++i)
    REJ(qlora_rope_freqs(rots[i], 1e4, QLORA_ROPE_PLAIN, 1.0, 1, 1.0, 2.0, f, &amplitude));
  REJ(qlora_rope_freqs(2, 1e4, QLORA_ROPE_NTK, 2.0, 1, 1.0, 2.0, f, &amplitude));
  REJ(qlora_rope_freqs(128, 1e4, 9, 2.0, 1, 1.0, 2.0, f, &amplitude));
  REJ(qlora_rope_freqs(128, 1e4, QLORA_ROPE_PARTS, 2.0, INT64_MIN, 1.0, 2.0, f, &amplitude));
  REJ(qlora_rope_freqs(128, 1e4, QLORA_ROPE_PLAIN, 1.0, 1, 1.0, 2.0, NULL, &amplitude));
  REJ(qlora_rope_freqs(128, 1e4, QLORA_ROPE_PLAIN, 1.0, 1, 1.0, 2.0, f, NULL));
  for (int kind = QLORA_ROPE_PLAIN; kind <= QLORA_ROPE_PARTS; ++kind)
    if (qlora_rope_freqs(128, 1e4, kind, 8.0, INT64_MAX, 1.0, 32.0, f, &amplitude) != QLORA_OK || f[0] > 1.0 || !(f[63] > 0.0)) {
      printf("FAIL frequencies %d\n", kind);
      ++failures;
    }
  const qlora_rope_heads q = {pool, pool, 4, 512, 128, 512, 128};
#define ROPE(q, k, rows, dim, rot, amp) qlora_rope_fwd(q, k, QLORA_BF16, rows, dim, rot, pool, 1, f, amp, 0, NULL)
  REACH(ROPE(&q, NULL, 7, 128, 128, 1.0));
  REACH(ROPE(&q, &q, 7, 128, 2, -1.0));
  REACH(qlora_rope_bwd(&q, &q, QLORA_F32, 1, 64, 64, pool, 0, f, 1.0, 1, NULL));
  REJ(ROPE(NULL, &q, 7, 128, 128, 1.0));
  REJ(ROPE(&q, NULL, 7, 128, 128, NAN));
  const int64_t rows[] = {0, -1, INT64_MIN, INT64_MAX};
  for (size_t i = 0; i < sizeof rows / sizeof *rows; ++i) REJ(ROPE(&q, NULL, rows[i], 128, 128, 1.0));
  for (size_t i = 0; i < sizeof rots / sizeof *rots; ++i) REJ(ROPE(&q, NULL, 7, rots[i], 2, 1.0));
  for (size_t i = 0; i < sizeof rots / sizeof *rots; ++i) REJ(ROPE(&q, NULL, 7, 128, rots[i], 1.0));
  const int64_t strides[] = {-1, INT64_MIN, INT64_MAX, ((int64_t)1 << 46) + 1};
  for (size_t i = 0; i < sizeof strides / sizeof *strides; ++i) {
    WITH(qlora_rope_heads, h, q, h.in_row = strides[i], REJ(ROPE(&h, NULL, 7, 128, 128, 1.0)));
    WITH(qlora_rope_heads, h, q, h.in_head = strides[i], REJ(ROPE(&h, NULL, 7, 128, 128, 1.0)));
    WITH(qlora_rope_heads, h, q, h.out_row = strides[i], REJ(ROPE(&q, &h, 7, 128, 128, 1.0)));
    WITH(qlora_rope_heads, h, q, h.out_head = strides[i], REJ(ROPE(&q, &h, 7, 128, 128, 1.0)));
    WITH(qlora_rope_heads, h, q, h.heads = strides[i], REJ(ROPE(&q, &h, 7, 128, 128, 1.0)));
  }
  WITH(qlora_rope_heads, h, q, h.out_head = 0, REJ(ROPE(&h, NULL, 7, 128, 128, 1.0)));
  WITH(qlora_rope_heads, h, q, h.out_row = 500, REJ(ROPE(&h, NULL, 7, 128, 128, 1.0)));
}

int main(void) {
  pool = aligned_alloc(256, 1 << 20);
  memset(pool, 0, 1 << 20);
  microscaled();
  block(QLORA_FMT_NF4_DQ);
  block(QLORA_FMT_NF4);
  rope();
  free(pool);
  if (failures) return 1;
  printf("reject_block: ok\n");
  return 0;
}
