/*
 * A plain C consumer of rows held in e4m3: no torch, no C++.
 *
 *   held check   host-only: error paths of the reading back, sizes of a list
 *   held run     on the GPU: N tokens of zero keys and values equal to a power of
 *                two of their position are appended, read back (exactly) and
 *                attended.  Equal scores make the result at position p the mean
 *                of the first p + 1 values, and its log-sum log(p + 1).
 */
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <hip/hip_runtime_api.h>

#include "gpb.h"

#define CHECK(x) do { int rc_ = (x); if (rc_ != GPB_OK) { \
  fprintf(stderr, "%s:%d %s -> %d (%s)\n", __FILE__, __LINE__, #x, rc_, gpb_strerror(rc_)); \
  return 2; } } while (0)
#define HCHECK(x) do { hipError_t e_ = (x); if (e_ != hipSuccess) { \
  fprintf(stderr, "%s:%d %s -> %s\n", __FILE__, __LINE__, #x, hipGetErrorString(e_)); \
  return 3; } } while (0)

enum { N = 100, HEADS = 4, KV_HEADS = 2, DIM = 64, VALUES = 2 * KV_HEADS * DIM, PAGE = 32,
       PAGES = 6, ROW = VALUES + 16 };
static const gpb_row_format kFormat = {GPB_BF16 | GPB_HELD_E4M3, KV_HEADS, DIM, DIM, 0, ROW};

static uint16_t bf16(float x) { /* of values that bf16 holds */
  uint32_t b;
  memcpy(&b, &x, 4);
  return (uint16_t)(b >> 16);
}
static float widen(uint16_t x) {
  uint32_t b = (uint32_t)x << 16;
  float f;
  memcpy(&f, &b, 4);
  return f;
}
static float value(int t) { return ldexpf(1.0f, t % 5 - 2); }

static int make_plan(gpb_attend_plan *plan, int32_t **list) {
  const int32_t q = N, kv = N;
  gpb_attend_shape shape;
  memset(&shape, 0, sizeof shape);
  shape.bs = 1; shape.n_heads = HEADS; shape.page_rows = PAGE;
  shape.h_q_lens = &q; shape.h_kv_lens = &kv;
  CHECK(gpb_attend_plan_build(&kFormat, &shape, plan, NULL, 0));
  *list = malloc((size_t)plan->list_ints * 4);
  if (!*list) return 4;
  CHECK(gpb_attend_plan_build(&kFormat, &shape, plan, *list, plan->list_ints));
  return 0;
}

static int check(void) {
  gpb_attend_plan plan;
  int32_t *list = NULL;
  int rc = make_plan(&plan, &list);
  if (rc) return rc;
  int bad = plan.n_tokens != N || plan.format.dtype != (GPB_BF16 | GPB_HELD_E4M3);
  gpb_row_format plain = kFormat;
  plain.dtype = GPB_BF16; plain.row_bytes = 2 * VALUES;
  void *at = (void *)4096; /* never dereferenced */
  bad |= gpb_rows_read(&plain, at, N, NULL, N, at, 2 * VALUES, NULL, NULL) != GPB_EINVAL;
  bad |= gpb_rows_read(&kFormat, at, N, NULL, N + 1, at, 2 * VALUES, NULL, NULL) != GPB_EINVAL;
  bad |= gpb_rows_read(&kFormat, at, N, NULL, N, at, 2 * VALUES - 16, NULL, NULL) != GPB_EINVAL;
  bad |= gpb_rows_read(&kFormat, at, N, NULL, N, at, 2 * VALUES + 8, NULL, NULL) != GPB_EALIGN;
  bad |= gpb_rows_read(&kFormat, NULL, 0, NULL, 0, NULL, 2 * VALUES, NULL, NULL) != GPB_OK;
  free(list);
  return bad;
}

static int run(void) {
  static uint16_t v[N][KV_HEADS][DIM], out[N * HEADS * DIM], back[N][VALUES];
  static float lse[N * HEADS];
  const int32_t pages[4] = {4, 1, 5, 2};
  int32_t locs[N], status = -1;
  gpb_attend_plan plan;
  int32_t *list = NULL;
  int rc = make_plan(&plan, &list);
  if (rc) return rc;
  for (int t = 0; t < N; ++t) {
    locs[t] = pages[t / PAGE] * PAGE + t % PAGE;
    for (int h = 0; h < KV_HEADS; ++h)
      for (int e = 0; e < DIM; ++e) v[t][h][e] = bf16(value(t));
  }
  void *k, *d_v, *q, *pool, *d_out, *d_lse, *d_list, *d_locs, *d_pages, *d_back, *ws = NULL;
  int32_t *d_status;
  HCHECK(hipMalloc(&k, sizeof v));
  HCHECK(hipMalloc(&d_v, sizeof v));
  HCHECK(hipMalloc(&q, sizeof out));
  HCHECK(hipMalloc(&pool, (size_t)ROW * PAGES * PAGE));
  HCHECK(hipMalloc(&d_out, sizeof out));
  HCHECK(hipMalloc(&d_lse, sizeof lse));
  HCHECK(hipMalloc(&d_back, sizeof back));
  HCHECK(hipMalloc(&d_list, (size_t)plan.list_ints * 4));
  HCHECK(hipMalloc(&d_locs, sizeof locs));
  HCHECK(hipMalloc(&d_pages, sizeof pages));
  HCHECK(hipMalloc((void **)&d_status, 4));
  if (plan.workspace_bytes) HCHECK(hipMalloc(&ws, (size_t)plan.workspace_bytes));
  HCHECK(hipMemset(k, 0, sizeof v));
  HCHECK(hipMemset(q, 0x3f, sizeof out));
  HCHECK(hipMemset(pool, 0xff, (size_t)ROW * PAGES * PAGE));
  HCHECK(hipMemset(d_status, 0, 4));
  HCHECK(hipMemcpy(d_v, v, sizeof v, hipMemcpyHostToDevice));
  HCHECK(hipMemcpy(d_list, list, (size_t)plan.list_ints * 4, hipMemcpyHostToDevice));
  HCHECK(hipMemcpy(d_locs, locs, sizeof locs, hipMemcpyHostToDevice));
  HCHECK(hipMemcpy(d_pages, pages, sizeof pages, hipMemcpyHostToDevice));

  gpb_append a;
  memset(&a, 0, sizeof a);
  a.n_rows = N;
  a.d_k = k; a.d_v = d_v;
  a.k_token_stride = a.v_token_stride = KV_HEADS * DIM;
  a.k_head_stride = a.v_head_stride = DIM;
  a.d_pool = pool; a.n_pool_rows = PAGES * PAGE; a.d_pool_locs = d_locs;
  CHECK(gpb_row_append(&kFormat, &a, d_status, NULL));
  CHECK(gpb_rows_read(&kFormat, pool, PAGES * PAGE, d_locs, N, d_back, 2 * VALUES, d_status,
                      NULL));
  HCHECK(hipMemcpy(back, d_back, sizeof back, hipMemcpyDeviceToHost));
  for (int t = 0; t < N; ++t)
    for (int e = 0; e < VALUES; ++e) {
      const float want = e < VALUES / 2 ? 0.0f : value(t);
      if (widen(back[t][e]) != want) {
        fprintf(stderr, "back %d %d: %g, not %g\n", t, e, widen(back[t][e]), want);
        return 1;
      }
    }

  gpb_attend_io io;
  memset(&io, 0, sizeof io);
  io.d_q = q; io.d_out = d_out; io.d_lse = d_lse; io.scale = 0.125f;
  io.q_token_stride = io.out_token_stride = HEADS * DIM;
  io.q_head_stride = io.out_head_stride = DIM;
  CHECK(gpb_attend_paged(&plan, d_list, &io, pool, PAGES * PAGE, d_pages, 4, NULL, 4, ws,
                         plan.workspace_bytes, d_status, NULL));
  HCHECK(hipMemcpy(out, d_out, sizeof out, hipMemcpyDeviceToHost));
  HCHECK(hipMemcpy(lse, d_lse, sizeof lse, hipMemcpyDeviceToHost));
  double sum = 0.0;
  for (int t = 0; t < N; ++t) {
    sum += value(t); /* weights of 1 and their sums are exact; the mean is rounded twice */
    const float want = (float)(sum / (t + 1)), z = logf((float)(t + 1));
    for (int h = 0; h < HEADS; ++h) {
      if (fabsf(lse[t * HEADS + h] - z) > 1e-5f * (1.0f + z)) {
        fprintf(stderr, "lse %d %d: %g, not %g\n", t, h, lse[t * HEADS + h], z);
        return 1;
      }
      for (int e = 0; e < DIM; ++e) {
        const float got = widen(out[(t * HEADS + h) * DIM + e]);
        if (fabsf(got - want) > want * (1.0f / 256.0f + 1e-5f)) {
          fprintf(stderr, "out %d %d %d: %g, not %g\n", t, h, e, got, want);
          return 1;
        }
      }
    }
  }
  HCHECK(hipMemcpy(&status, d_status, 4, hipMemcpyDeviceToHost));
  free(list);
  return status;
}

int main(int argc, char **argv) {
  if (argc == 2 && !strcmp(argv[1], "check")) return check();
  if (argc == 2 && !strcmp(argv[1], "run")) return run();
  fprintf(stderr, "usage: held check|run\n");
  return 9;
}
