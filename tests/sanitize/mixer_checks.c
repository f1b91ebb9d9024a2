/*
 * Host-side check of the C ABI (test infrastructure) of linear attention, window attention and the norms of queries and
 * keys, like abi_checks.c: linked against their host code built under AddressSanitizer and UndefinedBehaviorSanitizer, it
 * drives every entry point through argument validation and every workspace query through sizes up to the int64 limits.
 * No call here passes validation with device pointers: the fake addresses are never dereferenced, and nothing is
 * launched.
 */
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "mamba_scan.h"

#define FAKE ((void*)0x10000)
#define ODD ((void*)0x10001)

static int failures = 0;
static const int64_t extremes[] = {INT64_MAX, INT64_MAX - 15, (int64_t)1 << 62, ((int64_t)1 << 41) + 16, INT64_MIN, -1};
#define NEX ((int)(sizeof extremes / sizeof extremes[0]))

static void expect(int64_t got, int64_t want, const char* what, int line) {
  if (got != want) {
    fprintf(stderr, "line %d: %s returned %lld, expected %lld\n", line, what, (long long)got, (long long)want);
    ++failures;
  }
}
#define EXPECT(call, want) expect((int64_t)(call), (want), #call, __LINE__)
#define REFUSED(call) expect((call) != MAMBA_OK, 1, #call, __LINE__)

static int lin_fwd(const mamba_delta_dims* d, void* q, void* ws, size_t n, const int64_t* off) {
  return mamba_linear_attn_fwd(q, FAKE, FAKE, FAKE, NULL, off, 1.f, FAKE, NULL, d, ws, n, NULL);
}
static int lin_step(const mamba_delta_dims* d, float* state) {
  return mamba_linear_attn_update(state, FAKE, FAKE, FAKE, FAKE, 1.f, FAKE, d, NULL);
}
static int lin_bwd(const mamba_delta_dims* d, void* dq, void* ws, size_t n, const int64_t* off) {
  return mamba_linear_attn_bwd(FAKE, FAKE, FAKE, FAKE, NULL, off, 1.f, FAKE, NULL, dq, FAKE, FAKE, FAKE, NULL, d, ws, n,
                               NULL);
}
static int win_fwd(const mamba_window_dims* d, void* q, const int64_t* off) {
  return mamba_window_attn_fwd(q, FAKE, FAKE, off, off, 1.f, FAKE, NULL, d, NULL);
}
static int win_bwd(const mamba_window_dims* d, void* dq, void* ws, size_t n, const int64_t* off) {
  return mamba_window_attn_bwd(FAKE, FAKE, FAKE, off, off, 1.f, FAKE, FAKE, FAKE, dq, FAKE, FAKE, d, ws, n, NULL);
}
static int win_store(const mamba_window_dims* d, void* kc) {
  return mamba_window_cache_store(FAKE, FAKE, NULL, kc, FAKE, d, NULL);
}
static int win_step(const mamba_window_dims* d, void* kc, void* ws, size_t n) {
  return mamba_window_attn_update(kc, FAKE, FAKE, FAKE, FAKE, FAKE, 1.f, FAKE, d, ws, n, NULL);
}
static int qk_fwd(const mamba_qk_norm_rope_dims* d, void* q) {
  return mamba_qk_norm_rope_fwd(q, FAKE, FAKE, FAKE, FAKE, FAKE, 1e-5f, FAKE, FAKE, d, NULL);
}
static int qk_bwd(const mamba_qk_norm_rope_dims* d, void* dq, void* ws, size_t n) {
  return mamba_qk_norm_rope_bwd(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1e-5f, FAKE, FAKE, dq, FAKE, FAKE, FAKE, d, ws, n,
                                NULL);
}

static void linear(int io) {
  mamba_delta_dims d;
  memset(&d, 0, sizeof d);
  d.batch = 2; d.seqlen = 100; d.qk_heads = 2; d.v_heads = 4; d.dk = 64; d.dv = 64; d.io_dtype = io;
  const int64_t* off = FAKE;
  const mamba_delta_dims ok = d;
  EXPECT(lin_fwd(NULL, FAKE, FAKE, SIZE_MAX, NULL), MAMBA_ERR_NULL);
  EXPECT(lin_fwd(&ok, NULL, FAKE, SIZE_MAX, NULL), MAMBA_ERR_NULL);
  EXPECT(lin_fwd(&ok, ODD, FAKE, SIZE_MAX, NULL), MAMBA_ERR_ALIGN);
  EXPECT(lin_bwd(&ok, NULL, FAKE, SIZE_MAX, NULL), MAMBA_ERR_NULL);
  EXPECT(lin_bwd(&ok, ODD, FAKE, SIZE_MAX, NULL), MAMBA_ERR_ALIGN);
  EXPECT(lin_bwd(&ok, FAKE, NULL, SIZE_MAX, NULL), MAMBA_ERR_WORKSPACE);
  EXPECT(lin_bwd(&ok, FAKE, FAKE, mamba_linear_attn_bwd_workspace_bytes(&ok, 1) - 1, off), MAMBA_ERR_WORKSPACE);
  EXPECT(lin_bwd(&ok, FAKE, (char*)FAKE + 16, SIZE_MAX, NULL), MAMBA_ERR_ALIGN);
  EXPECT(lin_step(&ok, FAKE), MAMBA_ERR_SHAPE); /* more than one token */
  d.seqlen = 1;
  EXPECT(lin_step(&d, NULL), MAMBA_ERR_NULL);
  EXPECT(lin_step(&d, (float*)((char*)FAKE + 4)), MAMBA_ERR_ALIGN);
  int64_t* const fields[] = {&d.batch, &d.seqlen, &d.qk_heads, &d.v_heads, &d.dk, &d.dv, &d.q_stride, &d.k_stride,
                             &d.v_stride};
  for (int f = 0; f < 9; ++f)
    for (int e = 0; e < NEX; ++e)
      for (int packed = 0; packed < 2; ++packed) {
        d = ok;
        *fields[f] = extremes[e];
        EXPECT(mamba_linear_attn_workspace_bytes(&d, packed), 0);
        EXPECT(mamba_linear_attn_bwd_workspace_bytes(&d, packed), 0);
        REFUSED(lin_fwd(&d, FAKE, FAKE, SIZE_MAX, packed ? off : NULL));
        REFUSED(lin_bwd(&d, FAKE, FAKE, SIZE_MAX, packed ? off : NULL));
        REFUSED(lin_step(&d, FAKE));
      }
  /* the largest that the limits admit, and odd sizes on the way: queries only */
  for (int64_t tokens = 1; tokens <= (int64_t)1 << 40; tokens = tokens * 3 + 1)
    for (int64_t heads = 1; heads <= 65535; heads = heads * 7 + 1)
      for (int64_t batch = 1; batch <= (int64_t)1 << 30; batch = batch * 37 + 1)
        for (int packed = 0; packed < 2; ++packed) {
          d = ok;
          d.batch = batch; d.seqlen = tokens; d.qk_heads = 1; d.v_heads = heads; d.dk = 8; d.dv = 8;
          const size_t a = mamba_linear_attn_workspace_bytes(&d, packed), b = mamba_linear_attn_bwd_workspace_bytes(&d, packed);
          if (b && b < a) expect(0, 1, "the gradients hold what the forward holds", __LINE__);
        }
}

static void window(int io) {
  mamba_window_dims d;
  memset(&d, 0, sizeof d);
  d.batch = 2; d.seqlen = 100; d.kv_len = 100; d.q_heads = 4; d.kv_heads = 2; d.dim = 64; d.window = 10; d.sinks = 2;
  d.io_dtype = io;
  const int64_t* off = FAKE;
  const mamba_window_dims ok = d;
  EXPECT(win_fwd(NULL, FAKE, NULL), MAMBA_ERR_NULL);
  EXPECT(win_fwd(&ok, NULL, NULL), MAMBA_ERR_NULL);
  EXPECT(win_fwd(&ok, ODD, NULL), MAMBA_ERR_ALIGN);
  EXPECT(win_bwd(&ok, NULL, FAKE, SIZE_MAX, NULL), MAMBA_ERR_NULL);
  EXPECT(win_bwd(&ok, ODD, FAKE, SIZE_MAX, off), MAMBA_ERR_ALIGN);
  EXPECT(win_bwd(&ok, FAKE, NULL, SIZE_MAX, NULL), MAMBA_ERR_WORKSPACE);
  EXPECT(win_bwd(&ok, FAKE, FAKE, mamba_window_attn_bwd_workspace_bytes(&ok, 0) - 1, NULL), MAMBA_ERR_WORKSPACE);
  EXPECT(win_bwd(&ok, FAKE, ODD, SIZE_MAX, NULL), MAMBA_ERR_ALIGN);
  EXPECT(win_store(&ok, NULL), MAMBA_ERR_NULL);
  EXPECT(win_store(&ok, ODD), MAMBA_ERR_ALIGN);
  EXPECT(win_step(&ok, FAKE, FAKE, SIZE_MAX), MAMBA_ERR_SHAPE);
  d.seqlen = d.kv_len = 1;
  d.window = 5000;
  EXPECT(win_step(&d, NULL, FAKE, SIZE_MAX), MAMBA_ERR_NULL);
  EXPECT(win_step(&d, ODD, FAKE, SIZE_MAX), MAMBA_ERR_ALIGN);
  EXPECT(win_step(&d, FAKE, NULL, 0), MAMBA_ERR_WORKSPACE);
  EXPECT(win_step(&d, FAKE, FAKE, mamba_window_attn_update_workspace_bytes(&d) - 1), MAMBA_ERR_WORKSPACE);
  int64_t* const fields[] = {&d.batch, &d.seqlen, &d.kv_len, &d.q_heads, &d.kv_heads, &d.dim, &d.q_stride, &d.k_stride,
                             &d.v_stride, &d.window, &d.sinks};
  for (int f = 0; f < 11; ++f)
    for (int e = 0; e < NEX; ++e)
      for (int packed = 0; packed < 2; ++packed) {
        d = ok;
        *fields[f] = extremes[e];
        EXPECT(mamba_window_attn_bwd_workspace_bytes(&d, packed), 0);
        EXPECT(mamba_window_attn_update_workspace_bytes(&d), 0);
        REFUSED(win_fwd(&d, FAKE, packed ? off : NULL));
        REFUSED(win_bwd(&d, FAKE, FAKE, SIZE_MAX, packed ? off : NULL));
        REFUSED(win_step(&d, FAKE, FAKE, SIZE_MAX));
        if (f != 1 && f != 3 && f != 6) REFUSED(win_store(&d, FAKE)); /* (it has no queries) */
      }
  for (int64_t tokens = 1; tokens < ((int64_t)1 << 31) - 1024; tokens = tokens * 5 + 1)
    for (int64_t heads = 1; heads <= 65535; heads = heads * 9 + 1)
      for (int64_t sinks = 0; sinks <= (int64_t)1 << 40; sinks = sinks * 33 + 1)
        for (int64_t batch = 1; batch <= (int64_t)1 << 20; batch = batch * 37 + 1)
          for (int packed = 0; packed < 2; ++packed) {
            d = ok;
            d.batch = batch; d.seqlen = d.kv_len = tokens; d.q_heads = heads; d.kv_heads = 1; d.dim = 8; d.sinks = sinks;
            d.window = 1 + sinks / 2;
            const size_t b = mamba_window_attn_bwd_workspace_bytes(&d, packed);
            /* two numbers per query and head at least */
            if (b && (double)b < 8.0 * (double)(packed ? 1 : batch) * (double)tokens * (double)heads)
              expect(0, 1, "a workspace of window attention's gradients", __LINE__);
            d.seqlen = d.kv_len = 1;
            mamba_window_attn_update_workspace_bytes(&d);
          }
  /* sinks by the million: no size that a workspace could have */
  d = ok;
  d.batch = 1; d.seqlen = d.kv_len = (int64_t)1 << 30; d.q_heads = 8; d.kv_heads = 1; d.dim = 128; d.window = 1;
  d.sinks = (int64_t)1 << 30;
  expect(mamba_window_attn_bwd_workspace_bytes(&d, 0) > (size_t)1 << 60, 1, "a workspace past every memory", __LINE__);
}

static void qk(int io) {
  mamba_qk_norm_rope_dims d;
  memset(&d, 0, sizeof d);
  d.rows = 10; d.q_heads = 4; d.k_heads = 2; d.dim = 64; d.rotary_dim = 32; d.io_dtype = io;
  const mamba_qk_norm_rope_dims ok = d;
  EXPECT(qk_fwd(NULL, FAKE), MAMBA_ERR_NULL);
  EXPECT(qk_fwd(&ok, NULL), MAMBA_ERR_NULL);
  EXPECT(qk_fwd(&ok, ODD), MAMBA_ERR_ALIGN);
  EXPECT(qk_bwd(&ok, NULL, FAKE, SIZE_MAX), MAMBA_ERR_NULL);
  EXPECT(qk_bwd(&ok, ODD, FAKE, SIZE_MAX), MAMBA_ERR_ALIGN);
  EXPECT(qk_bwd(&ok, FAKE, FAKE, mamba_qk_norm_rope_bwd_workspace_bytes(&ok) - 1), MAMBA_ERR_WORKSPACE);
  EXPECT(qk_bwd(&ok, FAKE, ODD, SIZE_MAX), MAMBA_ERR_ALIGN);
  int64_t* const fields[] = {&d.rows, &d.q_heads, &d.k_heads, &d.dim, &d.rotary_dim, &d.q_stride, &d.k_stride};
  for (int f = 0; f < 7; ++f)
    for (int e = 0; e < NEX; ++e) {
      d = ok;
      *fields[f] = extremes[e];
      EXPECT(mamba_qk_norm_rope_bwd_workspace_bytes(&d), 0);
      REFUSED(qk_fwd(&d, FAKE));
      REFUSED(qk_bwd(&d, FAKE, FAKE, SIZE_MAX));
    }
}

int main(void) {
  for (int io = MAMBA_F32; io <= MAMBA_BF16; ++io) {
    linear(io);
    window(io);
    qk(io);
  }
  printf(failures ? "%d failures\n" : "clean\n", failures);
  return failures != 0;
}
