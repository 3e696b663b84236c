/* Drives the attention half's C ABI without a GPU: struct sizes for the binding, workspace
 * queries at the extremes of every argument (integer overflow in the size arithmetic would
 * be undefined behaviour), and calls that the library must reject, or accept with nothing to
 * enqueue. Each rejected call breaks one rule of an otherwise good call. Device pointers are
 * fake addresses that are never dereferenced. */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "qmoe.h"

#define FAKE(off) ((void*)(uintptr_t)(0x7f0000000000ull + (off)))
#define BAD MOE_ERR_INVALID_ARGUMENT
#define UNS MOE_ERR_UNSUPPORTED

static int failures = 0;

static void expect(const char* what, moe_status got, moe_status want) {
  if (got != want) {
    printf("MISMATCH %s: %s, expected %s\n", what, moe_status_string(got),
           moe_status_string(want));
    ++failures;
  }
}

static moe_heads heads(uint64_t off, int n, int D) {
  moe_heads h = {FAKE(off), (int64_t)n * D, D, n};
  return h;
}

static moe_kv_cache cache(void) {
  moe_kv_cache c = {FAKE(0x10000000), FAKE(0x20000000), NULL, NULL, MOE_BF16, 64, 16, 2, 64};
  return c;
}

/* one call of each entry point on good arguments, with one of them replaced */
struct call {
  moe_kv_cache c;
  moe_heads q, k, v, qo, ko;
  moe_norm_rope p;
  moe_pages pages;
  moe_attn a;
  const int32_t *positions, *slots, *starts;
  int n, dtype, D, window;
  void *out, *ws;
  size_t ws_bytes;
};

static struct call good(void) {
  struct call x;
  memset(&x, 0, sizeof x);
  x.c = cache();
  x.q = heads(0x1000000, 4, 64);
  x.k = heads(0x2000000, 2, 64);
  x.v = heads(0x3000000, 2, 64);
  x.qo = heads(0x4000000, 4, 64);
  x.ko = heads(0x5000000, 2, 64);
  x.p.q_norm = FAKE(0x6000000);
  x.p.k_norm = FAKE(0x6001000);
  x.p.inv_freq = FAKE(0x6002000);
  x.p.eps = 1e-6f;
  x.p.rot_dim = 64;
  x.pages.table = FAKE(0x7000000);
  x.pages.kv_lens = FAKE(0x7100000);
  x.pages.table_stride = 64;
  x.pages.n_seqs = 2;
  x.pages.max_pages = 64;
  x.a.scale = 0.125f;
  x.positions = FAKE(0x7200000);
  x.slots = FAKE(0x7300000);
  x.starts = FAKE(0x7400000);
  x.n = 8;
  x.dtype = MOE_BF16;
  x.D = 64;
  x.window = 4;
  x.out = FAKE(0x8000000);
  x.ws = FAKE(0x40000000);
  x.ws_bytes = (size_t)1 << 40;
  return x;
}

static moe_status rope(const struct call* x) {
  return moe_qk_norm_rope(&x->q, &x->k, x->positions, x->n, x->dtype, x->D, &x->p, &x->qo, &x->ko,
                          NULL);
}
static moe_status append(const struct call* x) {
  return moe_kv_append(&x->c, &x->k, &x->v, x->slots, x->positions, x->n, x->dtype, &x->p, &x->q,
                       &x->qo, NULL);
}
static moe_status decode(const struct call* x) {
  return moe_attn_decode(&x->c, &x->q, x->dtype, &x->pages, x->window, &x->a, x->out, x->ws,
                         x->ws_bytes, NULL);
}
static moe_status prefill(const struct call* x) {
  return moe_attn_prefill(&x->c, &x->q, x->dtype, x->starts, x->n, &x->pages, &x->a, x->out, x->ws,
                          x->ws_bytes, NULL);
}

#define TRY(fn, change, want)          \
  do {                                 \
    struct call x = good();            \
    change;                            \
    expect(#fn ": " #change, fn(&x), want); \
  } while (0)

#define ATTENTION(change, want) \
  TRY(decode, change, want);    \
  TRY(prefill, change, want)

int main(void) {
  static const int sizes[] = {INT_MIN, -1, 0, 1, 15, 16, 17, 64, 128, 256, 512, 513, 8192, 8193,
                              65536, INT_MAX};
  const int ns = (int)(sizeof sizes / sizeof sizes[0]);
  const float nan = (float)(INT_MAX * 1e300 * 1e300 * 0.0);
  size_t acc = 0;

  printf("sizeof moe_heads %zu\n", sizeof(moe_heads));
  printf("sizeof moe_kv_cache %zu\n", sizeof(moe_kv_cache));
  printf("sizeof moe_norm_rope %zu\n", sizeof(moe_norm_rope));
  printf("sizeof moe_pages %zu\n", sizeof(moe_pages));
  printf("sizeof moe_attn %zu\n", sizeof(moe_attn));

  for (int a = 0; a < ns; ++a)
    for (int b = 0; b < ns; ++b)
      for (int d = 0; d < ns; ++d) {
        moe_kv_cache c = cache();
        moe_attn w = {1.0f, 0, 0};
        c.num_pages = sizes[a];
        acc += moe_attn_decode_workspace_bytes(&c, sizes[b], sizes[d], 4, sizes[a], &w);
        c = cache();
        acc += moe_attn_decode_workspace_bytes(&c, 4, sizes[a], sizes[b], sizes[d], &w);
        acc += moe_attn_prefill_workspace_bytes(&c, 4, sizes[a], sizes[b], sizes[d], &w);
        w.window = sizes[a];
        w.sinks = sizes[b];
        acc += moe_attn_decode_workspace_bytes(&c, 4, 1, 1, sizes[d], &w);
        acc += moe_attn_prefill_workspace_bytes(&c, 4, 1, 9, sizes[d], &w);
        c.page_size = sizes[a];
        c.kv_heads = sizes[b];
        c.head_dim = sizes[d];
        acc += moe_attn_decode_workspace_bytes(&c, 512, 1, 1, 1 << 20, &w);
        acc += moe_attn_prefill_workspace_bytes(&c, 512, 1, 1, 1 << 20, &w);
      }
  acc += moe_attn_decode_workspace_bytes(NULL, 4, 1, 1, 4, NULL);

  /* norm and rotation */
  TRY(rope, x.n = 0, MOE_OK);
  TRY(rope, x.n = -1, BAD);
  TRY(rope, x.n = 8193, BAD);
  TRY(rope, x.dtype = MOE_E4M3, UNS);
  TRY(rope, x.D = 96, UNS);
  TRY(rope, x.p.rot_dim = 24, UNS);
  TRY(rope, x.p.rot_dim = 80, BAD);
  TRY(rope, x.p.rot_dim = -16, BAD);
  TRY(rope, x.p.inv_freq = NULL, BAD);
  TRY(rope, x.positions = NULL, BAD);
  TRY(rope, x.positions = FAKE(0x7200002), BAD);
  TRY(rope, x.p.eps = -1e-6f, BAD);
  TRY(rope, x.p.eps = nan, BAD);
  TRY(rope, x.p.weight_offset = nan, BAD);
  TRY(rope, x.q.data = FAKE(0x1000008), BAD);
  TRY(rope, x.q.token_stride = 260, BAD);
  TRY(rope, x.q.head_stride = -64, BAD);
  TRY(rope, x.q.token_stride = (int64_t)1 << 31, BAD);
  TRY(rope, x.q.heads = 513, BAD);
  TRY(rope, x.q.heads = 0, BAD);
  TRY(rope, x.qo.data = NULL, BAD);
  TRY(rope, x.qo.heads = 3, BAD);
  TRY(rope, x.qo.token_stride = 0, BAD);     /* every token on the same output */
  TRY(rope, x.qo.head_stride = 32, BAD);     /* heads overlap */
  TRY(rope, x.qo.data = FAKE(0x1000040), BAD); /* partly on its input */
  TRY(rope, x.ko.data = FAKE(0x1000000), BAD); /* on the other input */
  TRY(rope, x.ko.data = x.qo.data, BAD);

  /* append */
  TRY(append, x.n = 0, MOE_OK);
  TRY(append, x.n = 8193, BAD);
  TRY(append, x.dtype = MOE_F16, UNS); /* not the cache's */
  TRY(append, x.c.dtype = 3, UNS);
  TRY(append, x.c.page_size = 8, UNS);
  TRY(append, x.c.page_size = 48, UNS);
  TRY(append, x.c.head_dim = 80, UNS);
  TRY(append, x.c.kv_heads = 4, BAD);
  TRY(append, x.c.num_pages = 0, BAD);
  TRY(append, x.c.num_pages = 1 << 28, BAD); /* slots beyond 31 bits */
  TRY(append, x.c.k = NULL, BAD);
  TRY(append, x.c.v = FAKE(0x20000008), BAD);
  TRY(append, x.c.k_scale = FAKE(0x9000000), BAD); /* a 16-bit cache has none */
  TRY(append, x.slots = NULL, BAD);
  TRY(append, x.k.data = NULL, BAD);
  TRY(append, x.v.heads = 1, BAD);
  TRY(append, x.k.data = FAKE(0x10000100), BAD); /* inside the cache */
  TRY(append, x.c.v = FAKE(0x10000100), BAD);    /* keys and values overlap */
  TRY(append, x.qo.data = x.k.data, BAD);
  TRY(append, x.qo.data = FAKE(0x20000000), BAD);
  {
    struct call x = good();
    expect("append: q without p",
           moe_kv_append(&x.c, &x.k, &x.v, x.slots, x.positions, x.n, x.dtype, NULL, &x.q, &x.qo,
                         NULL),
           BAD);
    expect("append: no cache",
           moe_kv_append(NULL, &x.k, &x.v, x.slots, x.positions, x.n, x.dtype, &x.p, NULL, NULL,
                         NULL),
           BAD);
  }

  /* attention */
  TRY(decode, x.pages.n_seqs = 0, MOE_OK);
  TRY(prefill, x.n = 0, MOE_OK);
  TRY(prefill, x.pages.n_seqs = 0, MOE_OK);
  TRY(decode, x.window = 0, BAD);
  TRY(decode, x.window = 17, BAD);
  TRY(decode, x.pages.n_seqs = 129, BAD); /* 516 tokens */
  TRY(prefill, x.n = 8193, BAD);
  TRY(prefill, x.starts = NULL, BAD);
  TRY(prefill, x.starts = FAKE(0x7400001), BAD);
  ATTENTION(x.pages.n_seqs = -1, BAD);
  ATTENTION(x.q.heads = 5, BAD);
  ATTENTION(x.q.data = NULL, BAD);
  ATTENTION(x.dtype = MOE_E4M3, UNS);
  ATTENTION(x.dtype = MOE_F16, UNS);
  ATTENTION(x.pages.table = NULL, BAD);
  ATTENTION(x.pages.kv_lens = NULL, BAD);
  ATTENTION(x.pages.max_pages = 0, BAD);
  ATTENTION(x.pages.max_pages = 65, BAD); /* beyond the row stride */
  ATTENTION(x.a.scale = nan, BAD);
  ATTENTION(x.a.window = -1, BAD);
  ATTENTION(x.a.sinks = -1, BAD);
  ATTENTION(x.out = NULL, BAD);
  ATTENTION(x.out = FAKE(0x8000008), BAD);
  ATTENTION(x.out = x.q.data, BAD);
  ATTENTION(x.out = FAKE(0x10000000), BAD); /* on the cache */
  ATTENTION(x.c.k = FAKE(0x10000004), BAD);
  {
    struct call x = good();
    x.pages.max_pages = 4096;
    x.pages.table_stride = 4096;
    const size_t d = moe_attn_decode_workspace_bytes(&x.c, 4, 2, 4, 4096, &x.a);
    const size_t p = moe_attn_prefill_workspace_bytes(&x.c, 4, 2, 8, 4096, &x.a);
    if (d == 0 || p == 0 || d % 256 || p % 256) ++failures, printf("MISMATCH workspace sizes\n");
    x.ws_bytes = d - 1;
    expect("decode: small workspace", decode(&x), MOE_ERR_WORKSPACE_TOO_SMALL);
    x.ws_bytes = p - 1;
    expect("prefill: small workspace", prefill(&x), MOE_ERR_WORKSPACE_TOO_SMALL);
    x.ws_bytes = d + p;
    x.ws = FAKE(0x40000010);
    expect("decode: misaligned workspace", decode(&x), BAD);
    expect("prefill: misaligned workspace", prefill(&x), BAD);
    x.ws = x.out;
    expect("decode: workspace on the output", decode(&x), BAD);
    expect("prefill: workspace on the output", prefill(&x), BAD);
    x.ws = x.c.k;
    expect("decode: workspace on the cache", decode(&x), BAD);
    expect("prefill: workspace on the cache", prefill(&x), BAD);
  }
  printf("attention driver: %d mismatches (%zu)\n", failures, acc);
  return failures != 0;
}
