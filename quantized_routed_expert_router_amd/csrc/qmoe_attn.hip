// C ABI of the attention half: argument validation and workspace queries. Every check runs
// on the host before anything is enqueued.
#include "qmoe_attn_plan.h"

namespace qmoe {
namespace {

constexpr int kMaxLayoutInt = 0x7fffffff;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

Range range(const void* p, size_t bytes) { return {(uintptr_t)p, (uintptr_t)p + bytes}; }

bool disjoint(const Range& a, const Range& b) { return a.hi <= b.lo || b.hi <= a.lo; }

bool has(const moe_heads* h) { return h && h->data; }

// Bytes from the first to behind the last element of n tokens' heads (16-bit elements).
size_t span_bytes(const moe_heads& h, int n, int D) {
  return 2 * ((size_t)(n - 1) * (size_t)h.token_stride +
              (size_t)(h.heads - 1) * (size_t)h.head_stride + (size_t)D);
}

Range range(const moe_heads& h, int n, int D) { return range(h.data, span_bytes(h, n, D)); }

// Strides are below 2^31 elements: the kernels multiply them as 32-bit numbers.
moe_status check_heads(const moe_heads& h) {
  if (h.heads < 1 || h.heads > MOE_MAX_HEADS) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(h.data, 16)) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t most = kMaxLayoutInt;
  if (h.token_stride < 0 || h.head_stride < 0 || h.token_stride > most || h.head_stride > most)
    return MOE_ERR_INVALID_ARGUMENT;
  if (h.token_stride % 8 || h.head_stride % 8) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// Whether no two rows of the set share an element: tokens outside heads, or the reverse.
bool rows_distinct(const moe_heads& h, int n, int D) {
  const int64_t ts = h.token_stride, hs = h.head_stride;
  if (n > 1 && ts < D) return false;
  if (h.heads > 1 && hs < D) return false;
  if (n == 1 || h.heads == 1) return true;
  return ts >= (int64_t)(h.heads - 1) * hs + D || hs >= (int64_t)(n - 1) * ts + D;
}

bool same_view(const moe_heads& a, const moe_heads& b, int n) {
  return a.data == b.data && a.heads == b.heads && (n == 1 || a.token_stride == b.token_stride) &&
         (a.heads == 1 || a.head_stride == b.head_stride);
}

// Whether two row sets certainly share no element: their ranges are apart, or both step
// through tokens with one stride and their parts of a token are apart (two parts of one
// fused projection output).
bool views_apart(const moe_heads& a, const moe_heads& b, int n, int D) {
  if (disjoint(range(a, n, D), range(b, n, D))) return true;
  if (a.token_stride != b.token_stride || a.token_stride == 0) return false;
  const int64_t ts = 2 * a.token_stride;
  const int64_t la = 2 * ((int64_t)(a.heads - 1) * a.head_stride + D);
  const int64_t lb = 2 * ((int64_t)(b.heads - 1) * b.head_stride + D);
  const int64_t diff = (int64_t)((intptr_t)b.data - (intptr_t)a.data);
  const int64_t at = ((diff % ts) + ts) % ts;  // start of b behind a start of a
  return at >= la && at + lb <= ts;
}

bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

moe_status check_cache(const moe_kv_cache* c) {
  if (!c) return MOE_ERR_INVALID_ARGUMENT;
  if (c->dtype < MOE_BF16 || c->dtype > MOE_E4M3) return MOE_ERR_UNSUPPORTED;
  if (!head_dim_ok(c->head_dim)) return MOE_ERR_UNSUPPORTED;
  const int ps = c->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) return MOE_ERR_UNSUPPORTED;
  if (c->kv_heads < 1 || c->kv_heads > MOE_MAX_HEADS) return MOE_ERR_INVALID_ARGUMENT;
  if (c->num_pages < 1 || (long long)c->num_pages * ps > kMaxLayoutInt ||
      (long long)c->num_pages * c->kv_heads > kMaxLayoutInt)
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status check_cache_data(const moe_kv_cache* c) {
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return MOE_ERR_INVALID_ARGUMENT;
  if (c->dtype != MOE_E4M3 && (c->k_scale || c->v_scale)) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

size_t cache_bytes(const moe_kv_cache* c) {
  return (size_t)c->num_pages * c->page_size * c->kv_heads * c->head_dim *
         (c->dtype == MOE_E4M3 ? 1 : 2);
}

Range k_range(const moe_kv_cache* c) { return range(c->k, cache_bytes(c)); }
Range v_range(const moe_kv_cache* c) { return range(c->v, cache_bytes(c)); }

bool dtype_ok(int dtype) { return dtype == MOE_BF16 || dtype == MOE_F16; }

moe_status check_norm_rope(const moe_norm_rope* p, int D, const int32_t* positions) {
  if (p->rot_dim < 0 || p->rot_dim > D) return MOE_ERR_INVALID_ARGUMENT;
  if (p->rot_dim % 16) return MOE_ERR_UNSUPPORTED;
  if (p->rot_dim > 0 && (!p->inv_freq || !positions)) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(p->q_norm, 4) || !aligned(p->k_norm, 4) || !aligned(p->inv_freq, 4) ||
      !aligned(positions, 4))
    return MOE_ERR_INVALID_ARGUMENT;
  // finite, and eps not negative (both comparisons are false for NaN)
  if (!(p->eps >= 0.0f && p->eps <= 1.0f)) return MOE_ERR_INVALID_ARGUMENT;
  if (!(p->weight_offset >= -16.0f && p->weight_offset <= 16.0f)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// Whether a written range holds nothing that norm and rotation read beside the rows.
bool apart_from_parameters(const Range& written, const moe_norm_rope& p, int D,
                           const int32_t* positions, int n) {
  const size_t row = 4 * (size_t)D;
  return disjoint(written, range(positions, positions ? 4 * (size_t)n : 0)) &&
         disjoint(written, range(p.q_norm, p.q_norm ? row : 0)) &&
         disjoint(written, range(p.k_norm, p.k_norm ? row : 0)) &&
         disjoint(written, range(p.inv_freq, 2 * (size_t)p.rot_dim));
}

HeadView view(const moe_heads* h) {
  if (!has(h)) return HeadView{nullptr, 0, 0, 0};
  return HeadView{(char*)h->data, h->token_stride, h->head_stride, h->heads};
}

// One input set and its output set: same heads, output rows distinct, output either the
// input itself or apart from it.
moe_status check_pair(const moe_heads* in, const moe_heads* out, int n, int D) {
  if (!has(out)) return MOE_ERR_INVALID_ARGUMENT;
  moe_status s = check_heads(*in);
  if (s == MOE_OK) s = check_heads(*out);
  if (s != MOE_OK) return s;
  if (in->heads != out->heads || !rows_distinct(*out, n, D)) return MOE_ERR_INVALID_ARGUMENT;
  if (!same_view(*in, *out, n) && !views_apart(*in, *out, n, D)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status check_attn(const moe_attn* a) {
  if (!a) return MOE_ERR_INVALID_ARGUMENT;
  if (!(a->scale >= -1e30f && a->scale <= 1e30f)) return MOE_ERR_INVALID_ARGUMENT;
  if (a->window < 0 || a->sinks < 0) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// Sizes that the workspace depends on.
bool sizes_ok(const moe_kv_cache* cache, int q_heads, int n_seqs, int max_pages,
              const moe_attn* a) {
  if (check_cache(cache) != MOE_OK || check_attn(a) != MOE_OK) return false;
  if (q_heads < 1 || q_heads > MOE_MAX_HEADS || q_heads % cache->kv_heads) return false;
  if (n_seqs < 0 || n_seqs > MOE_MAX_PREFILL_TOKENS) return false;
  return max_pages >= 1 && (long long)max_pages * cache->page_size <= kMaxLayoutInt;
}

AttnPlan plan_decode(const moe_kv_cache* c, int q_heads, int n_seqs, int t, int max_pages,
                     const moe_attn* a) {
  return decode_plan(q_heads, c->kv_heads, c->head_dim, n_seqs, t, max_pages, c->page_size,
                     *a, device_cu_count());
}

AttnPlan plan_prefill(const moe_kv_cache* c, int q_heads, int n_seqs, int n, int max_pages,
                      const moe_attn* a) {
  return prefill_plan(q_heads, c->kv_heads, c->head_dim, n_seqs, n, max_pages, c->page_size,
                      *a, device_cu_count());
}

// The checks that decode and prefill share, for n tokens (n > 0) and a workspace of need
// bytes.
moe_status check_attention(const moe_kv_cache* cache, const moe_heads* q, int dtype, int n,
                           const moe_pages* pages, const void* out, const void* ws,
                           size_t ws_bytes, size_t need, const int32_t* q_starts) {
  moe_status s = check_cache_data(cache);
  if (s != MOE_OK) return s;
  s = check_heads(*q);
  if (s != MOE_OK) return s;
  const int D = cache->head_dim;
  if (!pages->table || !pages->kv_lens || !aligned(pages->table, 4) || !aligned(pages->kv_lens, 4))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!out || !aligned(out, 16)) return MOE_ERR_INVALID_ARGUMENT;
  if (need > 0) {
    if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(ws, 256)) return MOE_ERR_INVALID_ARGUMENT;
  }
  const Range o = range(out, 2 * (size_t)n * q->heads * D), w = range(ws, need);
  const Range inputs[] = {
      range(*q, n, D), k_range(cache), v_range(cache),
      range(pages->table, 4 * ((size_t)(pages->n_seqs - 1) * (size_t)pages->table_stride +
                               (size_t)pages->max_pages)),
      range(pages->kv_lens, 4 * (size_t)pages->n_seqs),
      range(q_starts, q_starts ? 4 * ((size_t)pages->n_seqs + 1) : 0),
      range(cache->k_scale, cache->k_scale ? 4 * (size_t)cache->kv_heads : 0),
      range(cache->v_scale, cache->v_scale ? 4 * (size_t)cache->kv_heads : 0)};
  for (const Range& in : inputs)
    if (!disjoint(o, in) || (need > 0 && !disjoint(w, in))) return MOE_ERR_INVALID_ARGUMENT;
  if (need > 0 && !disjoint(o, w)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// The arguments that are checked for a call without tokens, too.
moe_status check_attention_shape(const moe_kv_cache* cache, const moe_heads* q, int dtype,
                                 const moe_pages* pages, const moe_attn* a) {
  moe_status s = check_cache(cache);
  if (s == MOE_OK) s = check_attn(a);
  if (s != MOE_OK) return s;
  if (!q || !pages) return MOE_ERR_INVALID_ARGUMENT;
  if (!dtype_ok(dtype)) return MOE_ERR_UNSUPPORTED;
  if (cache->dtype != MOE_E4M3 && cache->dtype != dtype) return MOE_ERR_UNSUPPORTED;
  if (q->heads < 1 || q->heads > MOE_MAX_HEADS || q->heads % cache->kv_heads)
    return MOE_ERR_INVALID_ARGUMENT;
  if (pages->n_seqs < 0 || pages->n_seqs > MOE_MAX_PREFILL_TOKENS) return MOE_ERR_INVALID_ARGUMENT;
  if (pages->max_pages < 1 || (long long)pages->max_pages * cache->page_size > kMaxLayoutInt)
    return MOE_ERR_INVALID_ARGUMENT;
  if (pages->table_stride < pages->max_pages || pages->table_stride > ((int64_t)1 << 32))
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

}  // namespace
}  // namespace qmoe

using namespace qmoe;

extern "C" {

moe_status moe_qk_norm_rope(const moe_heads* q, const moe_heads* k, const int32_t* positions,
                            int n_tokens, int dtype, int head_dim, const moe_norm_rope* p,
                            const moe_heads* q_out, const moe_heads* k_out, void* stream) {
  if (!p) return MOE_ERR_INVALID_ARGUMENT;
  if (!dtype_ok(dtype) || !head_dim_ok(head_dim)) return MOE_ERR_UNSUPPORTED;
  if (n_tokens < 0 || n_tokens > MOE_MAX_PREFILL_TOKENS) return MOE_ERR_INVALID_ARGUMENT;
  if (n_tokens == 0) return MOE_OK;
  const int n = n_tokens, D = head_dim;
  moe_status s = check_norm_rope(p, D, positions);
  if (s == MOE_OK && has(q)) s = check_pair(q, q_out, n, D);
  if (s == MOE_OK && has(k)) s = check_pair(k, k_out, n, D);
  if (s != MOE_OK) return s;
  if (has(q) && has(k)) {
    if (!views_apart(*q_out, *k_out, n, D) || !views_apart(*q_out, *k, n, D) ||
        !views_apart(*k_out, *q, n, D))
      return MOE_ERR_INVALID_ARGUMENT;
  }
  if ((has(q) && !apart_from_parameters(range(*q_out, n, D), *p, D, positions, n)) ||
      (has(k) && !apart_from_parameters(range(*k_out, n, D), *p, D, positions, n)))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!has(q) && !has(k)) return MOE_OK;
  RowsArgs a{};
  a.q = view(q);
  a.k = view(k);
  a.q_out = has(q) ? view(q_out) : HeadView{};
  a.k_out = has(k) ? view(k_out) : HeadView{};
  a.positions = positions;
  a.n = n;
  a.dtype = dtype;
  a.D = D;
  a.p = *p;
  a.stream = (hipStream_t)stream;
  a.num_cus = device_cu_count();
  return launch_rows(a) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_kv_append(const moe_kv_cache* cache, const moe_heads* k, const moe_heads* v,
                         const int32_t* slots, const int32_t* positions, int n_tokens,
                         int dtype, const moe_norm_rope* p, const moe_heads* q,
                         const moe_heads* q_out, void* stream) {
  moe_status s = check_cache(cache);
  if (s != MOE_OK) return s;
  if (!dtype_ok(dtype)) return MOE_ERR_UNSUPPORTED;
  if (cache->dtype != MOE_E4M3 && cache->dtype != dtype) return MOE_ERR_UNSUPPORTED;
  if (n_tokens < 0 || n_tokens > MOE_MAX_PREFILL_TOKENS) return MOE_ERR_INVALID_ARGUMENT;
  if (n_tokens == 0) return MOE_OK;
  const int n = n_tokens, D = cache->head_dim;
  s = check_cache_data(cache);
  if (s != MOE_OK) return s;
  if (!has(k) || !has(v) || !slots || !aligned(slots, 4)) return MOE_ERR_INVALID_ARGUMENT;
  s = check_heads(*k);
  if (s == MOE_OK) s = check_heads(*v);
  if (s != MOE_OK) return s;
  if (k->heads != cache->kv_heads || v->heads != cache->kv_heads) return MOE_ERR_INVALID_ARGUMENT;
  if (!p && has(q)) return MOE_ERR_INVALID_ARGUMENT;
  const moe_norm_rope plain{};
  if (!p) p = &plain;
  s = check_norm_rope(p, D, positions);
  if (s == MOE_OK && has(q)) s = check_pair(q, q_out, n, D);
  if (s != MOE_OK) return s;
  // no input of the call lies in what it writes
  const Range kc = k_range(cache), vc = v_range(cache);
  const Range qo = has(q) ? range(*q_out, n, D) : Range{0, 0};
  const Range inputs[] = {range(*k, n, D), range(*v, n, D), has(q) ? range(*q, n, D) : Range{0, 0}};
  const Range kscale = range(cache->k_scale, cache->k_scale ? 4 * (size_t)cache->kv_heads : 0);
  const Range vscale = range(cache->v_scale, cache->v_scale ? 4 * (size_t)cache->kv_heads : 0);
  if (!disjoint(kc, vc) || !disjoint(kc, qo) || !disjoint(vc, qo)) return MOE_ERR_INVALID_ARGUMENT;
  for (const Range& in : inputs)
    if (!disjoint(kc, in) || !disjoint(vc, in)) return MOE_ERR_INVALID_ARGUMENT;
  for (const Range& out : {kc, vc, qo})
    if (!disjoint(out, range(slots, 4 * (size_t)n)) || !disjoint(out, kscale) ||
        !disjoint(out, vscale) || !apart_from_parameters(out, *p, D, positions, n))
      return MOE_ERR_INVALID_ARGUMENT;
  if (has(q) && (!views_apart(*q_out, *k, n, D) || !views_apart(*q_out, *v, n, D)))
    return MOE_ERR_INVALID_ARGUMENT;
  RowsArgs a{};
  a.q = view(q);
  a.k = view(k);
  a.v = view(v);
  a.q_out = has(q) ? view(q_out) : HeadView{};
  a.positions = positions;
  a.slots = slots;
  a.n = n;
  a.dtype = dtype;
  a.D = D;
  a.p = *p;
  a.cache = cache;
  a.stream = (hipStream_t)stream;
  a.num_cus = device_cu_count();
  return launch_rows(a) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

size_t moe_attn_decode_workspace_bytes(const moe_kv_cache* cache, int q_heads, int n_seqs,
                                       int window_tokens, int max_pages, const moe_attn* a) {
  if (!sizes_ok(cache, q_heads, n_seqs, max_pages, a) || n_seqs == 0) return 0;
  if (window_tokens < 1 || window_tokens > MOE_MAX_WINDOW_TOKENS) return 0;
  if ((long long)n_seqs * window_tokens > MOE_MAX_DECODE_TOKENS) return 0;
  return plan_decode(cache, q_heads, n_seqs, window_tokens, max_pages, a).total;
}

moe_status moe_attn_decode(const moe_kv_cache* cache, const moe_heads* q, int dtype,
                           const moe_pages* pages, int window_tokens, const moe_attn* a,
                           void* out, void* ws, size_t ws_bytes, void* stream) {
  moe_status s = check_attention_shape(cache, q, dtype, pages, a);
  if (s != MOE_OK) return s;
  if (window_tokens < 1 || window_tokens > MOE_MAX_WINDOW_TOKENS) return MOE_ERR_INVALID_ARGUMENT;
  if ((long long)pages->n_seqs * window_tokens > MOE_MAX_DECODE_TOKENS)
    return MOE_ERR_INVALID_ARGUMENT;
  if (pages->n_seqs == 0) return MOE_OK;
  const int n = pages->n_seqs * window_tokens;
  if (!has(q)) return MOE_ERR_INVALID_ARGUMENT;
  const AttnPlan plan =
      plan_decode(cache, q->heads, pages->n_seqs, window_tokens, pages->max_pages, a);
  s = check_attention(cache, q, dtype, n, pages, out, ws, ws_bytes, plan.total, nullptr);
  if (s != MOE_OK) return s;
  const AttnArgs args{view(q), dtype, *cache,     *pages,     *a, nullptr,
                      n,       window_tokens, (char*)out, (char*)ws,   (hipStream_t)stream};
  return launch_attn_decode(args, plan) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

size_t moe_attn_prefill_workspace_bytes(const moe_kv_cache* cache, int q_heads, int n_seqs,
                                        int n_tokens, int max_pages, const moe_attn* a) {
  if (!sizes_ok(cache, q_heads, n_seqs, max_pages, a) || n_seqs == 0) return 0;
  if (n_tokens < 1 || n_tokens > MOE_MAX_PREFILL_TOKENS) return 0;
  return plan_prefill(cache, q_heads, n_seqs, n_tokens, max_pages, a).total;
}

moe_status moe_attn_prefill(const moe_kv_cache* cache, const moe_heads* q, int dtype,
                            const int32_t* q_starts, int n_tokens, const moe_pages* pages,
                            const moe_attn* a, void* out, void* ws, size_t ws_bytes,
                            void* stream) {
  moe_status s = check_attention_shape(cache, q, dtype, pages, a);
  if (s != MOE_OK) return s;
  if (n_tokens < 0 || n_tokens > MOE_MAX_PREFILL_TOKENS) return MOE_ERR_INVALID_ARGUMENT;
  if (n_tokens == 0 || pages->n_seqs == 0) return MOE_OK;
  if (!has(q) || !q_starts || !aligned(q_starts, 4)) return MOE_ERR_INVALID_ARGUMENT;
  const AttnPlan plan =
      plan_prefill(cache, q->heads, pages->n_seqs, n_tokens, pages->max_pages, a);
  s = check_attention(cache, q, dtype, n_tokens, pages, out, ws, ws_bytes, plan.total, q_starts);
  if (s != MOE_OK) return s;
  const AttnArgs args{view(q),  dtype, *cache,     *pages,   *a,        q_starts,
                      n_tokens, 0,     (char*)out, (char*)ws, (hipStream_t)stream};
  return launch_attn_prefill(args, plan) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
