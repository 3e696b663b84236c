// C ABI of routing by a rule and of the microscaled 4-bit products: argument validation and
// workspace queries. Every check runs on the host before anything is enqueued.
#include "qmoe_mx_internal.h"

namespace qmoe {
namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

Range range(const void* p, size_t bytes) { return {(uintptr_t)p, (uintptr_t)p + (p ? bytes : 0)}; }

bool disjoint(const Range& a, const Range& b) {
  return a.lo == a.hi || b.lo == b.hi || a.hi <= b.lo || b.hi <= a.lo;
}

bool dtype_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }

constexpr int64_t kMost = (int64_t)1 << 40;  // rows times columns, and strides, stay below

// Rows of values: 16-byte words all through.
moe_status check_rows(const void* x, int dtype, int64_t rows, int cols, int64_t stride) {
  if (!dtype_ok(dtype)) return MOE_ERR_UNSUPPORTED;
  if (cols < kMxBlock || cols % kMxBlock || cols > MOE_MX_MAX_COLS) return MOE_ERR_INVALID_ARGUMENT;
  if (rows < 0 || rows > kMost / cols) return MOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MOE_OK;
  if (!x || !aligned(x, 16)) return MOE_ERR_INVALID_ARGUMENT;
  if (rows > 1 && (stride < 0 || stride > kMost / rows || stride * mx_type_size(dtype) % 16))
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

Range rows_range(const void* x, int dtype, int64_t rows, int cols, int64_t stride) {
  if (rows == 0) return range(x, 0);
  return range(x, ((size_t)(rows - 1) * (rows > 1 ? (size_t)stride : 0) + cols) * mx_type_size(dtype));
}

// Whether n rows of a and n of b certainly share no byte: their ranges are apart, or rows of both
// lie one distance apart and each row's parts side by side in it (columns of one buffer).
bool rows_apart(const void* a, int64_t a_step, int64_t a_bytes, const void* b, int64_t b_step, int64_t b_bytes,
                int n) {
  const Range ra = range(a, (size_t)((n - 1) * a_step + a_bytes)), rb = range(b, (size_t)((n - 1) * b_step + b_bytes));
  if (disjoint(ra, rb)) return true;
  if (n == 1 || a_step != b_step || a_step <= 0) return false;
  // from the start of a row of a to that of the next row of b
  const uintptr_t step = (uintptr_t)a_step, ahead = rb.lo % step, at = ra.lo % step;
  const uintptr_t gap = ahead >= at ? ahead - at : ahead + step - at;
  return gap >= (uintptr_t)a_bytes && gap + (uintptr_t)b_bytes <= step;
}

moe_status check_matrix(const moe_mx_matrix* m) {
  if (!m) return MOE_ERR_INVALID_ARGUMENT;
  if (m->rows < 1 || m->rows > MOE_MX_MAX_ROWS) return MOE_ERR_INVALID_ARGUMENT;
  if (m->cols < kMxBlock || m->cols % kMxBlock || m->cols > MOE_MX_MAX_COLS)
    return MOE_ERR_INVALID_ARGUMENT;
  if (!m->codes || !m->scales || !aligned(m->codes, 16) || !aligned(m->scales, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

Range codes_range(const moe_mx_matrix& m, int64_t count) {
  return range(m.codes, (size_t)count * m.rows * (m.cols / 2));
}
Range scales_range(const moe_mx_matrix& m, int64_t count) {
  return range(m.scales, (size_t)count * m.rows * (m.cols / kMxBlock));
}

moe_status check_out(const void* out, int dtype, int n, int cols, int64_t stride, Range* r) {
  if (!dtype_ok(dtype)) return MOE_ERR_UNSUPPORTED;
  const int size = mx_type_size(dtype);
  if (!out || !aligned(out, size)) return MOE_ERR_INVALID_ARGUMENT;
  if (n > 1 && (stride < cols || stride > kMost / n)) return MOE_ERR_INVALID_ARGUMENT;
  *r = rows_range(out, dtype, n, cols, stride);
  return MOE_OK;
}

moe_status status_of(hipError_t err) { return err == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

moe_status check_layer(const moe_mx_layer* L) {
  if (!L) return MOE_ERR_INVALID_ARGUMENT;
  const int d = L->d_model, f = L->d_ff, E = L->n_experts, k = L->top_k;
  if (d <= 0 || f <= 0 || d % 32 || f % 32 || d > 8192 || f > 8192) return MOE_ERR_INVALID_ARGUMENT;
  if (E < 1 || E > MOE_MAX_EXPERTS || k < 1 || k > E || k > MOE_MAX_TOP_K)
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

}  // namespace
}  // namespace qmoe

using namespace qmoe;

extern "C" {

moe_status moe_route_scored(const void* logits, int dtype, int n_tokens, int n_experts, int top_k,
                            const moe_route_rule* rule, const moe_routing* out, void* ws,
                            size_t ws_bytes, void* stream) {
  if (n_tokens < 0 || n_tokens > MOE_MAX_ROUTE_TOKENS) return MOE_ERR_INVALID_ARGUMENT;
  if (n_experts < 1 || n_experts > MOE_MAX_EXPERTS) return MOE_ERR_INVALID_ARGUMENT;
  if (top_k < 1 || top_k > n_experts || top_k > MOE_MAX_TOP_K) return MOE_ERR_INVALID_ARGUMENT;
  if (!dtype_ok(dtype)) return MOE_ERR_UNSUPPORTED;
  if (!rule) return MOE_ERR_INVALID_ARGUMENT;
  if (rule->score != MOE_SCORE_SIGMOID && rule->score != MOE_SCORE_SOFTMAX)
    return MOE_ERR_INVALID_ARGUMENT;
  if (rule->group_score != MOE_GROUP_MAX && rule->group_score != MOE_GROUP_TOP2)
    return MOE_ERR_INVALID_ARGUMENT;
  if (rule->groups < 1 || rule->groups > MOE_MAX_ROUTE_GROUPS || n_experts % rule->groups ||
      rule->top_groups < 1 || rule->top_groups > rule->groups ||
      rule->top_groups * (n_experts / rule->groups) < top_k)
    return MOE_ERR_INVALID_ARGUMENT;
  if (rule->renormalize != 0 && rule->renormalize != 1) return MOE_ERR_INVALID_ARGUMENT;
  if (!(rule->scale - rule->scale == 0.0f)) return MOE_ERR_INVALID_ARGUMENT;  // inf, NaN
  if (!aligned(rule->bias, 4)) return MOE_ERR_INVALID_ARGUMENT;
  if (!out || !out->expert_offsets || !aligned(out->expert_offsets, 4)) return MOE_ERR_INVALID_ARGUMENT;
  if (n_tokens > 0) {
    if (!out->topk_ids || !out->topk_w || !out->pair_index || !logits ||
        !aligned(logits, mx_type_size(dtype)))
      return MOE_ERR_INVALID_ARGUMENT;
    const size_t P = (size_t)n_tokens * top_k;
    const Range reads[] = {range(logits, (size_t)n_tokens * n_experts * mx_type_size(dtype)),
                           range(rule->bias, 4 * (size_t)n_experts)};
    const Range writes[] = {range(out->topk_ids, 4 * P), range(out->topk_w, 4 * P),
                            range(out->pair_index, 4 * P),
                            range(out->expert_offsets, 4 * ((size_t)n_experts + 1))};
    const size_t need = route_workspace_bytes(n_tokens, n_experts, top_k);
    if (need > 0) {
      if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
      if (!aligned(ws, 256)) return MOE_ERR_INVALID_ARGUMENT;
    }
    const Range work = range(ws, need);
    for (const Range& r : reads)
      if (!disjoint(work, r)) return MOE_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < 4; ++i) {
      if (!aligned((const void*)writes[i].lo, 4) || !disjoint(work, writes[i])) return MOE_ERR_INVALID_ARGUMENT;
      for (const Range& r : reads)
        if (!disjoint(writes[i], r)) return MOE_ERR_INVALID_ARGUMENT;
      for (int j = 0; j < i; ++j)
        if (!disjoint(writes[i], writes[j])) return MOE_ERR_INVALID_ARGUMENT;
    }
  }
  return status_of(launch_route_scored(logits, dtype, n_tokens, n_experts, top_k, *rule, out, ws,
                                       (hipStream_t)stream));
}

moe_status moe_mx_quantize(const void* x, int dtype, int64_t rows, int cols, int64_t row_stride,
                           uint8_t* codes, uint8_t* scales, void* stream) {
  const moe_status s = check_rows(x, dtype, rows, cols, row_stride);
  if (s != MOE_OK || rows == 0) return s;
  if (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16)) return MOE_ERR_INVALID_ARGUMENT;
  if (rows == 1) row_stride = cols;  // whatever it said
  const Range in = rows_range(x, dtype, rows, cols, row_stride);
  const Range c = range(codes, (size_t)rows * (cols / 2)), sc = range(scales, (size_t)rows * (cols / kMxBlock));
  if (!disjoint(in, c) || !disjoint(in, sc) || !disjoint(c, sc)) return MOE_ERR_INVALID_ARGUMENT;
  return status_of(launch_mx_quantize(MxQuantArgs{x, dtype, rows, row_stride, cols, codes, scales},
                                      (hipStream_t)stream));
}

moe_status moe_mx_dequantize(const moe_mx_matrix* m, int64_t rows, int dtype, void* out, void* stream) {
  if (!m) return MOE_ERR_INVALID_ARGUMENT;
  if (!dtype_ok(dtype)) return MOE_ERR_UNSUPPORTED;
  if (m->cols < kMxBlock || m->cols % kMxBlock || m->cols > MOE_MX_MAX_COLS || rows < 0 ||
      rows > kMost / m->cols)
    return MOE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MOE_OK;
  if (!m->codes || !m->scales || !out || !aligned(m->codes, 16) || !aligned(m->scales, 16) ||
      !aligned(out, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  const Range o = range(out, (size_t)rows * m->cols * mx_type_size(dtype));
  if (!disjoint(o, range(m->codes, (size_t)rows * (m->cols / 2))) ||
      !disjoint(o, range(m->scales, (size_t)rows * (m->cols / kMxBlock))))
    return MOE_ERR_INVALID_ARGUMENT;
  return status_of(launch_mx_dequantize(m->codes, m->scales, rows * (m->cols / kMxBlock), out, dtype,
                                        (hipStream_t)stream));
}

size_t moe_mx_linear_workspace_bytes(int n_tokens, int cols) {
  if (n_tokens < 0 || n_tokens > MOE_MAX_ROUTE_TOKENS || cols < kMxBlock || cols % kMxBlock ||
      cols > MOE_MX_MAX_COLS)
    return 0;
  return mx_linear_ws(n_tokens, cols);
}

moe_status moe_mx_linear(const void* x, int dtype, int64_t row_stride, int n_tokens,
                         const moe_mx_matrix* w, void* out, int out_dtype, int64_t out_stride,
                         void* ws, size_t ws_bytes, void* stream) {
  moe_status s = check_matrix(w);
  if (s != MOE_OK) return s;
  if (n_tokens < 0 || n_tokens > MOE_MAX_ROUTE_TOKENS) return MOE_ERR_INVALID_ARGUMENT;
  s = check_rows(x, dtype, n_tokens, w->cols, row_stride);
  if (s != MOE_OK) return s;
  if (n_tokens == 0) return dtype_ok(out_dtype) ? MOE_OK : MOE_ERR_UNSUPPORTED;
  if (n_tokens == 1) {
    row_stride = w->cols;
    out_stride = w->rows;
  }
  Range o{};
  s = check_out(out, out_dtype, n_tokens, w->rows, out_stride, &o);
  if (s != MOE_OK) return s;
  const Range in = rows_range(x, dtype, n_tokens, w->cols, row_stride);
  const int64_t xs = mx_type_size(dtype), os = mx_type_size(out_dtype);
  if (!rows_apart(x, row_stride * xs, w->cols * xs, out, out_stride * os, w->rows * os, n_tokens) ||
      !disjoint(o, codes_range(*w, 1)) || !disjoint(o, scales_range(*w, 1)))
    return MOE_ERR_INVALID_ARGUMENT;
  const size_t need = mx_linear_ws(n_tokens, w->cols);
  if (need > 0) {
    if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(ws, 256)) return MOE_ERR_INVALID_ARGUMENT;
    const Range wr = range(ws, need);
    if (!disjoint(wr, o) || !disjoint(wr, in) || !disjoint(wr, codes_range(*w, 1)) ||
        !disjoint(wr, scales_range(*w, 1)))
      return MOE_ERR_INVALID_ARGUMENT;
  }
  MxLinearArgs a{};
  a.x = x;
  a.dtype = dtype;
  a.row_stride = row_stride;
  a.n = n_tokens;
  a.N = w->rows;
  a.K = w->cols;
  a.w = w->codes;
  a.ws = w->scales;
  a.out = out;
  a.out_dtype = out_dtype;
  a.out_stride = out_stride;
  a.work = (char*)ws;
  return status_of(launch_mx_linear(a, (hipStream_t)stream));
}

moe_status moe_mx_linear_quantized(const moe_mx_matrix* x, const moe_mx_matrix* w, void* out,
                                   int out_dtype, int64_t out_stride, void* stream) {
  moe_status s = check_matrix(w);
  if (s != MOE_OK) return s;
  if (!x || x->cols != w->cols || x->rows < 0 || x->rows > MOE_MAX_ROUTE_TOKENS)
    return MOE_ERR_INVALID_ARGUMENT;
  if (x->rows == 0) return dtype_ok(out_dtype) ? MOE_OK : MOE_ERR_UNSUPPORTED;
  s = check_matrix(x);
  if (s != MOE_OK) return s;
  if (x->rows == 1) out_stride = w->rows;
  Range o{};
  s = check_out(out, out_dtype, x->rows, w->rows, out_stride, &o);
  if (s != MOE_OK) return s;
  if (!disjoint(o, codes_range(*x, 1)) || !disjoint(o, scales_range(*x, 1)) ||
      !disjoint(o, codes_range(*w, 1)) || !disjoint(o, scales_range(*w, 1)))
    return MOE_ERR_INVALID_ARGUMENT;
  MxLinearArgs a{};
  a.xq = x->codes;
  a.xs = x->scales;
  a.n = x->rows;
  a.N = w->rows;
  a.K = w->cols;
  a.w = w->codes;
  a.ws = w->scales;
  a.out = out;
  a.out_dtype = out_dtype;
  a.out_stride = out_stride;
  return status_of(launch_mx_linear(a, (hipStream_t)stream));
}

size_t moe_mx_ffn_workspace_bytes(const moe_mx_layer* L, int n_tokens) {
  if (check_layer(L) != MOE_OK || n_tokens < 0 || n_tokens > MOE_MAX_PREFILL_TOKENS) return 0;
  return n_tokens == 0 ? 0 : mx_ffn_ws(n_tokens, L->top_k, L->d_model, L->d_ff, L->n_experts).total;
}

moe_status moe_mx_ffn(const moe_mx_layer* L, const void* x, int dtype, int64_t row_stride,
                      int n_tokens, const moe_routing* r, const float* residual, float* out,
                      void* ws, size_t ws_bytes, void* stream) {
  moe_status s = check_layer(L);
  if (s != MOE_OK) return s;
  const int d = L->d_model, f = L->d_ff, E = L->n_experts, k = L->top_k;
  const moe_mx_matrix* mats[] = {&L->gate, &L->up, &L->down};
  for (const moe_mx_matrix* m : mats) {
    s = check_matrix(m);
    if (s != MOE_OK) return s;
    if (m->rows != (m == &L->down ? d : f) || m->cols != (m == &L->down ? f : d))
      return MOE_ERR_INVALID_ARGUMENT;
  }
  if (n_tokens < 0 || n_tokens > MOE_MAX_PREFILL_TOKENS) return MOE_ERR_INVALID_ARGUMENT;
  s = check_rows(x, dtype, n_tokens, d, row_stride);
  if (s != MOE_OK || n_tokens == 0) return s;
  if (n_tokens == 1) row_stride = d;
  if (!r || !r->topk_ids || !r->topk_w || !r->expert_offsets || !r->pair_index)
    return MOE_ERR_INVALID_ARGUMENT;
  if (!out || !aligned(out, 16) || !aligned(residual, 16)) return MOE_ERR_INVALID_ARGUMENT;
  const size_t need = mx_ffn_ws(n_tokens, k, d, f, E).total;
  if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(ws, 256)) return MOE_ERR_INVALID_ARGUMENT;
  const size_t rows = 4 * (size_t)n_tokens * d, P = (size_t)n_tokens * k;
  const Range o = range(out, rows), res = range(residual, rows), work = range(ws, need);
  if (residual != out && !disjoint(o, res)) return MOE_ERR_INVALID_ARGUMENT;
  if (!disjoint(work, o) || !disjoint(work, res)) return MOE_ERR_INVALID_ARGUMENT;
  const Range reads[] = {rows_range(x, dtype, n_tokens, d, row_stride),
                         codes_range(L->gate, E), scales_range(L->gate, E),
                         codes_range(L->up, E), scales_range(L->up, E),
                         codes_range(L->down, E), scales_range(L->down, E),
                         range(r->topk_ids, 4 * P), range(r->topk_w, 4 * P),
                         range(r->pair_index, 4 * P), range(r->expert_offsets, 4 * ((size_t)E + 1))};
  for (const Range& in : reads)
    if (!disjoint(o, in) || !disjoint(work, in)) return MOE_ERR_INVALID_ARGUMENT;
  MxFfnArgs a{L, x, dtype, n_tokens, row_stride, r, residual, out, (char*)ws};
  return status_of(launch_mx_ffn(a, (hipStream_t)stream));
}

}  // extern "C"
