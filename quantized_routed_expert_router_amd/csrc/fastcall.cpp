// Short path of the Python calls of the attention half, of routing by a rule and of the
// microscaled products: checks of the tensors, output allocation and the C ABI call in one
// native step. The kernels behind these calls run for a few microseconds, less than the same
// checks take in Python.
//
// Every function answers None when an argument is not exactly what the call needs (the
// Python side then checks one by one and says which), the status of the C call when it is
// not MOE_OK, and the outputs otherwise.
#include <Python.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include <algorithm>

#include "qmoe.h"

namespace {

using at::Tensor;

struct Mismatch {};  // caught at the entry: the answer is None

// Arguments of one call, read in order; every tensor is on the one GPU.
class Args {
 public:
  Args(PyObject* const* args, Py_ssize_t n, int device) : args_(args), n_(n), device_(device) {}

  const Tensor* tensor() {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_CheckExact(o)) throw Mismatch();
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device_ || t.layout() != at::kStrided) throw Mismatch();
    return &t;
  }
  const Tensor& required() {
    const Tensor* t = tensor();
    if (!t) throw Mismatch();
    return *t;
  }
  // The next argument, a tensor, which stays the next one.
  const Tensor* peek() {
    const Tensor& t = required();
    --at_;
    return &t;
  }
  // A contiguous tensor of a type and one dimension of n entries (n < 0: any), or none.
  const void* vector(at::ScalarType type, int64_t n) {
    const Tensor* t = tensor();
    if (!t) return nullptr;
    if (t->scalar_type() != type || t->dim() != 1 || (n >= 0 && t->size(0) != n) ||
        !t->is_contiguous())
      throw Mismatch();
    return t->data_ptr();
  }
  double number() {
    const double x = PyFloat_AsDouble(next());
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Mismatch();
    }
    return x;
  }
  int32_t integer() {
    const long long x = PyLong_AsLongLong(next());
    if (PyErr_Occurred() || x < 0 || x > 0x7fffffffll) {
      PyErr_Clear();
      throw Mismatch();
    }
    return (int32_t)x;
  }
  void* stream() {
    const unsigned long long x = PyLong_AsUnsignedLongLong(next());
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Mismatch();
    }
    return (void*)(uintptr_t)x;
  }

 private:
  PyObject* next() {
    if (at_ >= n_) throw Mismatch();
    return args_[at_++];
  }
  PyObject* const* args_;
  Py_ssize_t n_, at_ = 0;
  int device_;
};

int dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16:
      return MOE_BF16;
    case at::kHalf:
      return MOE_F16;
    case at::kFloat8_e4m3fn:
      return MOE_E4M3;
    default:
      throw Mismatch();
  }
}

// Heads [n, heads, D] of 16-bit elements.
moe_heads heads_of(const Tensor& t, const Tensor* like, bool same_heads) {
  if (t.dim() != 3 || t.stride(2) != 1 || dtype_of(t) == MOE_E4M3) throw Mismatch();
  if (like && (t.scalar_type() != like->scalar_type() || t.size(0) != like->size(0) ||
               t.size(2) != like->size(2) || (same_heads && t.size(1) != like->size(1))))
    throw Mismatch();
  if (t.size(0) > MOE_MAX_ROUTE_TOKENS || t.size(1) > MOE_MAX_HEADS || t.size(2) > 65536)
    throw Mismatch();
  return moe_heads{t.data_ptr(), t.stride(0), t.stride(1), (int32_t)t.size(1)};
}

moe_kv_cache cache_of(Args& a) {
  const Tensor &k = a.required(), &v = a.required();
  moe_kv_cache c{};
  c.dtype = dtype_of(k);
  if (k.dim() != 4 || v.dim() != 5 || v.scalar_type() != k.scalar_type() || !k.is_contiguous() ||
      !v.is_contiguous() || v.size(0) != k.size(0) || v.size(1) != k.size(1) ||
      v.size(2) != k.size(2) / 8 || v.size(3) != k.size(3) || v.size(4) != 8)
    throw Mismatch();
  for (int i = 0; i < 4; ++i)
    if (k.size(i) > 0x7fffffff) throw Mismatch();
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.num_pages = (int32_t)k.size(0);
  c.kv_heads = (int32_t)k.size(1);
  c.page_size = (int32_t)k.size(2);
  c.head_dim = (int32_t)k.size(3);
  c.k_scale = (const float*)a.vector(at::kFloat, c.kv_heads);
  c.v_scale = (const float*)a.vector(at::kFloat, c.kv_heads);
  return c;
}

moe_norm_rope norm_rope_of(Args& a, int64_t D) {
  moe_norm_rope p{};
  p.q_norm = (const float*)a.vector(at::kFloat, D);
  p.k_norm = (const float*)a.vector(at::kFloat, D);
  if (const Tensor* f = a.tensor()) {
    if (f->scalar_type() != at::kFloat || f->dim() != 1 || !f->is_contiguous() ||
        f->size(0) > 65536)
      throw Mismatch();
    p.inv_freq = (const float*)f->data_ptr();
    p.rot_dim = 2 * (int32_t)f->size(0);
  }
  p.eps = (float)a.number();
  p.weight_offset = (float)a.number();
  p.interleaved = a.integer() != 0;
  return p;
}

// Other Python threads run meanwhile: an allocation may have to wait for the device, a launch
// for room in the stream's queue. Held around everything from the first allocation to the
// launch; no Python object is made or read inside.
class WithoutGil {
 public:
  WithoutGil() : state_(PyEval_SaveThread()) {}
  ~WithoutGil() { PyEval_RestoreThread(state_); }
  WithoutGil(const WithoutGil&) = delete;

 private:
  PyThreadState* state_;
};

Tensor new_like(const Tensor& t) {
  return at::empty(t.sizes(), t.options(), at::MemoryFormat::Contiguous);
}

moe_heads dense(const Tensor& t) {
  return moe_heads{t.data_ptr(), t.size(1) * t.size(2), t.size(2), (int32_t)t.size(1)};
}

// Errors of torch (an allocation that fails) become the exceptions that torch's own calls raise.
template <typename F>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, F body) {
  HANDLE_TH_ERRORS
  try {
    const long device = n > 0 ? PyLong_AsLong(args[0]) : -1;
    if (PyErr_Occurred()) PyErr_Clear();
    if (device < 0) Py_RETURN_NONE;
    Args a(args + 1, n - 1, (int)device);
    return body(a);
  } catch (const Mismatch&) {
    Py_RETURN_NONE;
  }
  END_HANDLE_TH_ERRORS
}

// (device, q, k, positions, q_norm, k_norm, inv_freq, eps, weight_offset, interleaved, stream)
// -> (q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, [](Args& a) -> PyObject* {
    const Tensor &q = a.required(), &k = a.required();
    const moe_heads qs = heads_of(q, nullptr, false), ks = heads_of(k, &q, false);
    const int32_t* positions = (const int32_t*)a.vector(at::kInt, q.size(0));
    const moe_norm_rope p = norm_rope_of(a, q.size(2));
    void* stream = a.stream();
    Tensor qo, ko;
    moe_status s;
    {
      const WithoutGil free;
      qo = new_like(q);
      ko = new_like(k);
      const moe_heads qos = dense(qo), kos = dense(ko);
      s = moe_qk_norm_rope(&qs, &ks, positions, (int)q.size(0), dtype_of(q), (int)q.size(2), &p,
                           &qos, &kos, stream);
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    PyObject* pair = PyTuple_New(2);
    if (!pair) return nullptr;
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(std::move(qo)));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(ko)));
    return pair;
  });
}

// (device, cache k, v, k_scale, v_scale, k, v, slots, positions, q_norm, k_norm, inv_freq, eps,
// weight_offset, interleaved, q, stream) -> q_out
PyObject* kv_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, [](Args& a) -> PyObject* {
    const moe_kv_cache c = cache_of(a);
    const Tensor &k = a.required(), &v = a.required();
    const moe_heads ks = heads_of(k, nullptr, false), vs = heads_of(v, &k, true);
    if (k.size(1) != c.kv_heads || k.size(2) != c.head_dim) throw Mismatch();
    const int32_t* slots = (const int32_t*)a.vector(at::kInt, k.size(0));
    const int32_t* positions = (const int32_t*)a.vector(at::kInt, k.size(0));
    if (!slots) throw Mismatch();
    const moe_norm_rope p = norm_rope_of(a, k.size(2));
    const Tensor& q = a.required();
    const moe_heads qs = heads_of(q, &k, false);
    void* stream = a.stream();
    Tensor qo;
    moe_status s;
    {
      const WithoutGil free;
      qo = new_like(q);
      const moe_heads qos = dense(qo);
      s = moe_kv_append(&c, &ks, &vs, slots, positions, (int)k.size(0), dtype_of(k), &p, &qs, &qos,
                        stream);
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    return THPVariable_Wrap(std::move(qo));
  });
}

// (device, cache k, v, k_scale, v_scale, q, q_starts or None, page_table, kv_lens, scale,
// window, sinks, stream) -> out
PyObject* attend(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, [](Args& a) -> PyObject* {
    const moe_kv_cache c = cache_of(a);
    const Tensor& q = a.required();
    const moe_heads qs = heads_of(q, nullptr, false);
    if (q.size(2) != c.head_dim || q.size(0) == 0) throw Mismatch();
    const Tensor* starts = a.tensor();
    const Tensor& table = a.required();
    if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) < 1 ||
        table.size(0) > MOE_MAX_ROUTE_TOKENS || table.size(1) > 0x7fffffff ||
        (table.size(1) > 1 && table.stride(1) != 1) ||
        (table.size(0) > 1 && table.stride(0) < table.size(1)))
      throw Mismatch();
    const int b = (int)table.size(0);
    if (starts && (starts->scalar_type() != at::kInt || starts->dim() != 1 ||
                   starts->size(0) != b + 1 || !starts->is_contiguous()))
      throw Mismatch();
    const moe_pages pages{(const int32_t*)table.data_ptr(), (const int32_t*)a.vector(at::kInt, b),
                          b > 1 ? table.stride(0) : table.size(1), b, (int32_t)table.size(1)};
    moe_attn p{};
    p.scale = (float)a.number();
    p.window = a.integer();
    p.sinks = a.integer();
    void* stream = a.stream();
    const int tokens = (int)q.size(0), heads = qs.heads;
    if (!starts && tokens % b) throw Mismatch();
    const size_t need =
        starts ? moe_attn_prefill_workspace_bytes(&c, heads, b, tokens, pages.max_pages, &p)
               : moe_attn_decode_workspace_bytes(&c, heads, b, tokens / b, pages.max_pages, &p);
    Tensor out;
    moe_status s;
    {
      const WithoutGil free;
      Tensor ws;
      out = new_like(q);
      if (need) ws = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
      void* room = need ? ws.data_ptr() : nullptr;
      s = starts ? moe_attn_prefill(&c, &qs, dtype_of(q), (const int32_t*)starts->data_ptr(),
                                    tokens, &pages, &p, out.data_ptr(), room, need, stream)
                 : moe_attn_decode(&c, &qs, dtype_of(q), &pages, tokens / b, &p, out.data_ptr(),
                                   room, need, stream);
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    return THPVariable_Wrap(std::move(out));
  });
}

// ---- routing by a rule and microscaled products

int float_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat:
      return MOE_F32;
    case at::kBFloat16:
      return MOE_BF16;
    case at::kHalf:
      return MOE_F16;
    default:
      throw Mismatch();
  }
}

at::ScalarType type_of(int dtype) {
  return dtype == MOE_F32 ? at::kFloat : dtype == MOE_BF16 ? at::kBFloat16 : at::kHalf;
}

// Rows [n, cols] of floats, the last axis contiguous, and their stride.
const Tensor& rows_of(Args& a, int64_t cols, int64_t* stride) {
  const Tensor& t = a.required();
  float_of(t);
  if (t.dim() != 2 || (cols >= 0 && t.size(1) != cols) || t.size(0) > MOE_MAX_ROUTE_TOKENS ||
      t.size(1) > MOE_MX_MAX_COLS || (t.size(1) > 1 && t.stride(1) != 1))
    throw Mismatch();
  *stride = t.size(0) > 1 ? t.stride(0) : t.size(1);
  return t;
}

// Codes and scales of a matrix of `dims` axes.
moe_mx_matrix mx_of(Args& a, int dims, const Tensor** codes_out) {
  const Tensor &c = a.required(), &s = a.required();
  if (c.scalar_type() != at::kByte || s.scalar_type() != at::kByte || c.dim() != dims || s.dim() != dims ||
      !c.is_contiguous() || !s.is_contiguous())
    throw Mismatch();
  const int64_t half = c.size(dims - 1), rows = c.size(dims - 2);
  if (half % 16 || half < 16 || half > MOE_MX_MAX_COLS / 2 || rows < 1 || rows > MOE_MX_MAX_ROWS ||
      s.size(dims - 1) != half / 16)
    throw Mismatch();
  for (int i = 0; i + 1 < dims; ++i)
    if (s.size(i) != c.size(i)) throw Mismatch();
  if (codes_out) *codes_out = &c;
  return moe_mx_matrix{(const uint8_t*)c.data_ptr(), (const uint8_t*)s.data_ptr(), (int32_t)rows,
                       (int32_t)(2 * half)};
}

// (device, logits, top_k, score, bias, groups, top_groups, group_score, renormalize, scale, stream)
// -> (topk_ids, topk_w, expert_offsets, pair_index)
PyObject* route_scored(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  return guarded(args, n_args, [](Args& a) -> PyObject* {
    const Tensor& l = a.required();
    const int dtype = float_of(l);
    if (l.dim() != 2 || !l.is_contiguous() || l.size(0) > MOE_MAX_ROUTE_TOKENS || l.size(1) > MOE_MAX_EXPERTS)
      throw Mismatch();
    const int n = (int)l.size(0), E = (int)l.size(1), k = a.integer();
    if (k < 1 || k > E || k > MOE_MAX_TOP_K) throw Mismatch();
    moe_route_rule rule{};
    rule.score = a.integer();
    rule.bias = (const float*)a.vector(at::kFloat, E);
    rule.groups = a.integer();
    rule.top_groups = a.integer();
    rule.group_score = a.integer();
    rule.renormalize = a.integer();
    rule.scale = (float)a.number();
    void* stream = a.stream();
    Tensor out[4];
    moe_status s;
    {
      const WithoutGil free;
      const auto ints = l.options().dtype(at::kInt);
      out[0] = at::empty({n, k}, ints);
      out[1] = at::empty({n, k}, l.options().dtype(at::kFloat));
      out[2] = at::empty({E + 1}, ints);
      out[3] = at::empty({std::max(n * k, 1)}, ints);
      const moe_routing r{(int32_t*)out[0].data_ptr(), (float*)out[1].data_ptr(),
                          (int32_t*)out[2].data_ptr(), (int32_t*)out[3].data_ptr()};
      const size_t need = moe_route_workspace_bytes(n, E, k);
      Tensor ws;
      if (need) ws = at::empty({(int64_t)need}, l.options().dtype(at::kByte));
      s = moe_route_scored(l.data_ptr(), dtype, n, E, k, &rule, &r, need ? ws.data_ptr() : nullptr, need,
                           stream);
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    PyObject* all = PyTuple_New(4);
    if (!all) return nullptr;
    for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(all, i, THPVariable_Wrap(std::move(out[i])));
    return all;
  });
}

// (device, x, stream) -> (codes, scales)
PyObject* mx_quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, [](Args& a) -> PyObject* {
    int64_t stride;
    const Tensor& x = rows_of(a, -1, &stride);
    const int64_t rows = x.size(0), cols = x.size(1);
    if (cols < 32 || cols % 32) throw Mismatch();
    void* stream = a.stream();
    Tensor codes, scales;
    moe_status s;
    {
      const WithoutGil free;
      const auto bytes = x.options().dtype(at::kByte);
      codes = at::empty({rows, cols / 2}, bytes);
      scales = at::empty({rows, cols / 32}, bytes);
      s = moe_mx_quantize(x.data_ptr(), float_of(x), rows, (int)cols, stride, (uint8_t*)codes.data_ptr(),
                          (uint8_t*)scales.data_ptr(), stream);
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    PyObject* pair = PyTuple_New(2);
    if (!pair) return nullptr;
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(std::move(codes)));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(std::move(scales)));
    return pair;
  });
}

// (device, codes, scales, dtype, stream) -> values
PyObject* mx_dequantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, [](Args& a) -> PyObject* {
    const Tensor* codes;
    const moe_mx_matrix m = mx_of(a, 2, &codes);
    const int dtype = a.integer();
    if (dtype != MOE_F32 && dtype != MOE_BF16 && dtype != MOE_F16) throw Mismatch();
    void* stream = a.stream();
    Tensor out;
    moe_status s;
    {
      const WithoutGil free;
      out = at::empty({m.rows, m.cols}, codes->options().dtype(type_of(dtype)));
      s = moe_mx_dequantize(&m, m.rows, dtype, out.data_ptr(), stream);
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    return THPVariable_Wrap(std::move(out));
  });
}

// (device, x or its codes, None or its scales, w codes, w scales, dtype, out or None, stream) -> out
PyObject* mx_linear(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  return guarded(args, n_args, [](Args& a) -> PyObject* {
    const Tensor* x = a.peek();
    int64_t stride = 0;
    moe_mx_matrix xq{};
    if (x->scalar_type() == at::kByte) {
      xq = mx_of(a, 2, nullptr);
    } else {
      rows_of(a, -1, &stride);
      if (a.tensor()) throw Mismatch();
    }
    const moe_mx_matrix w = mx_of(a, 2, nullptr);
    if (xq.codes ? xq.cols != w.cols : x->size(1) != w.cols) throw Mismatch();
    if (x->size(0) > MOE_MAX_ROUTE_TOKENS) throw Mismatch();
    const int n = (int)x->size(0);
    const int dtype = a.integer();
    if (dtype != MOE_F32 && dtype != MOE_BF16 && dtype != MOE_F16) throw Mismatch();
    const Tensor* given = a.tensor();
    if (given && (given->scalar_type() != type_of(dtype) || given->dim() != 2 || given->size(0) != n ||
                  given->size(1) != w.rows || (w.rows > 1 && given->stride(1) != 1)))
      throw Mismatch();
    void* stream = a.stream();
    Tensor out;
    moe_status s;
    {
      const WithoutGil free;
      out = given ? *given : at::empty({n, w.rows}, x->options().dtype(type_of(dtype)));
      const int64_t step = n > 1 ? out.stride(0) : w.rows;
      if (xq.codes) {
        s = moe_mx_linear_quantized(&xq, &w, out.data_ptr(), dtype, step, stream);
      } else {
        const size_t need = moe_mx_linear_workspace_bytes(n, w.cols);
        Tensor ws;
        if (need) ws = at::empty({(int64_t)need}, x->options().dtype(at::kByte));
        s = moe_mx_linear(x->data_ptr(), float_of(*x), stride, n, &w, out.data_ptr(), dtype, step,
                          need ? ws.data_ptr() : nullptr, need, stream);
      }
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    return THPVariable_Wrap(std::move(out));
  });
}

// (device, gate codes, scales, up codes, scales, down codes, scales, top_k, x, topk_ids, topk_w,
// expert_offsets, pair_index, residual or None, out or None, stream) -> out
PyObject* mx_ffn(PyObject*, PyObject* const* args, Py_ssize_t n_args) {
  return guarded(args, n_args, [](Args& a) -> PyObject* {
    const Tensor *gate, *up, *down;
    moe_mx_layer L{};
    L.gate = mx_of(a, 3, &gate);
    L.up = mx_of(a, 3, &up);
    L.down = mx_of(a, 3, &down);
    if (gate->size(0) > MOE_MAX_EXPERTS || up->size(0) != gate->size(0) || down->size(0) != gate->size(0) ||
        L.up.rows != L.gate.rows || L.up.cols != L.gate.cols || L.down.rows != L.gate.cols ||
        L.down.cols != L.gate.rows)
      throw Mismatch();
    L.n_experts = (int32_t)gate->size(0);
    L.d_ff = L.gate.rows;
    L.d_model = L.gate.cols;
    L.top_k = a.integer();
    int64_t stride;
    const Tensor& x = rows_of(a, L.d_model, &stride);
    const int64_t n = x.size(0);
    auto routing = [&](at::ScalarType type, int64_t least) {
      const Tensor& t = a.required();
      if (t.scalar_type() != type || t.numel() < least || !t.is_contiguous()) throw Mismatch();
      return t.data_ptr();
    };
    moe_routing r;
    r.topk_ids = (int32_t*)routing(at::kInt, n * L.top_k);
    r.topk_w = (float*)routing(at::kFloat, n * L.top_k);
    r.expert_offsets = (int32_t*)routing(at::kInt, L.n_experts + 1);
    r.pair_index = (int32_t*)routing(at::kInt, n * L.top_k);
    auto stream_rows = [&]() -> const Tensor* {
      const Tensor* t = a.tensor();
      if (t && (t->scalar_type() != at::kFloat || t->dim() != 2 || t->size(0) != n ||
                t->size(1) != L.d_model || !t->is_contiguous()))
        throw Mismatch();
      return t;
    };
    const Tensor* residual = stream_rows();
    const Tensor* given = stream_rows();
    void* stream = a.stream();
    Tensor out;
    moe_status s;
    {
      const WithoutGil free;
      out = given ? *given : at::empty({n, L.d_model}, x.options().dtype(at::kFloat));
      const size_t need = moe_mx_ffn_workspace_bytes(&L, (int)n);
      Tensor ws;
      if (need) ws = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
      s = moe_mx_ffn(&L, x.data_ptr(), float_of(x), stride, (int)n, &r,
                     residual ? (const float*)residual->data_ptr() : nullptr, (float*)out.data_ptr(),
                     need ? ws.data_ptr() : nullptr, need, stream);
    }
    if (s != MOE_OK) return PyLong_FromLong(s);
    return THPVariable_Wrap(std::move(out));
  });
}

#define ENTRY(name) \
  { #name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr }
PyMethodDef methods[] = {ENTRY(qk_norm_rope), ENTRY(kv_append), ENTRY(attend), ENTRY(route_scored),
                         ENTRY(mx_quantize),  ENTRY(mx_dequantize), ENTRY(mx_linear), ENTRY(mx_ffn),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall",
                      "Short path of the calls whose kernels run for a few microseconds.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
