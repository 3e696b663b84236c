// Internal declarations of the attention half: kernel arguments, element types and the
// masks shared by the decode and prefill attention kernels.
#pragma once

#include "qmoe_internal.h"

namespace qmoe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNegInf = -__builtin_huge_valf();

// ------------------------------------------------------------------ element types

// 16-bit activation types: 8-element vectors, the matrix-core products and the expansion of
// e4m3 codes (exact in either type).
//
// A row's probabilities are 2^(score - reference + kBias), where the reference moves to the
// row's maximum only when that exceeds it by more than kLazy: sums are rescaled seldom. The
// factor 2^kBias is in numerator and denominator alike. bf16 has the exponents of fp32 and
// needs none. fp16 ends at 2^16 and has steps of 2^-24 below 2^-14: with probabilities up to
// 2^15, and 2^11 for the reference itself, what is lost of a small one is at most 2^-36 of the
// largest (without the factor 2^-25: a tail of 40000 keys at 2^-25 each vanished).
struct Bf16 {
  typedef __bf16 T;
  typedef bf16x8 V8;
  typedef bf16x4 V4;
  typedef bf16x2 V2;
  static constexpr uint32_t kExpMask = 0x7f80u, kOne = 0x3f80u;
  static constexpr float kLazy = 8.0f, kBias = 0.0f;
#if defined(__HIP_DEVICE_COMPILE__)
  static __device__ __forceinline__ f32x4 mfma16(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(V8 a, V8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  template <bool HI>
  static __device__ __forceinline__ V2 from_e4m3(uint32_t w) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI);
  }
#endif
};

struct F16 {
  typedef _Float16 T;
  typedef f16x8 V8;
  typedef f16x4 V4;
  typedef f16x2 V2;
  static constexpr uint32_t kExpMask = 0x7c00u, kOne = 0x3c00u;
  static constexpr float kLazy = 4.0f, kBias = 11.0f;
#if defined(__HIP_DEVICE_COMPILE__)
  static __device__ __forceinline__ f32x4 mfma16(V8 a, V8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x16 mfma32(V8 a, V8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  template <bool HI>
  static __device__ __forceinline__ V2 from_e4m3(uint32_t w) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI);
  }
#endif
};

template <typename TO, typename FROM>
__device__ __forceinline__ TO bits_as(const FROM& x) {
  static_assert(sizeof(TO) == sizeof(FROM), "size");
  TO y;
  __builtin_memcpy(&y, &x, sizeof(TO));
  return y;
}

#if defined(__HIP_DEVICE_COMPILE__)
// 8 e4m3 codes (two words) as 8 elements.
template <typename A>
__device__ __forceinline__ typename A::V8 expand_e4m3(uint32_t w0, uint32_t w1) {
  const u32x4 r = {bits_as<uint32_t>(A::template from_e4m3<false>(w0)),
                   bits_as<uint32_t>(A::template from_e4m3<true>(w0)),
                   bits_as<uint32_t>(A::template from_e4m3<false>(w1)),
                   bits_as<uint32_t>(A::template from_e4m3<true>(w1))};
  return bits_as<typename A::V8>(r);
}

// Two fp32 values as e4m3 codes in the low 16 bits: nearest even, clamped to +-448, NaN
// stays NaN (the clamp's comparisons are false for it).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  a = a > 448.0f ? 448.0f : a;
  a = a < -448.0f ? -448.0f : a;
  b = b > 448.0f ? 448.0f : b;
  b = b < -448.0f ? -448.0f : b;
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xffffu;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Workgroup barrier for LDS alone: global loads in flight stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Non-finite values behind a mask. A masked probability is 0, and 0 times NaN or infinity
// is NaN, so the products of a tile that not all rows see leave such values out
// (clear_nonfinite), and what they do to the rows that see them is added from counts:
// non_finite<kind> marks a kind's values by ones, their product with the mask counts them
// per row and column, and spread() turns a count into the value itself.
template <typename A>
__device__ __forceinline__ bool clear_nonfinite(typename A::V8& v) {
  u32x4 w = bits_as<u32x4>(v);
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = (w[i] & A::kExpMask) == A::kExpMask;
    const bool hi = ((w[i] >> 16) & A::kExpMask) == A::kExpMask;
    w[i] = (lo ? 0u : (w[i] & 0xffffu)) | (hi ? 0u : (w[i] & 0xffff0000u));
    any |= lo | hi;
  }
  v = bits_as<typename A::V8>(w);
  return any;
}

// The same for e4m3 codes (NaN is their only non-finite value).
__device__ __forceinline__ bool clear_nan_codes(u32x4& w) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const bool is = (w[i] >> (8 * b) & 0x7fu) == 0x7fu;
      w[i] &= is ? ~(0xffu << (8 * b)) : 0xffffffffu;
      any |= is;
    }
  return any;
}

template <typename A, bool F8>
__device__ __forceinline__ bool clear_word(u32x4& w) {
  if constexpr (F8) return clear_nan_codes(w);
  typename A::V8 v = bits_as<typename A::V8>(w);
  const bool any = clear_nonfinite<A>(v);
  w = bits_as<u32x4>(v);
  return any;
}

// One kind of non-finite value. The fields are opaque to the compiler (made in registers it
// cannot see through), so that it keeps one small loop over the kinds instead of three
// copies of its body.
struct NonFinite {
  uint32_t pattern;  // bits of the infinity
  uint32_t nan;      // all ones for the NaN kind
  float value;
};
template <typename A>
__device__ __forceinline__ NonFinite non_finite_kind(int kind) {  // 0, 1: +-infinity, 2: NaN
  NonFinite k{A::kExpMask | (kind == 1 ? 0x8000u : 0u), kind == 2 ? 0xffffffffu : 0u,
              kind == 0 ? -kNegInf : kind == 1 ? kNegInf : __builtin_nanf("")};
  asm volatile("" : "+v"(k.pattern), "+v"(k.nan), "+v"(k.value));
  return k;
}

template <typename A>
__device__ __forceinline__ typename A::V8 non_finite(const typename A::V8& v, const NonFinite& k) {
  const u32x4 w = bits_as<u32x4>(v);
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = 0;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const uint32_t x = (w[i] >> (16 * part)) & 0xffffu;
      // the sign bit of a difference: above the infinity's exponent, or equal to the pattern
      const uint32_t is =
          ((k.nan & (A::kExpMask - (x & 0x7fffu))) | (~k.nan & ((x ^ k.pattern) - 1u))) >> 31;
      r[i] |= is * (A::kOne << (16 * part));
    }
  }
  return bits_as<typename A::V8>(r);
}

__device__ __forceinline__ float spread(float count, const NonFinite& k) {
  return count > 0.0f ? k.value : 0.0f;
}

// 8 flags (bit j) as ones and zeros.
template <typename A>
__device__ __forceinline__ typename A::V8 mask_elements(uint32_t bits) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = ((bits >> (2 * i)) & 1 ? A::kOne : 0u) | ((bits >> (2 * i + 1)) & 1 ? A::kOne << 16 : 0u);
  return bits_as<typename A::V8>(r);
}

// The sign of the score scale goes into the queries, and a zero scale into them as a whole:
// the scale itself is then positive, so that masked scores stay -inf under it and maxima
// commute with it.
struct ScaleSplit {
  float scale;
  uint32_t flip, keep;  // query words: (w ^ flip) & keep
};
__device__ __forceinline__ ScaleSplit split_scale(float scale) {
  return {scale == 0.0f ? 1.0f : __builtin_fabsf(scale), scale < 0.0f ? 0x80008000u : 0u,
          scale == 0.0f ? 0u : 0xffffffffu};
}

// What is added to a row's scaled scores for its probabilities' exponents, with m its
// reference. (Without a bias a bare negation, which costs no instruction.)
template <typename A>
__device__ __forceinline__ float exponent_base(float m) {
  const float base = A::kBias == 0.0f ? -m : A::kBias - m;
  return m == kNegInf ? 0.0f : base;
}

// 2^x for rescaling sums: never 0, so that an infinite sum stays infinite.
__device__ __forceinline__ float rescale(float x) { return fmaxf(exp2_fast(x), 1e-38f); }
#endif

// ------------------------------------------------------------------ kernel arguments

struct HeadView {
  char* data;
  long long token_stride, head_stride;  // elements
  int heads;
};

struct RowsArgs {  // norm, rotation and append
  HeadView q, k, v, q_out, k_out;
  const int32_t* positions;
  const int32_t* slots;  // append: slot of each token
  int n, dtype, D;
  moe_norm_rope p;
  const moe_kv_cache* cache;  // nullptr: k goes to k_out
  hipStream_t stream;
  int num_cus;
};

struct AttnArgs {
  HeadView q;
  int dtype;
  moe_kv_cache cache;
  moe_pages pages;
  moe_attn a;
  const int32_t* q_starts;  // prefill
  int n;                    // tokens
  int window_tokens;        // decode
  char* out;
  char* ws;
  hipStream_t stream;
};

// Split of one attention call over the key axis: `splits` workgroups per row tile, each
// writing its partial sums (fp32 [rows][head_dim], with a maximum and a sum) to the
// workspace, joined by a second kernel. splits == 1: no workspace, no second kernel.
struct AttnPlan {
  int row_tiles;  // row tiles of one kv head (decode: per sequence; prefill: upper bound)
  int splits;
  int fill;       // decode: splits of each sequence that fill the card
  int tile_rows;
  size_t partial, stats, total;  // workspace offsets and size
};

hipError_t launch_rows(const RowsArgs& a);
hipError_t launch_attn_decode(const AttnArgs& a, const AttnPlan& plan);
hipError_t launch_attn_prefill(const AttnArgs& a, const AttnPlan& plan);

// ------------------------------------------------------------------ masks and tiles

struct KeyMask {
  int window, sinks;
};

// No window is one of 2^31-1 keys: positions are below that.
inline KeyMask key_mask(const moe_attn& a) {
  return {a.window == 0 ? 0x7fffffff : a.window, a.sinks};
}

// The last key behind the window of a query at pos, negative if there is none. A position may be
// negative (it sees no key at all): it is held at 0 to keep the difference in range.
__device__ __forceinline__ int behind_window(const KeyMask& m, int pos) {
  return max(pos, 0) - m.window;
}

__device__ __forceinline__ bool key_visible(const KeyMask& m, int key, int pos) {
  return key <= pos && (key > behind_window(m, pos) || key < m.sinks);
}

// The key tiles (of TILE keys) that queries at positions first..last can see: sink tiles
// 0..ns-1, then tiles lo..hi-1.
struct TileList {
  int ns, lo, count;
  __device__ __forceinline__ int tile(int i) const { return i < ns ? i : lo + (i - ns); }
};

template <int TILE>
__device__ __forceinline__ TileList visible_tiles(const KeyMask& m, int first, int last) {
  TileList t;
  if (last < 0) {
    t.ns = t.lo = t.count = 0;
    return t;
  }
  const int hi = last / TILE + 1;
  t.lo = max(0, behind_window(m, first) + 1) / TILE;
  t.ns = min((int)(((long long)m.sinks + TILE - 1) / TILE), t.lo);
  t.count = t.ns + (hi - t.lo);
  return t;
}

// ------------------------------------------------------------------ joining splits

constexpr int kJoinThreads = 256;
constexpr int kMaxSplits = kJoinThreads;  // one statistic a thread
constexpr int kJoinCols = 64;              // columns a workgroup joins

#if defined(__HIP_DEVICE_COMPILE__)
// kJoinCols columns (from blockIdx.y on) of one output row from its `live` splits, by a
// workgroup of kJoinThreads: each split's sums are relative to its own maximum.
// row = token * q heads + q head.
template <typename A, int D>
__device__ __forceinline__ void join_row(const float* partial, const float2* stats, long long row,
                                         int splits, int live, float v_scale, char* out) {
  constexpr int LANES = kJoinCols / 4, GROUPS = kJoinThreads / LANES, WAVES = kJoinThreads / kWave;
  __shared__ float weight[kMaxSplits];
  __shared__ float red[2][WAVES];
  __shared__ f32x4 part[GROUPS][LANES];
  const int tid = threadIdx.x;
  float2 st = make_float2(kNegInf, 0.0f);
  if (tid < live) st = stats[row * splits + tid];
  float top = st.x;
#pragma unroll
  for (int s = 1; s < kWave; s *= 2) top = fmaxf(top, __shfl_xor(top, s));
  if (tid % kWave == 0) red[0][tid / kWave] = top;
  __syncthreads();
#pragma unroll
  for (int s = 0; s < WAVES; ++s) top = fmaxf(top, red[0][s]);
  const float w = rescale(st.x - (top == kNegInf ? 0.0f : top));
  if (tid < live) weight[tid] = w;
  float sum = w * st.y;
#pragma unroll
  for (int s = 1; s < kWave; s *= 2) sum += __shfl_xor(sum, s);
  if (tid % kWave == 0) red[1][tid / kWave] = sum;
  __syncthreads();
  sum = red[1][0];
#pragma unroll
  for (int s = 1; s < WAVES; ++s) sum += red[1][s];
  const int lane = tid % LANES, grp = tid / LANES;
  const int col = blockIdx.y * kJoinCols + 4 * lane;
  const float* src = partial + row * splits * D + col;
  f32x4 y = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = grp; s < live; s += GROUPS) y += weight[s] * *reinterpret_cast<const f32x4*>(src + (long long)s * D);
  part[grp][lane] = y;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int s = 1; s < GROUPS; ++s) y += part[s][lane];
    u32x2 w2;
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = sum == 0.0f ? 0.0f : y[c] / sum * v_scale;
    w2 = bits_as<u32x2>(__builtin_convertvector(y, typename A::V4));
    *reinterpret_cast<u32x2*>(out + 2 * (row * D + col)) = w2;
  }
}
#endif

}  // namespace qmoe
