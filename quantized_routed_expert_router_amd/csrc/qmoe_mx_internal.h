// Microscaled 4-bit floats: device helpers and launchers shared by their translation units.
//
// A block of 32 values along the reduction axis holds 32 e2m1 codes (sign, two exponent
// bits, one fraction bit: 0, .5, 1, 1.5, 2, 3, 4, 6) and one e8m0 scale, a power of two.
// Even columns sit in the low half of a byte, so one lane's 16 bytes are the 32 codes of a
// block, which is what the scaled matrix instructions of gfx950 take per lane, with that
// block's scale in a byte of a register.
#pragma once

#include <cmath>

#include "qmoe_internal.h"

namespace qmoe {

constexpr int kMxBlock = 32;

typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(4))) float mx_f32x4;
typedef __attribute__((ext_vector_type(16))) float mx_f32x16;
typedef __attribute__((ext_vector_type(2))) __bf16 mx_bf16x2;
typedef __attribute__((ext_vector_type(2))) _Float16 mx_f16x2;

// The 128 bits of a lane's codes as the instruction's operand (its upper half is not read in
// the 4-bit formats).
__device__ __forceinline__ i32x8 mx_operand(i32x4 v) {
  return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

// c += a . b of 32 rows by 32 columns over 64 values: lane l holds row (column) l % 32 and the
// block l / 32; byte OP of each scale register. Products and sums of codes under scales within
// about 2^10 of each other are exact in fp32.
template <int OP>
__device__ __forceinline__ mx_f32x16 mx_mma32(i32x4 a, i32x4 b, mx_f32x16 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, OP,
                                                         sa, OP, sb);
}

// The same of 16 rows by 16 columns over 128 values: row l % 16, block l / 16, byte 0.
__device__ __forceinline__ mx_f32x4 mx_mma16(i32x4 a, i32x4 b, mx_f32x4 c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, 0,
                                                          sa, 0, sb);
}

// Scale byte of a block whose largest magnitude has the fp32 bits `amax`: the exponent of its
// leading bit less 2 (the exponent of 4, the largest power of two that e2m1 has), not below
// 2^-127; 255 (NaN) where the block holds an infinity or a NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const int field = (int)(amax >> 23);
  return field == 255 ? 255u : (uint32_t)max(field - 2, 0);
}

// The conversion instructions divide by the power of two in the exponent bits of their scale
// operand (0 there stands for 2^-127) and round to nearest even, magnitudes beyond 6 to 6.
__device__ __forceinline__ float mx_scale_float(uint32_t byte) { return __uint_as_float(byte << 23); }

// 8 consecutive values of a row as loaded, their largest magnitude, and their codes.
template <int DT>
struct MxValues;

template <>
struct MxValues<MOE_F32> {
  float v[8];
  __device__ __forceinline__ void load(const void* p) {
    const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
  }
};

// Largest of the 8 magnitudes (16-bit patterns without sign, two a word) of 4 words.
__device__ __forceinline__ uint32_t mx_amax16(const uint32_t (&w)[4]) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7fff7fffu;
    u16x2 p;
    __builtin_memcpy(&p, &a, 4);
    m = __builtin_elementwise_max(m, p);
  }
  return max((uint32_t)m[0], (uint32_t)m[1]);
}

template <>
struct MxValues<MOE_BF16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void* p) {
    const uint4 a = *static_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  __device__ __forceinline__ uint32_t amax() const { return mx_amax16(w) << 16; }
  __device__ __forceinline__ mx_bf16x2 pair(int i) const {
    mx_bf16x2 p;
    __builtin_memcpy(&p, &w[i], 4);
    return p;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, pair(0), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, pair(1), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, pair(2), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, pair(3), s, 3);
  }
};

template <>
struct MxValues<MOE_F16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const void* p) {
    const uint4 a = *static_cast<const uint4*>(p);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  __device__ __forceinline__ uint32_t amax() const {
    return __float_as_uint(half_bits_to_float(mx_amax16(w)));
  }
  __device__ __forceinline__ mx_f16x2 pair(int i) const {
    mx_f16x2 p;
    __builtin_memcpy(&p, &w[i], 4);
    return p;
  }
  __device__ __forceinline__ uint32_t codes(float s) const {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, pair(0), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, pair(1), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, pair(2), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, pair(3), s, 3);
  }
};

__host__ __device__ constexpr int mx_type_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// Maximum over the 4 lanes of a quad (one block of 32 values is held by a quad).
__device__ __forceinline__ uint32_t mx_quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
}

// Codes and scales of a workgroup's share of rows: a quad of lanes holds a block, a lane 8
// consecutive values (a word of codes). The loads of a thread's words are in flight at once.
constexpr int kMxQuantUnroll = 4;

template <int DT, bool STRIDED, int THREADS>
__device__ __forceinline__ void mx_quantize_words(const char* __restrict__ x, int64_t words, int row_words,
                                                  int64_t row_bytes, uint32_t* __restrict__ codes,
                                                  uint8_t* __restrict__ scales, int64_t block) {
  const int64_t first = block * (THREADS * kMxQuantUnroll) + threadIdx.x;
  MxValues<DT> v[kMxQuantUnroll];
#pragma unroll
  for (int i = 0; i < kMxQuantUnroll; ++i) {
    // words is a multiple of 4, so the lanes of a quad are inside or outside together
    const int64_t at = min(first + i * THREADS, words - 4 + (threadIdx.x & 3));
    if (STRIDED) {
      const int64_t row = at / row_words;
      v[i].load(x + row * row_bytes + (at - row * row_words) * (8 * mx_type_size(DT)));
    } else {
      v[i].load(x + at * (8 * mx_type_size(DT)));
    }
  }
#pragma unroll
  for (int i = 0; i < kMxQuantUnroll; ++i) {
    const int64_t at = first + i * THREADS;
    const uint32_t s = mx_scale_byte(mx_quad_max(v[i].amax()));
    // a block with an infinity or a NaN is NaN as a whole: its codes are zeros
    const uint32_t c = s == 255u ? 0u : v[i].codes(mx_scale_float(s));
    if (at < words) {
      codes[at] = c;
      if ((threadIdx.x & 3) == 0) scales[at >> 2] = (uint8_t)s;
    }
  }
}

// ---- the hidden vector's codes are those of its 64-bit value
//
// A 4-bit step is a quarter to a half of the value, so a last-bit difference in h next to a
// border would move an output by a hundredth. Every path takes the code of
// h = g / (1 + e^-g) * u in binary64 (g, u the fp32 sums).

__device__ __forceinline__ double mx_silu_up64(float g, float u) {
  return (double)g / (1.0 + exp(-(double)g)) * (double)u;
}

// Scale byte for a largest magnitude in binary64 (255 for infinity and NaN).
__device__ __forceinline__ uint32_t mx_scale_byte64(double amax) {
  const int field = (int)((uint64_t)__double_as_longlong(amax) >> 52) & 0x7ff;
  if (field == 0x7ff) return 255u;
  return (uint32_t)min(max(field - 1023 - 2 + 127, 0), 254);
}

// e2m1 code of a finite v / 2^(byte - 127), ties to the even code.
__device__ __forceinline__ uint32_t mx_code64(double v, uint32_t byte) {
  // 2^(127 - byte) as its bits: exact, and the product too (a power of two far from the ends)
  const double y = fabs(v) * __longlong_as_double((int64_t)(1023 + 127 - (int)byte) << 52);
  const uint32_t c = (y > 0.25) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) +
                     (y > 5.0);
  return c | (uint32_t)((uint64_t)__double_as_longlong(v) >> 63) << 3;
}

// ---------------------------------------------------------------- host side

struct MxQuantArgs {
  const void* x;
  int dtype;
  int64_t rows, row_stride;  // stride in elements
  int cols;
  uint8_t* codes;
  uint8_t* scales;
};

struct MxLinearArgs {
  const void* x;  // rows to quantize, or null: xq, xs hold them
  int dtype;
  int64_t row_stride;
  const uint8_t* xq;
  const uint8_t* xs;
  int n, N, K;
  const uint8_t* w;
  const uint8_t* ws;
  void* out;
  int out_dtype;
  int64_t out_stride;
  char* work;
};

struct MxFfnArgs {
  const moe_mx_layer* L;
  const void* x;
  int dtype, n;
  int64_t row_stride;
  const moe_routing* r;
  const float* residual;  // may be null
  float* out;
  char* work;
};

// Up to 16 tokens and 256 pairs the expert FFN runs on the window kernels (one workgroup per
// touched expert and 32 rows), above on the grouped products, which take two launches and some
// 13 us more but read an expert's down weights once for all its tokens. The window reads them
// for each pair, at about 3 TB/s where an expert comes again: it is left where these readings,
// with experts drawn evenly, are more than 40 MB. Measured, us, window and grouped: 512 experts of
// 768 x 2048, top 10, 16 tokens 83 and 94; 64 of 1024 x 2048, top 8, 8 tokens 45 and 48, 10 tokens
// 55 and 51; 8 of 4096 x 4096, top 2, 4 tokens 43 and 53, 6 tokens 65 and 56, 16 tokens 119 and 60.
constexpr int kMxWindowTokens = 16;
constexpr int kMxWindowPairs = 256;

inline bool mx_window(int n, int k, int d, int f, int E) {
  const int P = n * k;
  if (n > kMxWindowTokens || P > kMxWindowPairs) return false;
  const double again = P - E * (1.0 - std::pow(1.0 - 1.0 / E, P));
  return again * d * (f / 2 + f / kMxBlock) <= 40e6;
}

// Whether a linear product runs on the window kernel: the rows to multiply are then quantized in
// LDS (up to 70 KB at 16 rows of 8192) and need no workspace, which the query must know from
// the rows and columns alone. Weights with fewer than 16 scales in all run there too: the tiles
// fetch 16 at once. Columns past 8192 leave the window whatever the rows are, a limit that was not
// measured from both sides: 4 rows by 8192 columns and 7168 outputs take 10.8 us here, 4 rows by
// 18432 columns and 7168 outputs 4.8 + 36.8 us on the tiles (70 MB of weights at 1.9 TB/s).
inline bool mx_linear_window(int n, int N, int K) {
  return (n <= kMxWindowTokens && K <= 8192) || (int64_t)N * (K / kMxBlock) < 16;
}

// Workspace of a linear product: the same for every N, which the query is not told.
inline size_t mx_linear_ws(int n, int K) {
  if (n == 0 || (n <= kMxWindowTokens && K <= 8192)) return 0;
  return align256((size_t)n * (K / 2)) + align256((size_t)n * (K / kMxBlock));
}

// Pairs of one expert that a workgroup of the grouped product takes.
constexpr int kMxBM = 128;

inline int mx_max_mtiles(int P, int E) {
  const long long busy = std::min<long long>(E, P);
  return (int)(((long long)P + busy * (kMxBM - 1)) / kMxBM);
}

// ---- the split of the grouped products' tile list over the XCDs (used by the kernel that writes
// the list and by the host that sizes the grid)

constexpr int kMxXcds = 8;

// Cost of `count` tiles with `rows` rows of x: 4 a tile for its weights and 1 for each 32 rows
// of x. By loads alone it would be 8 to 1, by products 0; between them, since neither hides the
// other wholly.
constexpr int kMxTileCost = 4;
__host__ __device__ constexpr int mx_tiles_cost(int count, int rows) {
  return kMxTileCost * count + (rows + 31) / 32;
}

// XCD x starts at the first tile whose cost before it is x / 8 of the whole or more. Tile j, with
// the cost `before` it and `next` with it, finds the starts that are it or the tile behind it.
__host__ __device__ inline void mx_xcd_starts(int j, int before, int next, int total, int* first) {
#pragma unroll
  for (int x = 0; x < kMxXcds; ++x) {
    const long long at = (long long)x * total;
    if (at == (long long)before * kMxXcds) first[x] = j;
    else if (at > (long long)before * kMxXcds && at < (long long)next * kMxXcds) first[x] = j + 1;
  }
}

// Workgroups that cover the tiles of any XCD, `ntn` a tile: an XCD's share of the cost is at most
// an eighth of the whole and one tile, a tile costs kMxTileCost + 1 to kMxTileCost + 4.
inline int mx_list_grid(int max_mt, int ntn) {
  const int most = ((kMxTileCost + 4) * ((max_mt + kMxXcds - 1) / kMxXcds + 1)) / (kMxTileCost + 1) + 2;
  return kMxXcds * std::min(max_mt, most) * ntn;
}

struct MxFfnWs {
  size_t tiles;   // int4 [max M-tiles] (expert, first grouped pair, pairs, 0)
  size_t xcd_first;  // int [9] first tile of each XCD, and their number
  size_t place;   // int [P] grouped place of each pair
  size_t xq, xs;  // codes and scales of x [n]
  size_t hq, hs;  // codes and scales of the hidden rows [P]
  size_t y;       // fp32 [P][d], grouped pairs
  size_t total;
};

inline MxFfnWs mx_ffn_ws(int n, int k, int d, int f, int E) {
  MxFfnWs W{};
  size_t o = 0;
  const size_t P = (size_t)n * k;
  const bool window = mx_window(n, k, d, f, E);
  W.tiles = o;
  if (!window) o = align256(o + 16 * (size_t)(mx_max_mtiles((int)P, E) + 1));
  W.xcd_first = o;
  if (!window) o = align256(o + 64);
  W.place = o;
  if (!window) o = align256(o + 4 * P);
  W.xq = o;
  if (!window) o = align256(o + (size_t)n * (d / 2));
  W.xs = o;
  if (!window) o = align256(o + (size_t)n * (d / kMxBlock));
  W.hq = o;
  o = align256(o + P * (f / 2));
  W.hs = o;
  o = align256(o + P * (f / kMxBlock));
  W.y = o;
  if (!window) o = align256(o + 4 * P * d);
  W.total = o;
  return W;
}

hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t blocks,
                                void* out, int dtype, hipStream_t stream);
hipError_t launch_mx_linear(const MxLinearArgs& a, hipStream_t stream);
hipError_t launch_mx_ffn(const MxFfnArgs& a, hipStream_t stream);
hipError_t launch_mx_ffn_window(const MxFfnArgs& a, hipStream_t stream);
hipError_t launch_mx_linear_window(const MxLinearArgs& a, hipStream_t stream);

}  // namespace qmoe
