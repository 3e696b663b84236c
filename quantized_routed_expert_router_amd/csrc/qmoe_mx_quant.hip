// Rows to microscaled 4-bit floats and back.
//
//   e = floor(log2 max|x|) - 2 over a block of 32, at least -127; code = x / 2^e rounded to
//   nearest even on {0, .5, 1, 1.5, 2, 3, 4, 6} with its sign, beyond 6 to 6.
//
// Bound by memory: 2 (4) bytes read and 17/32 written a value. A quad of lanes holds a block,
// 8 consecutive values a lane: rows are read in whole 16-byte words side by side, the block's
// maximum takes two lane swaps, and the codes of a lane leave as one word.
#include "qmoe_mx_internal.h"

namespace qmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = kMxQuantUnroll;

template <int DT, bool STRIDED>
__global__ __launch_bounds__(kThreads) void k_mx_quantize(const char* __restrict__ x, int64_t words,
                                                          int row_words, int64_t row_bytes,
                                                          uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  mx_quantize_words<DT, STRIDED, kThreads>(x, words, row_words, row_bytes, codes, scales, blockIdx.x);
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_mx_dequantize(const uint32_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales,
                                                            int64_t words, char* __restrict__ out) {
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  uint32_t c[kUnroll], s[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t at = min(first + i * kThreads, words - 1);
    c[i] = codes[at];
    s[i] = scales[at >> 2];
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t at = first + i * kThreads;
    if (at >= words) break;
    const float scale = mx_scale_float(s[i]);
    typedef __attribute__((ext_vector_type(2))) float f32x2;
    f32x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 3);
    if (s[i] == 255u) {
      const float nan = __builtin_nanf("");
      v[0] = v[1] = v[2] = v[3] = f32x2{nan, nan};
    }
    if constexpr (DT == MOE_F32) {
      mx_f32x4* p = reinterpret_cast<mx_f32x4*>(out) + 2 * at;
      p[0] = mx_f32x4{v[0][0], v[0][1], v[1][0], v[1][1]};
      p[1] = mx_f32x4{v[2][0], v[2][1], v[3][0], v[3][1]};
    } else {
      uint4 r;
      if constexpr (DT == MOE_BF16) {
        mx_bf16x2 b[4];
        for (int j = 0; j < 4; ++j) b[j] = __builtin_convertvector(v[j], mx_bf16x2);
        __builtin_memcpy(&r, b, 16);
      } else {
        mx_f16x2 b[4];
        for (int j = 0; j < 4; ++j) b[j] = __builtin_convertvector(v[j], mx_f16x2);
        __builtin_memcpy(&r, b, 16);
      }
      reinterpret_cast<uint4*>(out)[at] = r;
    }
  }
}

template <int DT>
void quantize(const MxQuantArgs& a, hipStream_t stream) {
  const int64_t words = a.rows * (a.cols / 8);
  const dim3 grid((unsigned)((words + kThreads * kUnroll - 1) / (kThreads * kUnroll)));
  const char* x = static_cast<const char*>(a.x);
  uint32_t* codes = reinterpret_cast<uint32_t*>(a.codes);
  const int64_t row_bytes = a.row_stride * mx_type_size(DT);
  if (a.row_stride == a.cols || a.rows == 1)
    hipLaunchKernelGGL((k_mx_quantize<DT, false>), grid, dim3(kThreads), 0, stream, x, words,
                       a.cols / 8, row_bytes, codes, a.scales);
  else
    hipLaunchKernelGGL((k_mx_quantize<DT, true>), grid, dim3(kThreads), 0, stream, x, words,
                       a.cols / 8, row_bytes, codes, a.scales);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  if (a.dtype == MOE_BF16) quantize<MOE_BF16>(a, stream);
  else if (a.dtype == MOE_F16) quantize<MOE_F16>(a, stream);
  else quantize<MOE_F32>(a, stream);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t blocks,
                                void* out, int dtype, hipStream_t stream) {
  if (blocks == 0) return hipSuccess;
  const int64_t words = 4 * blocks;
  const dim3 grid((unsigned)((words + kThreads * kUnroll - 1) / (kThreads * kUnroll)));
  auto kern = dtype == MOE_BF16  ? k_mx_dequantize<MOE_BF16>
              : dtype == MOE_F16 ? k_mx_dequantize<MOE_F16>
                                 : k_mx_dequantize<MOE_F32>;
  hipLaunchKernelGGL(kern, grid, dim3(kThreads), 0, stream, reinterpret_cast<const uint32_t*>(codes),
                     scales, words, static_cast<char*>(out));
  return hipGetLastError();
}

}  // namespace qmoe
