// Microscaled 4-bit products of a few rows: single tokens and verify windows.
//
// Bound by the weights, read once: a workgroup takes 32 rows of a matrix and its four waves a
// quarter of the reduction axis each, every wave with the 16 bytes a lane of all its steps in
// flight before the first product. The rows to multiply (at most 16 a pass, the columns of
// the 16x16x128 instruction) are quantized by the workgroup itself while the weights arrive:
// one more launch would cost more than the window's few blocks.
//
//   k_mx_win_linear  y = Q(x) W^T
//   k_mx_win_gateup  per (expert, 32 rows of f): gate and up, h = silu(g) u in binary64, and
//                    its 4-bit block, which the 32 rows hold whole
//   k_mx_win_down    per (token, 16 rows of d): the k experts' down products, the
//                    routing-weighted sum in binary64 in slot order, the residual
#include "qmoe_mx_internal.h"

namespace qmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kCols = 16;   // rows of x a pass
constexpr int kStep = 128;  // values of the reduction axis an instruction takes
constexpr int kFlight = 4;  // steps a wave requests at once

// LDS of the rows to multiply: codes of 16 rows, padded to whole steps and by 16 bytes (so
// that the rows' words lie in different banks), and their scales.
__host__ __device__ inline int x_row_bytes(int K) { return (K + kStep - 1) / kStep * (kStep / 2) + 16; }
__host__ __device__ inline int x_scale_bytes(int K) { return (K + kStep - 1) / kStep * 4; }
__host__ __device__ inline size_t window_lds(int K, int cols, int mats) {
  return (size_t)cols * (x_row_bytes(K) + x_scale_bytes(K)) + (size_t)mats * 32 * (K / kMxBlock) + 16;
}

struct Window {
  char* xq;       // [cols][x_row_bytes]
  uint8_t* xs;    // [cols][x_scale_bytes]
  uint8_t* ws;    // [mats][32][K / 32]
  int K, row_bytes, scale_bytes;
  __device__ __forceinline__ Window(char* lds, int K_, int cols) : K(K_) {
    row_bytes = x_row_bytes(K);
    scale_bytes = x_scale_bytes(K);
    xq = lds;
    xs = reinterpret_cast<uint8_t*>(lds + cols * row_bytes);
    const size_t o = (size_t)cols * (row_bytes + scale_bytes);
    ws = reinterpret_cast<uint8_t*>(lds + ((o + 15) & ~(size_t)15));
  }
};

// Quantizes `rows` rows of x into LDS, a block of 32 a thread; blocks past K are zeros.
template <int DT, class RowOf>
__device__ __forceinline__ void stage_rows(const Window& w, int rows, RowOf row_of) {
  const int nb = w.K / kMxBlock, padded = w.scale_bytes;
  for (int i = threadIdx.x; i < rows * padded; i += blockDim.x) {
    const int row = i / padded, b = i - row * padded;
    uint4 c = make_uint4(0, 0, 0, 0);
    uint32_t s = 0;
    if (b < nb) {
      const char* p = row_of(row) + (size_t)b * (kMxBlock * mx_type_size(DT));
      MxValues<DT> v[4];
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j].load(p + j * 8 * mx_type_size(DT));
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max(m, v[j].amax());
      s = mx_scale_byte(m);
      if (s != 255u) {
        const float f = mx_scale_float(s);
        c = make_uint4(v[0].codes(f), v[1].codes(f), v[2].codes(f), v[3].codes(f));
      }
    }
    *reinterpret_cast<uint4*>(w.xq + row * w.row_bytes + b * 16) = c;
    w.xs[row * w.scale_bytes + b] = (uint8_t)s;
  }
}

// The same for rows that are quantized already.
template <class RowOf, class ScaleOf>
__device__ __forceinline__ void stage_quantized(const Window& w, int rows, RowOf row_of,
                                                ScaleOf scale_of) {
  const int nb = w.K / kMxBlock, padded = w.scale_bytes;
  for (int i = threadIdx.x; i < rows * padded; i += blockDim.x) {
    const int row = i / padded, b = i - row * padded;
    uint4 c = make_uint4(0, 0, 0, 0);
    uint32_t s = 0;
    if (b < nb) {
      c = *reinterpret_cast<const uint4*>(row_of(row) + 16 * b);
      s = scale_of(row)[b];
    }
    *reinterpret_cast<uint4*>(w.xq + row * w.row_bytes + b * 16) = c;
    w.xs[row * w.scale_bytes + b] = (uint8_t)s;
  }
}

// The scales of 32 neighbouring rows of a matrix (fewer at its end) are one piece of memory
// that starts at a multiple of 32 bytes; copied in words of 16 bytes, the last ones as bytes.
__device__ __forceinline__ void stage_scales(uint8_t* to, const uint8_t* from, int bytes) {
  const int words = bytes / 16;
  for (int i = threadIdx.x; i < words; i += blockDim.x)
    reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(from)[i];
  for (int i = 16 * words + threadIdx.x; i < bytes; i += blockDim.x) to[i] = from[i];
}

// Codes of up to kFlight steps of MATS matrices, two tiles of 16 rows each, as a lane holds them.
template <int MATS>
struct Flight {
  i32x4 c[kFlight][MATS][2];
};

// Requests the codes of steps s0 .. (clamped to valid blocks: the x codes past K are zeros, and
// scales past K are taken as 1, so what is read twice there adds zeros).
template <int MATS>
__device__ __forceinline__ void request(Flight<MATS>& f, const uint8_t* const (&base)[MATS][2], int nb,
                                        int s0, int chunk) {
#pragma unroll
  for (int s = 0; s < kFlight; ++s) {
    const int b = min(4 * (s0 + s) + chunk, nb - 1);
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        f.c[s][m][t] = *reinterpret_cast<const i32x4*>(base[m][t] + 16 * (size_t)b);
  }
}

template <int MATS>
__device__ __forceinline__ void multiply(const Flight<MATS>& f, const Window& w, int s0, int send, int col,
                                         int chunk, int r, mx_f32x4 (&acc)[MATS][2]) {
  const int nb = w.K / kMxBlock;
#pragma unroll
  for (int s = 0; s < kFlight; ++s) {
    if (s0 + s >= send) break;
    const int b = 4 * (s0 + s) + chunk;
    const i32x4 x = *reinterpret_cast<const i32x4*>(w.xq + col * w.row_bytes + 16 * b);
    const int xs = w.xs[col * w.scale_bytes + b];
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int ws = b < nb ? w.ws[(m * 32 + 16 * t + r) * nb + b] : 127;
        acc[m][t] = mx_mma16(f.c[s][m][t], x, acc[m][t], ws, xs);
      }
  }
}

// ---------------------------------------------------------------- linear

template <int DT>
struct OutType;
template <>
struct OutType<MOE_F32> {
  typedef float type;
};
template <>
struct OutType<MOE_BF16> {
  typedef __bf16 type;
};
template <>
struct OutType<MOE_F16> {
  typedef _Float16 type;
};

// DT: the type of x, or MOE_E4M3 where x is quantized already (xq, xs).
template <int DT>
__global__ __launch_bounds__(kThreads) void k_mx_win_linear(const char* __restrict__ x, int64_t row_bytes,
                                                            const uint8_t* __restrict__ xq,
                                                            const uint8_t* __restrict__ xs, int n, int N,
                                                            int K, const uint8_t* __restrict__ wq,
                                                            const uint8_t* __restrict__ wsc,
                                                            void* __restrict__ out, int out_dtype,
                                                            int64_t out_stride) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ float part[kWaves][32][kCols + 1];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = lane & 15, chunk = lane >> 4;
  const int nb = K / kMxBlock, steps = (K + kStep - 1) / kStep;
  const int n0 = blockIdx.x * 32, t0 = blockIdx.y * kCols, rows = min(kCols, n - t0);
  const int per = (steps + kWaves - 1) / kWaves;
  const int sbeg = min(steps, wave * per), send = min(steps, sbeg + per);
  const Window w(lds, K, min(n, kCols));
  const uint8_t* base[1][2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
    base[0][t] = wq + (size_t)min(n0 + 16 * t + r, N - 1) * (K / 2);
  Flight<1> f;
  request(f, base, nb, sbeg, chunk);
  stage_scales(w.ws, wsc + (size_t)n0 * nb, min(32, N - n0) * nb);
  if constexpr (DT == MOE_E4M3)
    stage_quantized(w, rows, [&](int i) { return xq + (size_t)(t0 + i) * (K / 2); },
                    [&](int i) { return xs + (size_t)(t0 + i) * nb; });
  else
    stage_rows<DT>(w, rows, [&](int i) { return x + (t0 + i) * row_bytes; });
  __syncthreads();
  mx_f32x4 acc[1][2] = {};
  const int col = min(r, rows - 1);
  for (int s0 = sbeg; s0 < send; s0 += kFlight) {
    if (s0 > sbeg) request(f, base, nb, s0, chunk);
    multiply(f, w, s0, send, col, chunk, r, acc);
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][16 * t + 4 * chunk + i][r] = acc[0][t][i];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * rows; i += kThreads) {
    const int c = i / 32, j = i & 31;
    if (n0 + j >= N) continue;
    float v = part[0][j][c];
#pragma unroll
    for (int q = 1; q < kWaves; ++q) v += part[q][j][c];
    const int64_t at = (t0 + c) * out_stride + n0 + j;
    if (out_dtype == MOE_F32) static_cast<float*>(out)[at] = v;
    else if (out_dtype == MOE_BF16) static_cast<__bf16*>(out)[at] = (__bf16)v;
    else static_cast<_Float16*>(out)[at] = (_Float16)v;
  }
}

// ---------------------------------------------------------------- gate and up

// Grid (f / 32, pairs). The workgroups of an expert's first pair take all of its pairs (16 a
// pass); the others leave. No work list has to be built before the launch.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_mx_win_gateup(
    const char* __restrict__ x, int64_t row_bytes, const int32_t* __restrict__ ids, int P, int k, int d,
    int f, const uint8_t* __restrict__ gq, const uint8_t* __restrict__ gs,
    const uint8_t* __restrict__ uq, const uint8_t* __restrict__ us, int E, uint8_t* __restrict__ hq,
    uint8_t* __restrict__ hs) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ float part[kWaves][2][32][kCols + 1];
  __shared__ int s_pairs[kMxWindowPairs];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = lane & 15, chunk = lane >> 4;
  const int p = blockIdx.y;
  const int e = ids[p];
  if ((unsigned)e >= (unsigned)E) return;
  int count = 0;
  for (int q0 = 0; q0 < P; q0 += kWave) {
    const bool mine = q0 + lane < P && ids[min(q0 + lane, P - 1)] == e;
    const uint64_t b = __ballot(mine);
    if (q0 <= p && (b & (q0 + kWave <= p ? ~0ull : (1ull << (p - q0)) - 1ull))) return;
    if (wave == 0 && mine) s_pairs[count + __popcll(b & ((1ull << lane) - 1ull))] = q0 + lane;
    count += __popcll(b);
  }
  const int nb = d / kMxBlock, steps = (d + kStep - 1) / kStep;
  const int per = (steps + kWaves - 1) / kWaves;
  const int sbeg = min(steps, wave * per), send = min(steps, sbeg + per);
  const int n0 = blockIdx.x * 32;
  const Window w(lds, d, min(P, kCols));
  const uint8_t* base[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const size_t row = (size_t)e * f + n0 + 16 * t + r;
    base[0][t] = gq + row * (d / 2);
    base[1][t] = uq + row * (d / 2);
  }
  Flight<2> fl;
  request(fl, base, nb, sbeg, chunk);
  stage_scales(w.ws, gs + ((size_t)e * f + n0) * nb, 32 * nb);
  stage_scales(w.ws + 32 * nb, us + ((size_t)e * f + n0) * nb, 32 * nb);
  for (int c0 = 0; c0 < count; c0 += kCols) {
    __syncthreads();  // s_pairs is written; the last pass has read its rows and sums
    const int rows = min(kCols, count - c0);
    stage_rows<DT>(w, rows, [&](int i) { return x + (s_pairs[c0 + i] / k) * row_bytes; });
    __syncthreads();
    mx_f32x4 acc[2][2] = {};
    const int col = min(r, rows - 1);
    for (int s0 = sbeg; s0 < send; s0 += kFlight) {
      if (s0 > sbeg || c0 > 0) request(fl, base, nb, s0, chunk);
      multiply(fl, w, s0, send, col, chunk, r, acc);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][m][16 * t + 4 * chunk + i][r] = acc[m][t][i];
    __syncthreads();
    // half a wave holds the 32 rows of one pair: its block
    for (int c = threadIdx.x / 32; c < rows; c += kThreads / 32) {
      const int j = threadIdx.x & 31;
      float g = part[0][0][j][c], u = part[0][1][j][c];
#pragma unroll
      for (int q = 1; q < kWaves; ++q) {
        g += part[q][0][j][c];
        u += part[q][1][j][c];
      }
      const double h = mx_silu_up64(g, u);
      double m = fabs(h);
      bool bad = !(m < __builtin_inf());
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        m = fmax(m, __shfl_xor(m, o));
        bad |= __shfl_xor((int)bad, o) != 0;
      }
      const uint32_t s = bad ? 255u : mx_scale_byte64(m);
      uint32_t code = bad ? 0u : mx_code64(h, s);
      code |= (uint32_t)__shfl_xor((int)code, 1) << 4;  // even lanes: their pair's byte
      code |= (uint32_t)__shfl_xor((int)code, 2) << 8;
      code |= (uint32_t)__shfl_xor((int)code, 4) << 16;
      const size_t pair = s_pairs[c0 + c];
      if ((j & 7) == 0)
        *reinterpret_cast<uint32_t*>(hq + pair * (f / 2) + n0 / 2 + j / 2) = code;
      if (j == 0) hs[pair * (f / kMxBlock) + n0 / kMxBlock] = (uint8_t)s;
    }
  }
}

// ---------------------------------------------------------------- down and combine

constexpr int kDownThreads = 512;
constexpr int kDownParts = 2;                                       // of the reduction axis
constexpr int kDownSlots = kDownThreads / kWave / kDownParts;       // slots at once

// The workgroups of one row tile (of all tokens) run on one XCD, whose L2 keeps the rows of an
// expert that several tokens of the window share.
__global__ __launch_bounds__(kDownThreads) void k_mx_win_down(
    const int32_t* __restrict__ ids, const float* __restrict__ wt, int n, int k, int d, int f, int E,
    const uint8_t* __restrict__ dq, const uint8_t* __restrict__ ds, const uint8_t* __restrict__ hq,
    const uint8_t* __restrict__ hs, const float* residual, float* out) {
  __shared__ float part[kDownParts][MOE_MAX_TOP_K][16];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = lane & 15, chunk = lane >> 4;
  const int slot = (int)blockIdx.x / 8;
  const int tile = (int)blockIdx.x % 8 + 8 * (slot / n), t = slot % n;
  const int r0 = 16 * tile;
  if (r0 >= d) return;
  const int nb = f / kMxBlock, steps = (f + kStep - 1) / kStep;
  const int kp = wave % kDownParts;
  const int per = (steps + kDownParts - 1) / kDownParts;
  const int sbeg = min(steps, kp * per), send = min(steps, sbeg + per);
  for (int j = wave / kDownParts; j < k; j += kDownSlots) {
    const size_t p = (size_t)t * k + j;
    const int e = ids[p];
    mx_f32x4 acc = {};
    if ((unsigned)e < (unsigned)E) {
      const size_t row = (size_t)e * d + r0 + r;  // d is a multiple of 32
      const uint8_t* wq = dq + row * (f / 2);
      const uint8_t* wsc = ds + row * nb;
      const uint8_t* xq = hq + p * (f / 2);
      const uint8_t* xs = hs + p * nb;
      for (int s = sbeg; s < send; ++s) {
        const int b = 4 * s + chunk, bc = min(b, nb - 1);
        const i32x4 a = *reinterpret_cast<const i32x4*>(wq + 16 * (size_t)bc);
        i32x4 h = *reinterpret_cast<const i32x4*>(xq + 16 * (size_t)bc);
        const int sa = b < nb ? wsc[bc] : 127, sh = b < nb ? xs[bc] : 127;
        if (b >= nb) h = i32x4{0, 0, 0, 0};
        acc = mx_mma16(a, h, acc, sa, sh);
      }
    }
    // every column holds the same sums
    if (r == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[kp][j][4 * chunk + i] = acc[i];
  }
  __syncthreads();
  if (threadIdx.x < 16) {
    const int i = threadIdx.x;
    double sum = 0.0;
    for (int j = 0; j < k; ++j) {
      float y = part[0][j][i];
#pragma unroll
      for (int q = 1; q < kDownParts; ++q) y += part[q][j][i];
      sum += (double)wt[(size_t)t * k + j] * (double)y;
    }
    const size_t at = (size_t)t * d + r0 + i;
    out[at] = (float)((residual ? (double)residual[at] : 0.0) + sum);
  }
}

}  // namespace

hipError_t launch_mx_linear_window(const MxLinearArgs& a, hipStream_t stream) {
  const int es = a.x ? mx_type_size(a.dtype) : 0;
  auto kern = !a.x                    ? k_mx_win_linear<MOE_E4M3>
              : a.dtype == MOE_BF16   ? k_mx_win_linear<MOE_BF16>
              : a.dtype == MOE_F16    ? k_mx_win_linear<MOE_F16>
                                      : k_mx_win_linear<MOE_F32>;
  hipLaunchKernelGGL(kern, dim3((a.N + 31) / 32, (a.n + kCols - 1) / kCols), dim3(kThreads),
                     window_lds(a.K, std::min(a.n, kCols), 1), stream, static_cast<const char*>(a.x),
                     a.row_stride * es, a.xq, a.xs, a.n, a.N, a.K, a.w, a.ws, a.out, a.out_dtype,
                     a.out_stride);
  return hipGetLastError();
}

hipError_t launch_mx_ffn_window(const MxFfnArgs& a, hipStream_t stream) {
  const moe_mx_layer& L = *a.L;
  const int d = L.d_model, f = L.d_ff, k = L.top_k, P = a.n * k;
  const MxFfnWs W = mx_ffn_ws(a.n, k, d, f, L.n_experts);
  uint8_t* hq = reinterpret_cast<uint8_t*>(a.work + W.hq);
  uint8_t* hs = reinterpret_cast<uint8_t*>(a.work + W.hs);
  auto kern = a.dtype == MOE_BF16  ? k_mx_win_gateup<MOE_BF16>
              : a.dtype == MOE_F16 ? k_mx_win_gateup<MOE_F16>
                                   : k_mx_win_gateup<MOE_F32>;
  hipLaunchKernelGGL(kern, dim3(f / 32, P), dim3(kThreads), window_lds(d, std::min(P, kCols), 2),
                     stream, static_cast<const char*>(a.x), a.row_stride * mx_type_size(a.dtype),
                     a.r->topk_ids, P, k, d, f, L.gate.codes, L.gate.scales, L.up.codes, L.up.scales,
                     L.n_experts, hq, hs);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int tiles = (d + 15) / 16;
  hipLaunchKernelGGL(k_mx_win_down, dim3((tiles + 7) / 8 * 8 * a.n), dim3(kDownThreads), 0, stream,
                     a.r->topk_ids, a.r->topk_w, a.n, k, d, f, L.n_experts, L.down.codes, L.down.scales,
                     hq, hs, a.residual, a.out);
  return hipGetLastError();
}

}  // namespace qmoe
