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

// What a thread brings into LDS in one go: a block of 32 values of x (or its codes and scale) and
// 16 bytes of weight scales. The first goes are requested before the weights, since memory
// answers in the order of the requests: the rows are then quantized while the weights arrive.
template <int DT>
struct XBlock {
  MxValues<DT> v[4];
  __device__ __forceinline__ void load(const char* row, const uint8_t*, int b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j].load(row + (b * 4 + j) * (8 * mx_type_size(DT)));
  }
  __device__ __forceinline__ void quantized(uint4& c, uint32_t& s) const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, v[j].amax());
    s = mx_scale_byte(m);
    const float f = mx_scale_float(s);
    c = s == 255u ? make_uint4(0, 0, 0, 0)
                  : make_uint4(v[0].codes(f), v[1].codes(f), v[2].codes(f), v[3].codes(f));
  }
};

template <>
struct XBlock<MOE_E4M3> {  // rows that are quantized already
  uint4 c;
  uint32_t s;
  __device__ __forceinline__ void load(const char* row, const uint8_t* scales, int b) {
    c = reinterpret_cast<const uint4*>(row)[b];
    s = scales[b];
  }
  __device__ __forceinline__ void quantized(uint4& codes, uint32_t& scale) const {
    codes = c;
    scale = s;
  }
};

// Block i of `rows` rows, row by row (padded to whole steps: blocks past K are zeros).
template <int DT>
struct Rows {
  XBlock<DT> first;
  template <class RowOf, class ScaleOf>
  __device__ __forceinline__ void read(XBlock<DT>& x, const Window& w, int rows, int i, RowOf row_of,
                                       ScaleOf scale_of) const {
    const int row = i / w.scale_bytes, b = i - row * w.scale_bytes;
    if (row < rows && b < w.K / kMxBlock) x.load(row_of(row), scale_of(row), b);
  }
  __device__ __forceinline__ void write(const XBlock<DT>& x, const Window& w, int rows, int i) const {
    const int row = i / w.scale_bytes, b = i - row * w.scale_bytes;
    if (row >= rows) return;
    uint4 c = make_uint4(0, 0, 0, 0);
    uint32_t s = 0;
    if (b < w.K / kMxBlock) x.quantized(c, s);
    *reinterpret_cast<uint4*>(w.xq + row * w.row_bytes + b * 16) = c;
    w.xs[row * w.scale_bytes + b] = (uint8_t)s;
  }
  template <class RowOf, class ScaleOf>
  __device__ __forceinline__ void request(const Window& w, int rows, RowOf row_of, ScaleOf scale_of) {
    read(first, w, rows, threadIdx.x, row_of, scale_of);
  }
  template <class RowOf, class ScaleOf>
  __device__ __forceinline__ void store(const Window& w, int rows, RowOf row_of, ScaleOf scale_of) const {
    write(first, w, rows, threadIdx.x);
    for (int i = threadIdx.x + blockDim.x; i < rows * w.scale_bytes; i += blockDim.x) {
      XBlock<DT> x;
      read(x, w, rows, i, row_of, scale_of);
      write(x, w, rows, i);
    }
  }
};

// The scales of 32 neighbouring rows of a matrix (fewer at its end) are one piece of memory
// that starts at a multiple of 32 bytes: 16-byte words, the last ones as bytes.
struct ScalePiece {
  uint4 first;
  __device__ __forceinline__ void request(const uint8_t* from, int bytes, int i) {
    if (i < bytes / 16) first = reinterpret_cast<const uint4*>(from)[i];
  }
  __device__ __forceinline__ void store(uint8_t* to, const uint8_t* from, int bytes, int i, int step) const {
    const int words = bytes / 16;
    if (i < words) reinterpret_cast<uint4*>(to)[i] = first;
    for (int j = i + step; j < words; j += step)
      reinterpret_cast<uint4*>(to)[j] = reinterpret_cast<const uint4*>(from)[j];
    for (int j = 16 * words + i; j < bytes; j += step) to[j] = from[j];
  }
};

// A barrier for LDS alone: the weights stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Codes of up to kFlight steps of MATS matrices, two tiles of 16 rows each, as a lane holds them.
// The rows' buffers start at the workgroup's first row; blocks past K read as zeros.
template <int MATS>
struct Flight {
  i32x4 c[kFlight][MATS][2];
};

constexpr int kOutside = (int)0x80000000u;

template <int MATS>
__device__ __forceinline__ void request(Flight<MATS>& f, const __amdgpu_buffer_rsrc_t (&buf)[MATS],
                                        const int (&off)[2], int nb, int s0, int chunk) {
#pragma unroll
  for (int s = 0; s < kFlight; ++s) {
    const bool in = 4 * (s0 + s) + chunk < nb;
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        f.c[s][m][t] = __builtin_amdgcn_raw_buffer_load_b128(buf[m], in ? off[t] : kOutside, 64 * (s0 + s), 0);
  }
}

// Steps s0 .. of the flight (past `send` none are left).
template <int MATS>
__device__ __forceinline__ void multiply(const Flight<MATS>& f, const Window& w, int s0, int send, int col,
                                         int chunk, int r, mx_f32x4 (&acc)[MATS][2]) {
  const int nb = w.K / kMxBlock;
#pragma unroll
  for (int s = 0; s < kFlight; ++s) {
    if (s0 + s >= send) continue;
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
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = lane & 15, chunk = lane >> 4;
  const int nb = K / kMxBlock, steps = (K + kStep - 1) / kStep;
  const int n0 = blockIdx.x * 32, t0 = blockIdx.y * kCols, rows = min(kCols, n - t0);
  const int per = (steps + kWaves - 1) / kWaves;
  const int sbeg = min(steps, wave * per), send = min(steps, sbeg + per);
  const Window w(lds, K, min(n, kCols));
  const __amdgpu_buffer_rsrc_t buf[1] = {buffer_rsrc(wq + (size_t)n0 * (K / 2), 0x80000000u)};
  const int last = N - 1 - n0;  // rows past the matrix: its last, never stored
  const int off[2] = {min(r, last) * (K / 2) + 16 * chunk, min(16 + r, last) * (K / 2) + 16 * chunk};
  auto row_of = [&](int i) {
    return DT == MOE_E4M3 ? reinterpret_cast<const char*>(xq) + (size_t)(t0 + i) * (K / 2)
                          : x + (t0 + i) * row_bytes;
  };
  auto scale_of = [&](int i) { return xs + (size_t)(t0 + i) * nb; };
  const uint8_t* scales = wsc + (size_t)n0 * nb;
  const int bytes = min(32, N - n0) * nb;
  Rows<DT> xr;
  ScalePiece sp;
  xr.request(w, rows, row_of, scale_of);
  sp.request(scales, bytes, threadIdx.x);
  Flight<1> f;
  request(f, buf, off, nb, sbeg, chunk);
  xr.store(w, rows, row_of, scale_of);
  sp.store(w.ws, scales, bytes, threadIdx.x, kThreads);
  lds_barrier();
  mx_f32x4 acc[1][2] = {};
  const int col = min(r, rows - 1);
  multiply(f, w, sbeg, send, col, chunk, r, acc);
  for (int s0 = sbeg + kFlight; s0 < send; s0 += kFlight) {
    request(f, buf, off, nb, s0, chunk);
    multiply(f, w, s0, send, col, chunk, r, acc);
  }
  // the waves' parts take the rows' place in LDS: with 16 rows of 8192 two workgroups a CU then fit
  // (28672 columns: 69 -> 47 us)
  lds_barrier();
  auto part = reinterpret_cast<float(*)[32][kCols + 1]>(lds);
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

// Grid (f / 32, pairs). A workgroup takes 16 pairs of one expert: those from its own pair on, when
// a multiple of 16 of the expert's pairs come before it; the others leave. No work list has to
// be built before the launch.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_mx_win_gateup(
    const char* __restrict__ x, int64_t row_bytes, const int32_t* __restrict__ ids, int P, int k, int d,
    int f, const uint8_t* __restrict__ gq, const uint8_t* __restrict__ gs,
    const uint8_t* __restrict__ uq, const uint8_t* __restrict__ us, int E, uint8_t* __restrict__ hq,
    uint8_t* __restrict__ hs) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ float part[kWaves][2][32][kCols + 1];
  __shared__ int s_pairs[kCols];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int r = lane & 15, chunk = lane >> 4;
  const int p = blockIdx.y;
  // every wave looks at all the ids: they are requested at once
  int id[kMxWindowPairs / kWave];
#pragma unroll
  for (int i = 0; i < kMxWindowPairs / kWave; ++i) id[i] = ids[min(kWave * i + lane, P - 1)];
  const int e = __builtin_amdgcn_readfirstlane(ids[p]);
  if ((unsigned)e >= (unsigned)E) return;
  int before = 0, rows = 0;
#pragma unroll
  for (int i = 0; i < kMxWindowPairs / kWave; ++i) {
    const int q = kWave * i + lane;
    const uint64_t same = __ballot(q < P && id[i] == e);
    const uint64_t from = __ballot(q >= p) & same;  // this pair and later ones
    before += __popcll(same & ~from);
    const int at = rows + __popcll(from & ((1ull << lane) - 1ull));
    if (wave == 0 && (from >> lane & 1) && at < kCols) s_pairs[at] = q;
    rows += __popcll(from);
  }
  if (before % kCols) return;
  rows = min(rows, kCols);
  const int nb = d / kMxBlock, steps = (d + kStep - 1) / kStep;
  const int per = (steps + kWaves - 1) / kWaves;
  const int sbeg = min(steps, wave * per), send = min(steps, sbeg + per);
  const int n0 = blockIdx.x * 32;
  const Window w(lds, d, min(P, kCols));
  const size_t first = (size_t)e * f + n0;
  const __amdgpu_buffer_rsrc_t buf[2] = {buffer_rsrc(gq + first * (d / 2), 0x80000000u),
                                         buffer_rsrc(uq + first * (d / 2), 0x80000000u)};
  const int off[2] = {r * (d / 2) + 16 * chunk, (16 + r) * (d / 2) + 16 * chunk};
  auto row_of = [&](int i) { return x + (s_pairs[i] / k) * row_bytes; };
  auto scale_of = [](int) { return (const uint8_t*)nullptr; };
  lds_barrier();  // s_pairs is written
  Rows<DT> xr;
  xr.request(w, rows, row_of, scale_of);
  // the first half of the threads brings in gate's scales, the second up's
  const int half = threadIdx.x / (kThreads / 2), i = threadIdx.x % (kThreads / 2);
  const uint8_t* scales = (half ? us : gs) + first * nb;
  ScalePiece sp;
  sp.request(scales, 32 * nb, i);
  Flight<2> fl;
  request(fl, buf, off, nb, sbeg, chunk);
  xr.store(w, rows, row_of, scale_of);
  sp.store(w.ws + half * 32 * nb, scales, 32 * nb, i, kThreads / 2);
  lds_barrier();
  mx_f32x4 acc[2][2] = {};
  const int col = min(r, rows - 1);
  multiply(fl, w, sbeg, send, col, chunk, r, acc);
  for (int s0 = sbeg + kFlight; s0 < send; s0 += kFlight) {
    request(fl, buf, off, nb, s0, chunk);
    multiply(fl, w, s0, send, col, chunk, r, acc);
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) part[wave][m][16 * t + 4 * chunk + q][r] = acc[m][t][q];
  lds_barrier();
  // half a wave holds the 32 rows of one pair: its block
#pragma unroll 1
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
    const size_t pair = s_pairs[c];
    if ((j & 7) == 0) *reinterpret_cast<uint32_t*>(hq + pair * (f / 2) + n0 / 2 + j / 2) = code;
    if (j == 0) hs[pair * (f / kMxBlock) + n0 / kMxBlock] = (uint8_t)s;
  }
}

// ---------------------------------------------------------------- down and combine

constexpr int kDownRows = 16;  // of d
constexpr int kDownParts = 2;  // of the reduction axis

// 16 rows of d of one token. An instruction multiplies one slot's rows; its columns all hold the
// slot's hidden row (a window has too few rows to fill them). The workgroups of one row tile (of
// all tokens) run on one XCD, whose L2 keeps the rows of an expert that several tokens share.
// THREADS: 4 or 8 slots at once. 8 where every workgroup has a CU of its own (d = 2048, top 10, us a
// call with 512 and 1024 threads: 1 token 16.3 and 14.8, 2 tokens 18.3 and 17.4), 4 where they
// share CUs (8 tokens 28.4 and 29.4, 16 tokens 44.3 and 46.5).
template <int THREADS>
__global__ __launch_bounds__(THREADS, 4) void k_mx_win_down(
    const int32_t* __restrict__ ids, const float* __restrict__ wt, int n, int k, int d, int f, int E,
    const uint8_t* __restrict__ dq, const uint8_t* __restrict__ ds, const uint8_t* __restrict__ hq,
    const uint8_t* __restrict__ hs, const float* residual, float* out) {
  constexpr int kDownLanes = THREADS / kWave / kDownParts;  // slots at once
  __shared__ __attribute__((aligned(16))) float part[kDownParts][MOE_MAX_TOP_K][kDownRows];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int r = lane & 15, chunk = lane >> 4;
  const int place = (int)blockIdx.x / 8;
  const int tile = (int)blockIdx.x % 8 + 8 * (place / n), t = place % n;
  const int r0 = kDownRows * tile;
  if (r0 >= d) return;  // d is a multiple of 32
  const int nb = f / kMxBlock, steps = (f + kStep - 1) / kStep;
  const int kp = wave % kDownParts;
  const int per = (steps + kDownParts - 1) / kDownParts;
  const int sbeg = min(steps, kp * per), send = min(steps, sbeg + per);
  const int first = wave / kDownParts;
  // the experts and the weights of the token's slots, one a lane, and the residual that the end
  // needs: requested together
  const int my_e = ids[(size_t)t * k + min(lane, k - 1)];
  const float slot_w = wt[(size_t)t * k + min(lane, k - 1)];
  // a pair of no expert adds nothing, whatever its weight
  const float my_w = (unsigned)my_e < (unsigned)E ? slot_w : 0.0f;
  const size_t at = (size_t)t * d + r0 + r;
  const float my_r = residual ? residual[at] : 0.0f;
  for (int j = first; j < k; j += kDownLanes) {
    const int e = __builtin_amdgcn_readlane(my_e, j);
    mx_f32x4 acc = {};
    if ((unsigned)e < (unsigned)E) {
      const size_t row = (size_t)e * d + r0 + r, p = (size_t)t * k + j;
      const uint8_t *wq = dq + row * (f / 2), *wsc = ds + row * nb;
      const uint8_t *xq = hq + p * (f / 2), *xs = hs + p * nb;
      for (int s = sbeg; s < send; ++s) {
        const int b = 4 * s + chunk, bc = min(b, nb - 1);
        const i32x4 a = *reinterpret_cast<const i32x4*>(wq + 16 * bc);
        i32x4 h = *reinterpret_cast<const i32x4*>(xq + 16 * bc);
        const int sa = b < nb ? wsc[bc] : 127, sh = b < nb ? xs[bc] : 127;
        if (b >= nb) h = i32x4{0, 0, 0, 0};  // past f
        acc = mx_mma16(a, h, acc, sa, sh);
      }
    }
    // lane r holds column r of rows 4 chunk ..
    if (r == 0) *reinterpret_cast<mx_f32x4*>(&part[kp][j][4 * chunk]) = acc;
  }
  __syncthreads();
  if (wave == 0) {
    double sum = 0.0;
    for (int j0 = 0; j0 < k; j0 += 8) {
      float y[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        y[q] = part[0][min(j0 + q, k - 1)][r];
        y[q] += part[1][min(j0 + q, k - 1)][r];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t w = __builtin_amdgcn_readlane(__float_as_uint(my_w), min(j0 + q, k - 1));
        if (j0 + q < k) sum += (double)__uint_as_float(w) * (double)y[q];
      }
    }
    if (lane < kDownRows) out[at] = (float)((double)my_r + sum);
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
                     std::max(window_lds(a.K, std::min(a.n, kCols), 1), sizeof(float) * kWaves * 32 * (kCols + 1)),
                     stream, static_cast<const char*>(a.x),
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
  const int tiles = d / kDownRows;
  const bool alone = tiles * a.n <= device_cu_count();
  auto down = alone ? k_mx_win_down<1024> : k_mx_win_down<512>;
  hipLaunchKernelGGL(down, dim3((tiles + 7) / 8 * 8 * a.n), dim3(alone ? 1024 : 512), 0, stream, a.r->topk_ids,
                     a.r->topk_w, a.n, k, d, f, L.n_experts, L.down.codes, L.down.scales, hq, hs, a.residual,
                     a.out);
  return hipGetLastError();
}

}  // namespace qmoe
