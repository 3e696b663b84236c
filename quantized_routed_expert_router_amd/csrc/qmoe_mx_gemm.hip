// Microscaled 4-bit matrix products of many rows: y = Q(x) W^T, and the routed experts'
// products of a batch or a prefill chunk.
//
//   k_mx_tiles    M-tile work list of the grouped product (expert, first grouped pair, pairs)
//   k_mx_gemm     one workgroup per tile of the product; as the gate and up products it ends
//                 in h = silu(g) u and its 4-bit blocks, as the down product in fp32 rows
//   k_mx_combine  out[t] = residual[t] + sum_j w[t][j] y[t k + j], slot order, binary64 sum
#include "qmoe_mx_internal.h"

namespace qmoe {
namespace {

typedef __attribute__((address_space(3))) void* lptr_t;
typedef const __attribute__((address_space(1))) void* gptr_t;

constexpr int kThreads = 256;
constexpr int kStepBytes = 64;  // codes of a row in one stage: 128 values, 4 blocks

// Blocks past the end of the reduction axis are read from here: codes of 0 under scale 1.
__device__ __align__(16) const uint8_t mx_zero_block[16] = {};
__device__ const uint8_t mx_unit_scale[4] = {127, 127, 127, 127};

enum Mode { kLinear, kGateUp, kDown };

struct GemmArgs {
  const uint8_t *w0, *s0;  // weight codes and scales (gate)
  const uint8_t *w1, *s1;  // up
  const uint8_t *xq, *xs;  // codes and scales of the rows to multiply
  const int32_t* pair_index;
  const int4* tiles;
  const int* ntiles;
  int rows;   // linear: rows of x
  int N, K;   // weight rows (of one expert) and the reduction axis
  int k;      // top_k
  void* out;  // linear: rows; down: fp32 [P][N]
  int out_dtype;
  int64_t out_stride;
  uint8_t *hq, *hs;  // gate and up: codes and scales of h [P]
};

__device__ __forceinline__ int swz(int row, int seg) { return seg ^ ((row >> 2) & 3); }

// One stage of the ring in LDS: 128 values of the reduction axis. Row r's four 16-byte blocks
// sit at positions swz(r, block), so that 16 neighbouring rows' reads of one block fall into
// different banks; its four scales are one word (TAIL: a word a scale).
template <int BN, int BM, bool TAIL>
struct Stage {
  static constexpr int kXRows = BM < 64 ? 64 : BM;  // a direct load brings in 64 rows
  uint4 w[BN * 4];
  uint4 x[kXRows * 4];
  uint32_t ws[TAIL ? 4 : 1][kThreads];
  uint32_t xs[TAIL ? 4 : 1][kThreads];
};

// A workgroup of 4 waves multiplies BM rows of x by BN weight rows. The waves lie WM by 4 / WM
// over the tile; a wave holds NW x NX accumulators of 32 x 32 (weight rows by rows of x, so
// that a lane holds 16 weight rows of one row of x: half of a block of h). A ring of SLOTS
// stages is filled by direct loads into LDS. A stage is two instructions deep: while the first
// half multiplies, the second half's operands are read, and while the second multiplies, those
// of the next stage. Between them the stage's reads are complete and its slot is refilled.
template <int WM, int NW, int NX, int SLOTS, bool TAIL, int MODE>
struct Tile {
  static constexpr int WN = 4 / WM;
  static constexpr int BN = 32 * NW * WN, BM = 32 * NX * WM;
  static constexpr int kGroupsW = NW, kGroupsX = NX;  // 32-row groups a wave
  typedef Stage<BN, BM, TAIL> S;
  static constexpr int kWLoads = BN / 64, kXLoads = S::kXRows / 64;
  static constexpr int kOps = kWLoads + kXLoads + (TAIL ? 8 : 2);
  static_assert(BN >= 64 && BN <= kThreads && BM <= kThreads, "one scale word a thread");

  S* ring;
  const uint8_t* wp[kWLoads];  // this thread's weight rows, at its block of stage 0
  const uint8_t* xp[kXLoads];
  const uint8_t *wsp, *xsp;  // its scale words at stage 0
  int tid, lane, wave, wm, wn, nk, nb;
  mx_f32x16 acc[NW][NX];

  struct Ops {
    i32x4 w[NW], x[NX];
  };
  struct Scales {
    int w[TAIL ? 2 : 1][NW], x[TAIL ? 2 : 1][NX];
  };

  __device__ __forceinline__ int block_of() const { return swz(tid >> 2, tid & 3); }

  __device__ __forceinline__ void load(int stage, int slot) const {
    const int s = min(stage, nk - 1);
    S& st = ring[slot];
    const int b = 4 * s + block_of();
    const size_t off = (size_t)s * kStepBytes;
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) {
      const uint8_t* p = wp[i] + off;
      if (TAIL && b >= nb) p = mx_zero_block;
      __builtin_amdgcn_global_load_lds((gptr_t)p, (lptr_t)(st.w + kThreads * i + kWave * wave), 16, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
      const uint8_t* p = xp[i] + off;
      if (TAIL && b >= nb) p = mx_zero_block;
      __builtin_amdgcn_global_load_lds((gptr_t)p, (lptr_t)(st.x + kThreads * i + kWave * wave), 16, 0, 0);
    }
    if constexpr (TAIL) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = 4 * s + j < nb;
        __builtin_amdgcn_global_load_lds((gptr_t)(in ? wsp + 4 * s + j : mx_unit_scale),
                                         (lptr_t)(st.ws[j] + kWave * wave), 1, 0, 0);
        __builtin_amdgcn_global_load_lds((gptr_t)(in ? xsp + 4 * s + j : mx_unit_scale),
                                         (lptr_t)(st.xs[j] + kWave * wave), 1, 0, 0);
      }
    } else {
      __builtin_amdgcn_global_load_lds((gptr_t)(wsp + 4 * s), (lptr_t)(st.ws[0] + kWave * wave), 4, 0, 0);
      __builtin_amdgcn_global_load_lds((gptr_t)(xsp + 4 * s), (lptr_t)(st.xs[0] + kWave * wave), 4, 0, 0);
    }
  }

  // Lane l of the half h = l / 32 takes blocks 2h (first instruction) and 2h + 1 (second).
  __device__ __forceinline__ Ops read(int slot, int half) const {
    const S& st = ring[slot];
    const int r = lane & 31, b = 2 * (lane >> 5) + half;
    Ops o;
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      const int row = (wn * NW + q) * 32 + r;
      __builtin_memcpy(&o.w[q], &st.w[4 * row + swz(row, b)], 16);
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int row = (wm * NX + i) * 32 + r;
      __builtin_memcpy(&o.x[i], &st.x[4 * row + swz(row, b)], 16);
    }
    return o;
  }

  __device__ __forceinline__ Scales scales(int slot) const {
    const S& st = ring[slot];
    const int r = lane & 31, h = lane >> 5;
    Scales o;
#pragma unroll
    for (int q = 0; q < NW; ++q) {
      const int row = (wn * NW + q) * 32 + r;
      if constexpr (TAIL) {
        o.w[0][q] = (int)st.ws[2 * h][row];
        o.w[1][q] = (int)st.ws[2 * h + 1][row];
      } else {
        o.w[0][q] = (int)(st.ws[0][row] >> (16 * h));
      }
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int row = (wm * NX + i) * 32 + r;
      if constexpr (TAIL) {
        o.x[0][i] = (int)st.xs[2 * h][row];
        o.x[1][i] = (int)st.xs[2 * h + 1][row];
      } else {
        o.x[0][i] = (int)(st.xs[0][row] >> (16 * h));
      }
    }
    return o;
  }

  template <int HALF>
  __device__ __forceinline__ void multiply(const Ops& o, const Scales& s) {
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
      for (int q = 0; q < NW; ++q)
        acc[q][i] = mx_mma32<TAIL ? 0 : HALF>(o.w[q], o.x[i], acc[q][i], s.w[TAIL ? HALF : 0][q],
                                              s.x[TAIL ? HALF : 0][i]);
  }

  __device__ __forceinline__ void run() {
#pragma unroll
    for (int q = 0; q < NW; ++q)
#pragma unroll
      for (int i = 0; i < NX; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[q][i][j] = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) load(s, s);
    wait_vmcnt<(SLOTS - 1) * kOps>();
    barrier_after_lds_dma();
    Ops a = read(0, 0);
    Scales sc = scales(0);
    int slot = 0;
    for (int s = 0; s < nk; ++s) {
      const Ops b = read(slot, 1);
      multiply<0>(a, sc);
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's reads of the stage are done
      wait_vmcnt<(SLOTS - 2) * kOps>();    // and its loads of the next one
      barrier_after_lds_dma();
      load(s + SLOTS, slot);
      slot = slot + 1 == SLOTS ? 0 : slot + 1;
      const Scales next = scales(slot);
      a = read(slot, 0);
      multiply<1>(b, sc);
      sc = next;
    }
    wait_vmcnt<0>();  // the loads past the last stage have landed
  }

  // e: expert (its weights); n0: first weight row (gate and up: first row of f); m0, rows: this
  // tile's rows of x (gate and up: grouped pairs; down: grouped pairs; linear: rows)
  __device__ __forceinline__ void init(S* ring_, const GemmArgs& a, int e, int n0, int m0, int rows) {
    ring = ring_;
    tid = threadIdx.x;
    lane = tid & (kWave - 1);
    wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    wm = wave % WM;
    wn = wave / WM;
    nb = a.K / kMxBlock;
    nk = (nb + 3) / 4;
    const size_t codes = (size_t)a.K / 2;
    auto weight = [&](int tr, const uint8_t*& c, const uint8_t*& s) {
      // tile row tr: 32-row group tr / 32 of wave column tr / (32 NW)
      int row = n0 + tr;
      bool up = false;
      if constexpr (MODE == kGateUp) {
        // a wave's groups: NW / 2 of gate, then the same rows of up
        const int group = tr / 32, q = group % NW;
        up = q >= NW / 2;
        row = n0 + ((group / NW) * (NW / 2) + q % (NW / 2)) * 32 + tr % 32;
      }
      // past the matrix: its last row, never stored
      const size_t at = (size_t)e * a.N + min(row, a.N - 1);
      c = (up ? a.w1 : a.w0) + at * codes;
      s = (up ? a.s1 : a.s0) + at * nb;
    };
    auto source = [&](int i) -> size_t {
      const int g = m0 + min(i, rows - 1);
      return MODE == kGateUp ? (size_t)(a.pair_index[g] / a.k) : (size_t)g;
    };
    const uint8_t* unused;
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) {
      weight(64 * i + (tid >> 2), wp[i], unused);
      wp[i] += 16 * block_of();
    }
    weight(min(tid, BN - 1), unused, wsp);
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      xp[i] = a.xq + source(64 * i + (tid >> 2)) * codes + 16 * block_of();
    xsp = a.xs + source(min(tid, BM - 1)) * nb;
  }
};

// The four pieces and the scale of a block of h from its 64-bit values. The gate and up sums of
// the block lie in LDS as gu[value][lane], gate first; lanes l and l + 32 hold its two halves.
// Rolled loops: taken by a block in some two hundred.
__device__ __forceinline__ void hidden_block64(float* gu, int lane, uint32_t (&pieces)[4], uint32_t& scale) {
  double m = 0.0;
  bool bad = false;
#pragma unroll 1
  for (int j = 0; j < 16; ++j) {
    float *lo = gu + j * kWave + lane, *hi = lo + 16 * kWave;
    const double h = mx_silu_up64(*lo, *hi);
    bad |= !(fabs(h) < __builtin_inf());
    m = fmax(m, fabs(h));
    const uint64_t bits = (uint64_t)__double_as_longlong(h);  // h in the place of its sums
    *lo = __uint_as_float((uint32_t)bits);
    *hi = __uint_as_float((uint32_t)(bits >> 32));
  }
  m = fmax(m, __shfl_xor(m, 32));
  bad |= __shfl_xor((int)bad, 32) != 0;
  scale = bad ? 255u : mx_scale_byte64(m);
  uint64_t all = 0;
#pragma unroll 1
  for (int j = 0; j < 16; ++j) {
    const float *lo = gu + j * kWave + lane, *hi = lo + 16 * kWave;
    const uint64_t bits = (uint64_t)__float_as_uint(*hi) << 32 | __float_as_uint(*lo);
    const uint64_t c = bad ? 0u : mx_code64(__longlong_as_double((int64_t)bits), scale);
    all |= c << (4 * j);
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) pieces[p] = (uint32_t)(all >> (16 * p)) & 0xffffu;
}

// A value is off by at most 2^-20 of itself (the exponential 2 ulp, the sum half of one, the
// reciprocal 1, two products half each: 4.5 * 2^-23 < 2^-20).
__device__ __forceinline__ float silu_up(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + expf(-g)) * u;
}

// 16 values of h (half of a block; lane ^ 32 holds the other half) to four pieces of four codes
// and the scale. The fast values decide where the slightly smaller and the slightly larger
// block give the same codes; otherwise the block is computed again in binary64.
template <class Stage16>
__device__ __forceinline__ void hidden_block(const mx_f32x16& g, const mx_f32x16& u, int lane,
                                             uint32_t (&pieces)[4], uint32_t& scale, Stage16 stage) {
  float h[16];
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    h[j] = silu_up(g[j], u[j]);
    m = fmaxf(m, fabsf(h[j]));
  }
  m = fmaxf(m, __shfl_xor(m, 32));
  constexpr float kLess = 1.0f - 0x1p-20f, kMore = 1.0f + 0x1p-20f;
  scale = mx_scale_byte(__float_as_uint(m * kMore));
  // tiny blocks (the products above may have lost bits) and ones that are not finite, too
  bool redo = mx_scale_byte(__float_as_uint(m * kLess)) != scale || !(m < 0x1p120f) || m < 0x1p-90f;
#pragma unroll
  for (int j = 0; j < 16; ++j) redo |= !(fabsf(h[j]) <= m);  // NaN, which the maximum passes over
  const float f = mx_scale_float(scale);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, h[4 * p] * kLess, h[4 * p + 1] * kLess, f, 0);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, h[4 * p + 2] * kLess, h[4 * p + 3] * kLess, f, 1);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, h[4 * p] * kMore, h[4 * p + 1] * kMore, f, 0);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, h[4 * p + 2] * kMore, h[4 * p + 3] * kMore, f, 1);
    redo |= lo != hi;
    pieces[p] = lo;
  }
  // a block of zeros (a row of zeros) is what it is
  bool some = false;
#pragma unroll
  for (int j = 0; j < 16; ++j) some |= g[j] != 0.0f && u[j] != 0.0f;
  some |= __shfl_xor((int)some, 32) != 0;
  redo = redo && (some || m != 0.0f);
  if (__ballot(redo)) {
    float* gu = stage();
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      gu[j * kWave + lane] = g[j];
      gu[(16 + j) * kWave + lane] = u[j];
    }
    __builtin_amdgcn_wave_barrier();
    hidden_block64(gu, lane, pieces, scale);
    __builtin_amdgcn_wave_barrier();
  }
}

template <class T>
__device__ __forceinline__ void gateup_epilogue(T& c, const GemmArgs& a, int n0, int g0, int rows,
                                                float* lds) {
  constexpr int NG = T::kGroupsW / 2, NX = T::kGroupsX;  // gate groups a wave, groups of pairs
  __syncthreads();  // every wave is done with the ring
  const int lane = c.lane, r = lane & 31, half = lane >> 5;
  float* mine = lds + c.wave * (32 * kWave);
#pragma unroll
  for (int i = 0; i < NX; ++i)
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      uint32_t pc[4], scale;
      hidden_block(c.acc[q][i], c.acc[NG + q][i], lane, pc, scale, [&] { return mine; });
      // piece p holds rows 8p + 4 half .. + 3 of the block: word p is piece p of the lower half
      // and then of the upper; each half stores two words
      const uint32_t mine0 = half ? pc[2] : pc[0], mine1 = half ? pc[3] : pc[1];
      const uint32_t give0 = half ? pc[0] : pc[2], give1 = half ? pc[1] : pc[3];
      const uint32_t got = (uint32_t)__shfl_xor((int)(give0 | give1 << 16), 32);
      const uint32_t g0w = got & 0xffffu, g1w = got >> 16;
      uint2 word;
      word.x = half ? (g0w | mine0 << 16) : (mine0 | g0w << 16);
      word.y = half ? (g1w | mine1 << 16) : (mine1 | g1w << 16);
      const int row = (c.wm * NX + i) * 32 + r;
      const int f0 = n0 + (c.wn * NG + q) * 32;
      if (row < rows && f0 < a.N) {
        const size_t g = (size_t)(g0 + row);
        *reinterpret_cast<uint2*>(a.hq + g * (a.N / 2) + f0 / 2 + 8 * half) = word;
        if (half == 0) a.hs[g * (a.N / kMxBlock) + f0 / kMxBlock] = (uint8_t)scale;
      }
    }
}

// Lane l holds, of row l % 32 of x, the outputs 8p + 4 (l / 32) .. + 3, p = 0..3, of each group.
template <class T, int MODE>
__device__ __forceinline__ void rows_epilogue(T& c, const GemmArgs& a, int n0, int m0, int rows) {
  constexpr int NX = T::kGroupsX, NW = T::kGroupsW;
  const int lane = c.lane, r = lane & 31, half = lane >> 5;
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int row = (c.wm * NX + i) * 32 + r;
    if (row >= rows) continue;
    const size_t at = MODE == kDown ? (size_t)a.pair_index[m0 + row] : (size_t)(m0 + row);
#pragma unroll
    for (int q = 0; q < NW; ++q)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int col = n0 + (c.wn * NW + q) * 32 + 8 * p + 4 * half;
        const float v0 = c.acc[q][i][4 * p], v1 = c.acc[q][i][4 * p + 1], v2 = c.acc[q][i][4 * p + 2],
                    v3 = c.acc[q][i][4 * p + 3];
        if constexpr (MODE == kDown) {
          if (col < a.N) {  // a multiple of 32
            const mx_f32x4 v = {v0, v1, v2, v3};
            __builtin_nontemporal_store(
                v, reinterpret_cast<mx_f32x4*>(static_cast<float*>(a.out) + at * a.N + col));
          }
        } else {
          const float v[4] = {v0, v1, v2, v3};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (col + j >= a.N) break;
            const int64_t o = (int64_t)at * a.out_stride + col + j;
            if (a.out_dtype == MOE_F32) static_cast<float*>(a.out)[o] = v[j];
            else if (a.out_dtype == MOE_BF16) static_cast<__bf16*>(a.out)[o] = (__bf16)v[j];
            else static_cast<_Float16*>(a.out)[o] = (_Float16)v[j];
          }
        }
      }
  }
}

template <int WM, int NW, int NX, int SLOTS, bool TAIL, int MODE>
__device__ __forceinline__ void tile(char* lds, const GemmArgs& a, int e, int n0, int m0, int rows) {
  typedef Tile<WM, NW, NX, SLOTS, TAIL, MODE> T;
  T c;
  c.init(reinterpret_cast<typename T::S*>(lds), a, e, n0, m0, rows);
  c.run();
  if constexpr (MODE == kGateUp)
    gateup_epilogue(c, a, n0, m0, rows, reinterpret_cast<float*>(lds));
  else
    rows_epilogue<T, MODE>(c, a, n0, m0, rows);
}

// M-tile mt of the list runs on XCD mt % 8, which takes its column tiles one after another (they
// share the rows of x in that XCD's L2).
__device__ __forceinline__ bool list_tile(int ntiles, int ntn, int& mt, int& nt) {
  const int slot = (int)(blockIdx.x / 8);
  mt = (int)(blockIdx.x % 8) + 8 * (slot / ntn);
  nt = slot % ntn;
  return mt < ntiles;
}

// The grouped product: 256 weight rows by up to 128 pairs.
template <bool TAIL, int MODE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_mx_grouped(GemmArgs a) {
  constexpr int SLOTS = TAIL ? 2 : 3;
  __shared__ __attribute__((aligned(16))) char lds[sizeof(Stage<256, 128, TAIL>) * SLOTS];
  constexpr int kN = MODE == kGateUp ? 128 : 256;  // rows of f, or of d, a workgroup
  const int ntn = (a.N + kN - 1) / kN;
  int mt, nt;
  if (!list_tile(load_uniform(a.ntiles), ntn, mt, nt)) return;
  const int4 t = load_uniform(a.tiles + mt);
  if (t.z <= 32)
    tile<1, 2, 1, SLOTS, TAIL, MODE>(lds, a, t.x, nt * kN, t.y, t.z);
  else if (t.z <= 64)
    tile<1, 2, 2, SLOTS, TAIL, MODE>(lds, a, t.x, nt * kN, t.y, t.z);
  else
    tile<1, 2, 4, SLOTS, TAIL, MODE>(lds, a, t.x, nt * kN, t.y, t.z);
}

template <int WM, int NW, int NX, int SLOTS, bool TAIL>
__global__ __launch_bounds__(kThreads) void k_mx_linear(GemmArgs a) {
  typedef Tile<WM, NW, NX, SLOTS, TAIL, kLinear> T;
  __shared__ __attribute__((aligned(16))) char lds[sizeof(typename T::S) * SLOTS];
  const int ntn = (a.N + T::BN - 1) / T::BN;
  int mt, nt;
  if (!list_tile((a.rows + T::BM - 1) / T::BM, ntn, mt, nt)) return;
  tile<WM, NW, NX, SLOTS, TAIL, kLinear>(lds, a, 0, nt * T::BN, mt * T::BM, min(T::BM, a.rows - mt * T::BM));
}

// ---------------------------------------------------------------- work list

// One workgroup, one thread an expert: every full tile in expert order, then the partly filled
// ones by the rows they compute (128, 64, 32), so that the longest start first.
__global__ __launch_bounds__(1024) void k_mx_tiles(const int32_t* __restrict__ offsets, int E,
                                                   int4* __restrict__ tiles, int* __restrict__ ntiles) {
  __shared__ int s_wsum[16];
  __shared__ int s_total;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int beg = tid < E ? offsets[tid] : 0;
  const int m = tid < E ? offsets[tid + 1] - beg : 0;
  const int nfull = m / kMxBM, rem = m - nfull * kMxBM;
  const int cls = rem == 0 ? -1 : rem > 64 ? 0 : rem > 32 ? 1 : 2;
  int start = 0;
  auto place = [&](int v) {
    int incl = v;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int o = __shfl_up(incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == kWave - 1) s_wsum[wave] = incl;
    __syncthreads();
    int base = incl - v;
    for (int w = 0; w < wave; ++w) base += s_wsum[w];
    if (tid == 1023) s_total = base + v;
    __syncthreads();
    const int pos = start + base;
    start += s_total;
    __syncthreads();
    return pos;
  };
  const int fb = place(nfull);
  for (int i = 0; i < nfull; ++i) tiles[fb + i] = make_int4(tid, beg + i * kMxBM, kMxBM, 0);
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    const int pb = place(cls == c ? 1 : 0);
    if (cls == c) tiles[pb] = make_int4(tid, beg + nfull * kMxBM, rem, 0);
  }
  if (tid == 0) *ntiles = start;
}

// ---------------------------------------------------------------- combine

constexpr int kCombineBatch = 16;

__global__ __launch_bounds__(1024) void k_mx_combine(const float* __restrict__ y, const float* __restrict__ w,
                                                     int d, int k, const float* residual, float* out) {
  const int t = blockIdx.x;
  for (int c = 4 * threadIdx.x; c < d; c += 4 * blockDim.x) {
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    for (int j0 = 0; j0 < k; j0 += kCombineBatch) {
      mx_f32x4 v[kCombineBatch];
      float wj[kCombineBatch];
#pragma unroll
      for (int i = 0; i < kCombineBatch; ++i)
        if (j0 + i < k) {
          const size_t p = (size_t)t * k + j0 + i;
          wj[i] = w[p];
          v[i] = __builtin_nontemporal_load(reinterpret_cast<const mx_f32x4*>(y + p * d + c));
        }
#pragma unroll
      for (int i = 0; i < kCombineBatch; ++i)
        if (j0 + i < k)
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q] += (double)wj[i] * (double)v[i][q];
    }
    const size_t at = (size_t)t * d + c;
    mx_f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
    if (residual) r = *reinterpret_cast<const mx_f32x4*>(residual + at);
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = (float)((double)r[q] + acc[q]);
    *reinterpret_cast<mx_f32x4*>(out + at) = r;
  }
}

inline int list_grid(int max_mt, int ntn) { return (max_mt + 7) / 8 * 8 * ntn; }

template <int WM, int NW, int NX, int SLOTS, int TSLOTS>
void linear(const GemmArgs& g, hipStream_t stream) {
  constexpr int BN = 32 * NW * (4 / WM), BM = 32 * NX * WM;
  const dim3 grid(list_grid((g.rows + BM - 1) / BM, (g.N + BN - 1) / BN));
  if (g.K % 128 == 0)
    hipLaunchKernelGGL((k_mx_linear<WM, NW, NX, SLOTS, false>), grid, dim3(kThreads), 0, stream, g);
  else
    hipLaunchKernelGGL((k_mx_linear<WM, NW, NX, TSLOTS, true>), grid, dim3(kThreads), 0, stream, g);
}

}  // namespace

hipError_t launch_mx_linear(const MxLinearArgs& a, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  if (mx_linear_window(a.n, a.K)) return launch_mx_linear_window(a, stream);
  GemmArgs g{};
  g.w0 = a.w;
  g.s0 = a.ws;
  g.xq = a.xq;
  g.xs = a.xs;
  g.rows = a.n;
  g.N = a.N;
  g.K = a.K;
  g.out = a.out;
  g.out_dtype = a.out_dtype;
  g.out_stride = a.out_stride;
  if (a.x) {
    uint8_t* xq = reinterpret_cast<uint8_t*>(a.work);
    uint8_t* xs = xq + align256((size_t)a.n * (a.K / 2));
    const hipError_t err = launch_mx_quantize(
        MxQuantArgs{a.x, a.dtype, a.n, a.row_stride, a.K, xq, xs}, stream);
    if (err != hipSuccess) return err;
    g.xq = xq;
    g.xs = xs;
  }
  if ((long long)a.n * a.N <= 1024ll * 1024)
    linear<1, 1, 2, 4, 3>(g, stream);
  else
    linear<2, 4, 4, 4, 2>(g, stream);
  return hipGetLastError();
}

hipError_t launch_mx_ffn(const MxFfnArgs& a, hipStream_t stream) {
  const moe_mx_layer& L = *a.L;
  const int n = a.n, d = L.d_model, f = L.d_ff, k = L.top_k, E = L.n_experts, P = n * k;
  if (P == 0) return hipSuccess;
  if (mx_window(n, k)) return launch_mx_ffn_window(a, stream);
  const MxFfnWs W = mx_ffn_ws(n, k, d, f, E);
  uint8_t* xq = reinterpret_cast<uint8_t*>(a.work + W.xq);
  uint8_t* xs = reinterpret_cast<uint8_t*>(a.work + W.xs);
  uint8_t* hq = reinterpret_cast<uint8_t*>(a.work + W.hq);
  uint8_t* hs = reinterpret_cast<uint8_t*>(a.work + W.hs);
  float* y = reinterpret_cast<float*>(a.work + W.y);
  int4* tiles = reinterpret_cast<int4*>(a.work + W.tiles);
  int* ntiles = reinterpret_cast<int*>(a.work + W.ntiles);
  hipLaunchKernelGGL(k_mx_tiles, dim3(1), dim3(1024), 0, stream, a.r->expert_offsets, E, tiles, ntiles);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  err = launch_mx_quantize(MxQuantArgs{a.x, a.dtype, n, a.row_stride, d, xq, xs}, stream);
  if (err != hipSuccess) return err;

  const int max_mt = mx_max_mtiles(P, E);
  GemmArgs g{};
  g.pair_index = a.r->pair_index;
  g.tiles = tiles;
  g.ntiles = ntiles;
  g.k = k;
  g.w0 = L.gate.codes;
  g.s0 = L.gate.scales;
  g.w1 = L.up.codes;
  g.s1 = L.up.scales;
  g.xq = xq;
  g.xs = xs;
  g.N = f;
  g.K = d;
  g.hq = hq;
  g.hs = hs;
  const dim3 gu(list_grid(max_mt, (f + 127) / 128));
  if (d % 128 == 0)
    hipLaunchKernelGGL((k_mx_grouped<false, kGateUp>), gu, dim3(kThreads), 0, stream, g);
  else
    hipLaunchKernelGGL((k_mx_grouped<true, kGateUp>), gu, dim3(kThreads), 0, stream, g);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  g.w0 = L.down.codes;
  g.s0 = L.down.scales;
  g.w1 = g.s1 = nullptr;
  g.xq = hq;
  g.xs = hs;
  g.N = d;
  g.K = f;
  g.out = y;
  const dim3 dn(list_grid(max_mt, (d + 255) / 256));
  if (f % 128 == 0)
    hipLaunchKernelGGL((k_mx_grouped<false, kDown>), dn, dim3(kThreads), 0, stream, g);
  else
    hipLaunchKernelGGL((k_mx_grouped<true, kDown>), dn, dim3(kThreads), 0, stream, g);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int threads = std::min(1024, ((d / 4 + kWave - 1) / kWave) * kWave);
  hipLaunchKernelGGL(k_mx_combine, dim3(n), dim3(threads), 0, stream, y, a.r->topk_w, d, k, a.residual,
                     a.out);
  return hipGetLastError();
}

}  // namespace qmoe
