// Microscaled 4-bit matrix products of many rows: y = Q(x) W^T, and the routed experts'
// products of a batch or a prefill chunk.
//
//   k_mx_linear   one workgroup per tile of the product; rows out through LDS
//   k_mx_prepare  M-tile work list of the grouped products (expert, first grouped pair, pairs), and
//                 the rows of x in 4 bits
//   k_mx_grouped  one workgroup per tile of an expert's product; as gate and up it ends in
//                 h = silu(g) u and its 4-bit blocks, as the down product in fp32 rows
//   k_mx_combine  out[t] = residual[t] + sum_j w[t][j] y[place of pair t k + j], slot order, binary64
//
// Measured (kernel traces): 8192 rows, a reduction of 4096 and 8192 outputs 157-162 us, 3.4-3.5
// PFLOP/s, a reduction of 8192 and 4096 outputs 142-148, 3.7-3.9 (the bare scaled matrix
// instructions reach 6.6 on random codes, which the power limit sets, a bf16 product of the
// library 1.25); 512 experts of 768 by 2048, top 10: 256 tokens 162 + 102 us (gate and up, down),
// the weights at 5 TB/s; 8192 tokens 257-300 + 227-250 us, and 137 us (5.4 TB/s) for the sum over
// the slots.
#include "qmoe_mx_internal.h"

namespace qmoe {
namespace {

typedef __attribute__((address_space(3))) void* lptr_t;
typedef __attribute__((address_space(3))) float lds_float;
typedef __attribute__((address_space(3))) mx_f32x4 lds_f32x4;

__device__ __forceinline__ uint32_t lds_address(void* p) { return (uint32_t)(uintptr_t)(lptr_t)p; }

constexpr int kThreads = 256;
constexpr int kTileRows = 256;  // most weight rows, and rows of x, of a tile

enum Mode { kLinear, kGateUp, kDown };

struct GemmArgs {
  const uint8_t *w0, *s0;  // weight codes and scales (gate)
  const uint8_t *w1, *s1;  // up
  const uint8_t *xq, *xs;  // codes and scales of the rows to multiply
  const int32_t* pair_index;
  int32_t* place;        // [P] grouped place of each pair, which gate and up write
  const int4* tiles;
  const int* xcd_first;  // [kXcds + 1] first tile of each XCD
  int xcd_m;             // linear: XCDs side by side over the rows of x; an XCD's tiles are
  int xcd_rm, xcd_rn;    // xcd_rm x xcd_rn, taken in panels of `panel` column tiles
  int panel;
  int64_t wrows, xrows;  // rows of the weights' and of x's tensors
  int rows;   // linear: rows of x
  int N, K;   // weight rows (of one expert) and the reduction axis
  int k;      // top_k
  void* out;  // linear: rows; down: fp32 [P][N], in the order of the grouped pairs
  int out_dtype;
  int64_t out_stride;
  uint8_t *hq, *hs;  // gate and up: codes and scales of h [P]
};

// Buffers are declared 2^31 bytes long: every offset is kept inside the tensor by construction,
// and an offset of 2^31 reads zeros.
constexpr uint32_t kBufferBytes = 0x80000000u;
constexpr int kOutside = (int)0x80000000u;

// One stage of the ring in LDS: KB blocks (of 32 values) of the reduction axis. Row r's 16-byte
// blocks sit at positions swz(r, block), so that 16 neighbouring rows' reads of one block fall
// into different banks.
template <int BN, int BM, int KB>
struct Stage {
  static constexpr int kBlocks = KB;
  uint4 w[BN * KB];
  uint4 x[(BM < 64 ? 64 : BM) * KB];
  __device__ static __forceinline__ int swz(int row, int seg) {
    static_assert(KB == 4 || KB == 8, "64 or 128 bytes a row");
    return KB == 4 ? seg ^ ((row >> 2) & 3) : seg ^ ((row >> 1) & 7);
  }
};

// Scales of two rounds: WORDS words (of four blocks) a row and round.
template <int BN, int BM, int WORDS>
struct ScaleRing {
  static constexpr int kWords = WORDS;
  uint32_t s[2][WORDS][BN + BM];
};

// The ring's slots by name: an array of them would be kept in memory.
template <class S, class SC, int N>
struct Slots {
  typedef S Slot;
  typedef SC Scale;
  static constexpr int kCount = N;
  S *s0, *s1, *s2, *s3;
  SC* scales;
  template <int I>
  __device__ __forceinline__ S* get() const {
    if constexpr (I == 0) return s0;
    else if constexpr (I == 1) return s1;
    else if constexpr (I == 2) return s2;
    else return s3;
  }
};

// A workgroup of WM x WN waves multiplies BM rows of x by BN weight rows; a wave holds NW x NX
// accumulators of 32 x 32 (weight rows by rows of x, so that a lane holds 16 weight rows of one
// row of x: half of a block of h). For gate and up the first half of the tile's weight rows are
// gate, the second the same rows of up, and a wave holds both of its rows.
//
// A ring of SLOTS stages is filled by direct loads into LDS; the offset of a lane never changes
// and the stage is a scalar offset, so a load costs no arithmetic. Every slot is an LDS variable
// of its own: the compiler then sees that the slots being filled are not the one being read, and
// adds no wait for them. While an instruction's products run, the next one's operands are read;
// before the last of a stage all reads of its slot are complete, and the slot is refilled.
//
// A stage of eight blocks is 128 bytes of a row, whole lines of memory: with four, every line is
// asked for twice, which cost the 256 x 256 tile 1.06 us per 128 values instead of 0.95 (8192
// rows by 8192 columns) although its four slots reach a stage further ahead than two.
//
// Scales come through registers, ROUND stages of a row at once: a word a row and stage would
// cost the memory path as many requests as the codes do (a line a lane), and rows of scales need
// not be whole words. They are requested a round ahead and go to LDS a word per four blocks.
//
// TAIL: K is not a whole number of rounds. Codes and scales past K are zeros.
template <class R, int WM, int WN, int NW, int NX, bool TAIL, int MODE>
struct Tile {
  typedef typename R::Slot S;
  typedef typename R::Scale SC;
  static constexpr int SLOTS = R::kCount, KB = S::kBlocks, WORDS = SC::kWords;
  static constexpr int ROUND = 4 * WORDS / KB;  // stages a round of scales
  static constexpr int NT = kWave * WM * WN;  // threads: each load brings in NT / KB rows
  static constexpr int BN = 32 * NW * WN, BM = 32 * NX * WM;
  static constexpr int kGroupsW = NW, kGroupsX = NX;  // 32-row groups a wave
  static constexpr int kRows = NT / KB;
  static constexpr int kWLoads = BN / kRows, kXLoads = BM < kRows ? 1 : BM / kRows;
  static constexpr int kOps = kWLoads + kXLoads;  // direct loads a thread and stage
  // rows of scales a thread fetches: with 8 waves, each half those of one matrix
  static constexpr int kKinds = NT == 2 * kTileRows ? 1 : 2;
  static_assert(NT == kTileRows || NT == 2 * kTileRows, "a row of scales a thread and kind");
  static_assert(BN >= kRows && BN <= kTileRows && BM <= kTileRows, "whole loads");
  static_assert(MODE != kGateUp || BN == 256, "gate rows and up rows in loads and waves of their own");

  R st;
  __amdgpu_buffer_rsrc_t wbuf[MODE == kGateUp ? 2 : 1], xbuf;
  int woff[kWLoads], xoff[kXLoads];  // byte offsets of this thread at stage 0
  const uint8_t* sbase[kKinds];      // scales: the tensor from the tile's first row on,
  int soff[kKinds], send[kKinds];    // this thread's row in it, and its last 4 WORDS bytes (before
                                     // its start where it is shorter: only in the workspace)
  int srow[kKinds];                  // its place in the scale ring (-1: none)
  uint32_t held[kKinds][WORDS];      // the round that is requested
  int held_by[kKinds];               // bytes that its words lie further on
  int tid, lane, wave, wm, wn, nk, nb;
  mx_f32x16 acc[NW][NX];

  struct Ops {
    i32x4 w[NW], x[NX];
  };
  struct Scales {
    int w[NW], x[NX];
  };

  __device__ __forceinline__ int block_of() const { return S::swz(tid / KB, tid % KB); }

  // 16 bytes a lane, into LDS in the order of the lanes
  __device__ __forceinline__ void bring(__amdgpu_buffer_rsrc_t b, void* lds, int off, int at) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lptr_t)lds, 16, off, at, 0, 0);
  }

  template <int SLOT>
  __device__ __forceinline__ void load(int stage) const {
    const int s = min(stage, nk - 1);
    S& g = *st.template get<SLOT>();
    const bool in = !TAIL || KB * s + block_of() < nb;
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      bring(wbuf[MODE == kGateUp ? i / (kWLoads / 2) : 0], g.w + NT * i + kWave * wave, in ? woff[i] : kOutside,
            s * (16 * KB));
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
      bring(xbuf, g.x + NT * i + kWave * wave, in ? xoff[i] : kOutside, s * (16 * KB));
  }

  // Requests this thread's scales of a round (TAIL: the last bytes of the tensor from where a
  // whole request ends with them).
  __device__ __forceinline__ void fetch(int round) {
#pragma unroll
    for (int t = 0; t < kKinds; ++t) {
      const int want = soff[t] + 4 * WORDS * min(round, (nb - 1) / (4 * WORDS));
      const int at = TAIL ? min(want, send[t]) : want;
      if constexpr (TAIL) held_by[t] = want - at;
      __builtin_memcpy(held[t], sbase[t] + at, 4 * WORDS);
    }
  }

  // Stores the requested round.
  __device__ __forceinline__ void keep(int round) {
#pragma unroll
    for (int t = 0; t < kKinds; ++t) {
      if constexpr (TAIL) {
        static_assert(!TAIL || WORDS == 2, "a round is one 64-bit word");
        const int there = nb - 8 * round;  // scales of the row from this round on
        const uint64_t mask = there >= 8 ? ~0ull : there <= 0 ? 0ull : (1ull << (8 * there)) - 1ull;
        const uint64_t v = ((uint64_t)held[t][1] << 32 | held[t][0]) >> (8 * held_by[t]) & mask;
        held[t][0] = (uint32_t)v;
        held[t][1] = (uint32_t)(v >> 32);
      }
#pragma unroll
      for (int j = 0; j < WORDS; ++j)
        if (srow[t] >= 0) st.scales->s[round & 1][j][srow[t]] = held[t][j];
    }
  }

  // Tile row of weight group q of this wave
  __device__ __forceinline__ int wrow(int q) const {
    const int r = lane & 31;
    if constexpr (MODE == kGateUp) {
      constexpr int NG = NW / 2;
      return (q / NG) * (BN / 2) + (wn * NG + q % NG) * 32 + r;
    }
    return (wn * NW + q) * 32 + r;
  }
  __device__ __forceinline__ int xrow(int i) const { return (wm * NX + i) * 32 + (lane & 31); }

  // Of four blocks, lane l of the half h = l / 32 takes blocks 2h (even instruction PART) and
  // 2h + 1 (odd).
  template <int SLOT, int PART>
  __device__ __forceinline__ void read(Ops& o) const {
    const S& g = *st.template get<SLOT>();
    const int b = 4 * (PART / 2) + 2 * (lane >> 5) + PART % 2;
#pragma unroll
    for (int i = 0; i < NX; ++i)
      __builtin_memcpy(&o.x[i], &g.x[KB * xrow(i) + S::swz(lane & 31, b)], 16);
#pragma unroll
    for (int q = 0; q < NW; ++q)
      __builtin_memcpy(&o.w[q], &g.w[KB * wrow(q) + S::swz(lane & 31, b)], 16);
  }

  __device__ __forceinline__ void scales(int word, Scales& o) const {
    const uint32_t* p = st.scales->s[word / WORDS & 1][word % WORDS];
#pragma unroll
    for (int q = 0; q < NW; ++q) o.w[q] = (int)p[wrow(q)];
#pragma unroll
    for (int i = 0; i < NX; ++i) o.x[i] = (int)p[BN + xrow(i)];
  }

  template <int HALF>
  __device__ __forceinline__ void multiply(const Ops& o, const Scales& s) {
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
      for (int q = 0; q < NW; ++q)
        acc[q][i] = mx_mma32<HALF>(o.w[q], o.x[i], acc[q][i], s.w[q], s.x[i]);
  }

  // The two scales of this lane's half to the lower half of each word (where the words are used,
  // not where they are read: that would wait for them).
  __device__ __forceinline__ void halve(Scales& o) const {
    const int sh = (lane >> 5) * 16;
#pragma unroll
    for (int q = 0; q < NW; ++q) o.w[q] = (int)((uint32_t)o.w[q] >> sh);
#pragma unroll
    for (int i = 0; i < NX; ++i) o.x[i] = (int)((uint32_t)o.x[i] >> sh);
  }

  // The operands are in registers at this point: without it the loads of the next stage are
  // moved behind the loop's branch, in front of the products that need them.
  __device__ __forceinline__ static void pin(Ops& o) {
#pragma unroll
    for (int i = 0; i < NX; ++i) asm volatile("" : "+v"(o.x[i]));
#pragma unroll
    for (int q = 0; q < NW; ++q) asm volatile("" : "+v"(o.w[q]));
  }
  __device__ __forceinline__ static void pin(Scales& o) {
#pragma unroll
    for (int i = 0; i < NX; ++i) asm volatile("" : "+v"(o.x[i]));
#pragma unroll
    for (int q = 0; q < NW; ++q) asm volatile("" : "+v"(o.w[q]));
  }

  // One product, then a share of the LDS reads and direct loads: the waves' reads and loads are
  // spread over the stage and do not hold up the matrix cores.
  template <int READS, int LOADS>
  __device__ __forceinline__ static void interleave() {
    constexpr int M = NW * NX;
    constexpr int kReads = (READS + M - 1) / M, kLoads = (LOADS + M - 1) / M;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a matrix-core op
      __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);  // LDS reads
      if (LOADS) __builtin_amdgcn_sched_group_barrier(0x020, kLoads, 0);  // direct loads
      __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // VALU
    }
  }

  // Instruction PART of a stage, not the last one: the next one's operands are read meanwhile,
  // and where it begins another word of scales, these.
  template <int SLOT, int PART>
  __device__ __forceinline__ void part(int s, Ops& a, Scales& sc) {
    constexpr bool kWord = PART % 2 == 1;
    Ops b;
    Scales next;
    if constexpr (PART % 2 == 0) halve(sc);
    if constexpr (kWord) scales(s * (KB / 4) + (PART + 1) / 2, next);
    read<SLOT, PART + 1>(b);
    multiply<PART % 2>(a, sc);
    interleave<(kWord ? 2 : 1) * (NW + NX), 0>();
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (PART + 2 < KB / 2) pin(b);
    a = b;
    if constexpr (kWord) {
      pin(next);
      sc = next;
    }
  }

  // Stage s, s modulo SLOTS = I: its first operands and scales are in a and sc.
  template <int I>
  __device__ __forceinline__ void step(int s, Ops& a, Scales& sc) {
    constexpr int SLOT = I % SLOTS, NEXT = (I + 1) % SLOTS;
    const bool round = SLOTS % ROUND == 0 ? I % ROUND == ROUND - 1 : (s + 1) % ROUND == 0;
    // the last stage of a round: the next one's scales to LDS, the one after it requested (before
    // this stage's barrier, behind which the next stage's scales are read)
    if (round) {
      keep((s + 1) / ROUND);
      fetch((s + 1) / ROUND + 1);
    }
    part<SLOT, 0>(s, a, sc);
    if constexpr (KB == 8) {
      part<SLOT, 1>(s, a, sc);
      part<SLOT, 2>(s, a, sc);
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's reads of the stage are done
    wait_vmcnt<(SLOTS - 2) * kOps>();    // and its loads of the next one
    barrier_after_lds_dma();
    __builtin_amdgcn_sched_barrier(0);
    load<SLOT>(s + SLOTS);
    Ops b;
    Scales next;
    scales((s + 1) * (KB / 4), next);
    read<NEXT, 0>(b);
    multiply<1>(a, sc);
    interleave<2 * (NW + NX), kOps>();
    __builtin_amdgcn_sched_barrier(0);
    pin(b);
    pin(next);
    a = b;
    sc = next;
  }

  template <int I>
  __device__ __forceinline__ void steps(int s, Ops& a, Scales& sc) {
    step<I>(s + I, a, sc);
    if constexpr (I + 1 < SLOTS) steps<I + 1>(s, a, sc);
  }
  template <int I>
  __device__ __forceinline__ void rest(int s, Ops& a, Scales& sc) {
    if (s + I >= nk) return;
    step<I>(s + I, a, sc);
    if constexpr (I + 2 < SLOTS) rest<I + 1>(s, a, sc);
  }

  template <int SLOT>
  __device__ __forceinline__ void first_loads() const {
    load<SLOT>(SLOT);
    if constexpr (SLOT + 1 < SLOTS) first_loads<SLOT + 1>();
  }

  __device__ __forceinline__ void run() {
#pragma unroll
    for (int q = 0; q < NW; ++q)
#pragma unroll
      for (int i = 0; i < NX; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[q][i][j] = 0.0f;
    fetch(0);
    first_loads<0>();
    keep(0);
    fetch(1);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the scales are in LDS
    wait_vmcnt<(SLOTS - 1) * kOps>();
    barrier_after_lds_dma();
    Ops a;
    Scales sc;
    read<0, 0>(a);
    scales(0, sc);
    pin(a);
    pin(sc);
    // SLOTS stages at a time, so that slots and places in a round are known, then the rest:
    // leaving the loop in its middle would make the compiler drain the ring at the loop's head
    int s = 0;
    for (; s + SLOTS <= nk; s += SLOTS) steps<0>(s, a, sc);
    rest<0>(s, a, sc);
    wait_vmcnt<0>();  // the loads past the last stage have landed
  }

  // e: expert (its weights); n0: first weight row (gate and up: first row of f); m0, rows: this
  // tile's rows of x (gate and up, down: grouped pairs)
  __device__ __forceinline__ void init(const R& slots, const GemmArgs& a, int e, int n0, int m0, int rows) {
    st = slots;
    tid = threadIdx.x;
    lane = tid & (kWave - 1);
    wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    wm = wave % WM;
    wn = wave / WM;
    nb = a.K / kMxBlock;
    nk = (nb + KB - 1) / KB;
    const int codes = a.K / 2;
    // weights: a buffer from the tile's first row; rows past the matrix: its last, never stored
    const size_t first = (size_t)e * a.N + n0;
    const int last = a.N - 1 - n0;
    wbuf[0] = buffer_rsrc(a.w0 + first * codes, kBufferBytes);
    if constexpr (MODE == kGateUp) wbuf[1] = buffer_rsrc(a.w1 + first * codes, kBufferBytes);
    constexpr int kOwn = MODE == kGateUp ? BN / 2 : BN;  // tile rows of one matrix
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
      woff[i] = min((kRows * i + tid / KB) % kOwn, last) * codes + 16 * block_of();
    // rows of x: those of the pairs' tokens (gate and up), or the tile's own from its first
    const size_t x0 = MODE == kGateUp ? 0 : (size_t)m0;
    xbuf = buffer_rsrc(a.xq + x0 * codes, kBufferBytes);
    auto source = [&](int i) {
      const int j = min(i, rows - 1);
      return MODE == kGateUp ? a.pair_index[m0 + j] / a.k : j;
    };
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) xoff[i] = source(kRows * i + tid / KB) * codes + 16 * block_of();
    auto row_of_scales = [&](int t, const uint8_t* base, int64_t tensor_rows, int row, int place) {
      sbase[t] = base;
      soff[t] = row * nb;
      send[t] = (int)min((int64_t)1 << 30, tensor_rows * nb - 4 * WORDS);
      srow[t] = place;
    };
    const uint8_t* ws = (MODE == kGateUp && wave >= 2 ? a.s1 : a.s0) + first * nb;
    const uint8_t* xs = a.xs + x0 * nb;
    const int64_t wleft = a.wrows - (int64_t)first, xleft = a.xrows - (int64_t)x0;
    const int row = tid % kTileRows;
    const int wplace = row < BN ? row : -1, xplace = row < BM ? BN + row : -1;
    const int wr = min(row % kOwn, last), xr = source(min(row, BM - 1));
    if constexpr (kKinds == 1) {
      if (wave < 4) row_of_scales(0, ws, wleft, wr, wplace);
      else row_of_scales(0, xs, xleft, xr, xplace);
    } else {
      row_of_scales(0, ws, wleft, wr, wplace);
      row_of_scales(1, xs, xleft, xr, xplace);
    }
  }
};

// The four pieces and the scale of a block of h from its 64-bit values. The gate and up sums of
// the block lie in LDS as gu[value][lane], gate first; lanes l and l + 32 hold its two halves.
// Rolled loops: only blocks whose scale the bounds leave open and odd ones (hidden_block) come here,
// with the rest of their wave.
__device__ __forceinline__ void hidden_block64(lds_float* gu, int lane, uint32_t (&pieces)[4], uint32_t& scale) {
  double m = 0.0;
  bool bad = false;
#pragma unroll 1
  for (int j = 0; j < 16; ++j) {
    lds_float *lo = gu + j * kWave + lane, *hi = lo + 16 * kWave;
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
    const lds_float *lo = gu + j * kWave + lane, *hi = lo + 16 * kWave;
    const uint64_t bits = (uint64_t)__float_as_uint(*hi) << 32 | __float_as_uint(*lo);
    const uint64_t c = bad ? 0u : mx_code64(__longlong_as_double((int64_t)bits), scale);
    all |= c << (4 * j);
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) pieces[p] = (uint32_t)(all >> (16 * p)) & 0xffffu;
}

// h = silu(g) u in fp32, from above: h (1 + 2^-20) within 4.1 2^-23 of itself (the exponential,
// whose argument's rounding is made good, 1.6 2^-23, the sum half of that unit, the reciprocal 1,
// two products half each), so that it is at least h, and less 2^-19 of itself at most h. For
// |g|, |u| <= 2^32, where the exponential is cut off or a product is subnormal, it is off by at
// most 2^-76: |g| e^g < 2^-108 for g <= -80, and a subnormal's last bit is 2^-149.
__device__ __forceinline__ float silu_up_above(float g, float u) {
  constexpr float kHigh = -0x1.715476p+0f, kLow = -0x1.4ae0cp-26f;  // -1 / ln 2
  const float c = fmaxf(g, -80.0f);
  const float t = c * kHigh;
  const float r = fmaf(c, kLow, fmaf(c, kHigh, -t));
  float e = __builtin_amdgcn_exp2f(t);
  e = fmaf(e, r * 0x1.62e43p-1f, e);
  constexpr float kLess = 1.0f - 0x1p-20f;
  return c * __builtin_amdgcn_rcpf(fmaf(e, kLess, kLess)) * u;
}

// 16 values of h (half of a block; lane ^ 32 holds the other half) to four pieces of four codes
// and the scale. Where a value's bounds have different codes, a value in some six thousand, it is
// computed again in binary64; where the scale's have, and for values that are tiny, huge or not
// finite, the whole block.
template <class Stage16>
__device__ __forceinline__ void hidden_block(const mx_f32x16& g, const mx_f32x16& u, int lane,
                                             uint32_t (&pieces)[4], uint32_t& scale, Stage16 stage) {
  constexpr float kBelow = 1.0f - 0x1p-19f;
  float h[16];
  float m = 0.0f, most = 0.0f;
  bool odd = false;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    h[j] = silu_up_above(g[j], u[j]);
    m = fmaxf(m, fabsf(h[j]));
    most = fmaxf(most, fmaxf(fabsf(g[j]), fabsf(u[j])));
    odd |= __builtin_isunordered(g[j], u[j]);  // which the maxima pass over
  }
  m = fmaxf(m, __shfl_xor(m, 32));
  scale = mx_scale_byte(__float_as_uint(m));
  // 2^-76 must be less than a thousandth of the largest value: far below the first border
  odd |= mx_scale_byte(__float_as_uint(m * kBelow)) != scale || !(m < 0x1p120f) || m < 0x1p-60f || most > 0x1p32f;
  const float f = mx_scale_float(scale);
  uint32_t differ = 0;
  uint32_t by[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, h[4 * p] * kBelow, h[4 * p + 1] * kBelow, f, 0);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, h[4 * p + 2] * kBelow, h[4 * p + 3] * kBelow, f, 1);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, h[4 * p], h[4 * p + 1], f, 0);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi, h[4 * p + 2], h[4 * p + 3], f, 1);
    by[p] = lo ^ hi;
    differ |= by[p];
    pieces[p] = lo;
  }
  if (!__ballot(odd || differ)) return;
  // a block of zeros (a row of zeros) is what it is; a NaN or an infinity times 0 is no zero
  bool some = m != 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float size = fabsf(g[j]) + fabsf(u[j]);
    some |= (g[j] != 0.0f && u[j] != 0.0f) || !(size < __builtin_inff());
  }
  some |= __shfl_xor((int)some, 32) != 0;
  odd = odd && some;
  lds_float* gu = stage();
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    gu[j * kWave + lane] = g[j];
    gu[(16 + j) * kWave + lane] = u[j];
  }
  __builtin_amdgcn_wave_barrier();
  if (__ballot(odd)) {
    hidden_block64(gu, lane, pieces, scale);
  } else {
    uint64_t all = 0, open = 0;  // codes; those to decide
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      all |= (uint64_t)pieces[p] << (16 * p);
      open |= (uint64_t)by[p] << (16 * p);
    }
#pragma unroll 1
    while (__ballot(open != 0)) {
      const int at = open ? __builtin_ctzll(open) & ~3 : 0;
      const lds_float* v = gu + (at >> 2) * kWave + lane;
      const uint64_t code = mx_code64(mx_silu_up64(v[0], v[16 * kWave]), scale);
      const uint64_t mask = open ? 15ull << at : 0ull;
      all = (all & ~mask) | (code << at & mask);
      open &= ~mask;
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) pieces[p] = (uint32_t)(all >> (16 * p)) & 0xffffu;
  }
  __builtin_amdgcn_wave_barrier();
}

// LDS that a wave has for itself once the ring is free: WAVES / SLOTS waves (rounded up) share a
// slot.
template <class R, int WAVES>
struct WaveLds {
  typedef typename R::Slot S;
  static constexpr int SLOTS = R::kCount;
  static constexpr int kShare = (WAVES + SLOTS - 1) / SLOTS;
  static constexpr size_t kBytes = sizeof(S) / kShare / 16 * 16;
  __device__ static __forceinline__ lds_float* of(const R& slots, int wave) {
    uint32_t at = lds_address(slots.s0);
    if (wave / kShare == 1) at = lds_address(slots.s1);
    if (SLOTS > 2 && wave / kShare == 2) at = lds_address(slots.s2);
    if (SLOTS > 3 && wave / kShare == 3) at = lds_address(slots.s3);
    return reinterpret_cast<lds_float*>(at + wave % kShare * (uint32_t)kBytes);
  }
};

template <class T>
__device__ __forceinline__ void gateup_epilogue(T& c, const GemmArgs& a, int n0, int g0, int rows,
                                                lds_float* lds) {
  constexpr int NG = T::kGroupsW / 2, NX = T::kGroupsX;  // gate groups a wave, groups of pairs
  __syncthreads();  // every wave is done with the ring
  const int lane = c.lane, half = lane >> 5;
#pragma unroll
  for (int i = 0; i < NX; ++i)
#pragma unroll
    for (int q = 0; q < NG; ++q) {
      uint32_t pc[4], scale;
      hidden_block(c.acc[q][i], c.acc[NG + q][i], lane, pc, scale, [&] { return lds; });
      // piece p holds rows 8p + 4 half .. + 3 of the block: word p is piece p of the lower half
      // and then of the upper; each half stores two words
      const uint32_t mine0 = half ? pc[2] : pc[0], mine1 = half ? pc[3] : pc[1];
      const uint32_t give0 = half ? pc[0] : pc[2], give1 = half ? pc[1] : pc[3];
      const uint32_t got = (uint32_t)__shfl_xor((int)(give0 | give1 << 16), 32);
      const uint32_t g0w = got & 0xffffu, g1w = got >> 16;
      uint2 word;
      word.x = half ? (g0w | mine0 << 16) : (mine0 | g0w << 16);
      word.y = half ? (g1w | mine1 << 16) : (mine1 | g1w << 16);
      const int row = c.xrow(i);
      const int f0 = n0 + (c.wn * NG + q) * 32;
      if (row < rows && f0 < a.N) {
        const size_t g = (size_t)(g0 + row);
        *reinterpret_cast<uint2*>(a.hq + g * (a.N / 2) + f0 / 2 + 8 * half) = word;
        if (half == 0) a.hs[g * (a.N / kMxBlock) + f0 / kMxBlock] = (uint8_t)scale;
      }
    }
}

// Lane l holds, of row l % 32 of x, the outputs 8p + 4 (l / 32) .. + 3, p = 0..3, of each group.
// 32 rows at a time go through LDS, so that a row's outputs of the wave leave side by side, 16
// bytes a lane; where out's rows or its last columns are not whole 16-byte words, a value a lane.
template <class T, int MODE>
__device__ __forceinline__ void rows_epilogue(T& c, const GemmArgs& a, int n0, int m0, int rows, lds_float* lds) {
  constexpr int NX = T::kGroupsX, NW = T::kGroupsW, kCols = 32 * NW, kPitch = kCols + 4;
  __syncthreads();  // every wave is done with the ring
  const int lane = c.lane, half = lane >> 5;
  const int col0 = n0 + c.wn * kCols;
  const bool words = MODE == kDown || (a.out_stride % 8 == 0 && a.N % 8 == 0 &&
                                       (reinterpret_cast<uintptr_t>(a.out) & 15) == 0);
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int first = (c.wm * NX + i) * 32;
    if (first >= rows) break;
#pragma unroll
    for (int q = 0; q < NW; ++q)
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const mx_f32x4 v = {c.acc[q][i][4 * p], c.acc[q][i][4 * p + 1], c.acc[q][i][4 * p + 2],
                            c.acc[q][i][4 * p + 3]};
        *reinterpret_cast<lds_f32x4*>(lds + (lane & 31) * kPitch + 32 * q + 8 * p + 4 * half) = v;
      }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const int count = min(32, rows - first);
    if (words && (MODE == kDown || a.out_dtype == MOE_F32)) {
      constexpr int kLanes = kCols / 4, kStep = kWave / kLanes;  // lanes a row, rows at once
      const int col = 4 * (lane % kLanes);
#pragma unroll
      for (int j = 0; j < 32 / kStep; ++j) {
        const int r = j * kStep + lane / kLanes;
        if (r >= count || col0 + col >= a.N) continue;
        const mx_f32x4 v = *reinterpret_cast<const lds_f32x4*>(lds + r * kPitch + col);
        const size_t at = (size_t)(m0 + first + r) * (MODE == kDown ? a.N : a.out_stride);
        __builtin_nontemporal_store(
            v, reinterpret_cast<mx_f32x4*>(static_cast<float*>(a.out) + at + col0 + col));
      }
    } else if (words) {
      constexpr int kLanes = kCols / 8, kStep = kWave / kLanes;
      const int col = 8 * (lane % kLanes);
#pragma unroll
      for (int j = 0; j < 32 / kStep; ++j) {
        const int r = j * kStep + lane / kLanes;
        if (r >= count || col0 + col >= a.N) continue;
        const mx_f32x4 v = *reinterpret_cast<const lds_f32x4*>(lds + r * kPitch + col);
        const mx_f32x4 w = *reinterpret_cast<const lds_f32x4*>(lds + r * kPitch + col + 4);
        i32x4 o;
        if (a.out_dtype == MOE_BF16) {
          typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
          const bf16x8 h = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3],
                            (__bf16)w[0], (__bf16)w[1], (__bf16)w[2], (__bf16)w[3]};
          __builtin_memcpy(&o, &h, 16);
        } else {
          typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
          const f16x8 h = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3],
                           (_Float16)w[0], (_Float16)w[1], (_Float16)w[2], (_Float16)w[3]};
          __builtin_memcpy(&o, &h, 16);
        }
        *reinterpret_cast<i32x4*>(static_cast<uint16_t*>(a.out) +
                                  (size_t)(m0 + first + r) * a.out_stride + col0 + col) = o;
      }
    } else {
      for (int j = lane; j < count * kCols; j += kWave) {
        const int r = j / kCols, col = j % kCols;
        if (col0 + col >= a.N) continue;
        const float v = lds[r * kPitch + col];
        const size_t at = (size_t)(m0 + first + r) * a.out_stride + col0 + col;
        if (a.out_dtype == MOE_F32) static_cast<float*>(a.out)[at] = v;
        else if (a.out_dtype == MOE_BF16) static_cast<__bf16*>(a.out)[at] = (__bf16)v;
        else static_cast<_Float16*>(a.out)[at] = (_Float16)v;
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <class R, int WM, int WN, int NW, int NX, bool TAIL, int MODE>
__device__ __forceinline__ void tile(const R& ring, const GemmArgs& a, int e, int n0, int m0, int rows) {
  typedef Tile<R, WM, WN, NW, NX, TAIL, MODE> T;
  typedef WaveLds<R, WM * WN> Lds;
  T c;
  c.init(ring, a, e, n0, m0, rows);
  c.run();
  lds_float* lds = Lds::of(ring, c.wave);
  if constexpr (MODE == kGateUp) {
    static_assert(Lds::kBytes >= 32 * kWave * 4, "a block's gate and up sums");
    gateup_epilogue(c, a, n0, m0, rows, lds);
  } else {
    static_assert(Lds::kBytes >= 32 * (32 * NW + 4) * 4, "32 rows of the wave's outputs");
    rows_epilogue<T, MODE>(c, a, n0, m0, rows, lds);
  }
}

// Workgroups are dealt to the 8 XCDs round robin. Each XCD has a run of the tile list, whose
// tiles of one expert are neighbours, and takes a tile's column tiles one after another: the
// tiles of an expert then read its weights, and a tile's workgroups its rows of x, through one
// L2. (Gate and up of 8192 tokens 282 us dealt out tile by tile, 267 in runs; of 256 tokens, whose
// experts have one tile each, 162 and 161.)
constexpr int kXcds = kMxXcds;

__device__ __forceinline__ bool list_tile(const int* xcd_first, int ntn, int& mt, int& nt) {
  const int x = (int)blockIdx.x % kXcds, slot = (int)blockIdx.x / kXcds;
  mt = load_uniform(xcd_first + x) + slot / ntn;
  nt = slot % ntn;
  return mt < load_uniform(xcd_first + x + 1);
}

// Linear: an XCD has a rectangle of tiles and takes it in panels, so that the workgroups that
// run at once share rows and columns about evenly.
__device__ __forceinline__ bool grid_tile(const GemmArgs& a, int mtiles, int ntiles, int& mt, int& nt) {
  const int x = (int)blockIdx.x % kXcds;
  int slot = (int)blockIdx.x / kXcds;
  const int per = a.xcd_rm * a.panel, p = slot / per;
  slot -= p * per;
  const int width = min(a.panel, a.xcd_rn - p * a.panel);
  mt = x % a.xcd_m * a.xcd_rm + slot / width;
  nt = x / a.xcd_m * a.xcd_rn + p * a.panel + slot % width;
  return mt < mtiles && nt < ntiles;
}

// The grouped product: 256 weight rows by up to 128 pairs, two workgroups a CU (80 KB of LDS), one's
// start and end beside the other's loop. Few rows an expert: bound by the weights from memory.
// Many: by the direct loads (without them 180 of 260 us, without the LDS reads 255, without the
// end 250). Stages of whole lines would need 128 x 128 tiles (10% slower at 256 and at 8192
// tokens) or one workgroup of 256 x 256 a CU (15% slower at 256 tokens, 1% at 8192). The down form
// with a TAIL (f no multiple of 256) keeps 4 of its 256 registers in scratch memory: 4096 tokens of
// 64 experts, top 6, d = 2048, 104-110 us at f = 1408 and 93-102 at f = 1536.
template <bool TAIL, int MODE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_mx_grouped(GemmArgs a) {
  typedef Stage<256, 128, 4> S;
  typedef ScaleRing<256, 128, 2> SC;
  __shared__ S slot0, slot1, slot2;
  __shared__ SC scales;
  const Slots<S, SC, 3> ring{&slot0, &slot1, &slot2, nullptr, &scales};
  constexpr int kN = MODE == kGateUp ? 128 : 256;  // rows of f, or of d, a workgroup
  const int ntn = (a.N + kN - 1) / kN;
  int mt, nt;
  if (!list_tile(a.xcd_first, ntn, mt, nt)) return;
  const int4 t = load_uniform(a.tiles + mt);
  if (MODE == kGateUp && nt == 0 && (int)threadIdx.x < t.z)
    a.place[a.pair_index[t.y + threadIdx.x]] = t.y + threadIdx.x;
  if (t.z <= 32)
    tile<Slots<S, SC, 3>, 1, 4, 2, 1, TAIL, MODE>(ring, a, t.x, nt * kN, t.y, t.z);
  else if (t.z <= 64)
    tile<Slots<S, SC, 3>, 1, 4, 2, 2, TAIL, MODE>(ring, a, t.x, nt * kN, t.y, t.z);
  else
    tile<Slots<S, SC, 3>, 1, 4, 2, 4, TAIL, MODE>(ring, a, t.x, nt * kN, t.y, t.z);
}

// The dense product: stages of whole lines, two slots. Of the 256 x 256 tile's 0.95 us per 128
// values, the matrix instructions need 0.76 (without loads and LDS reads); a tile's start and end
// cost 8 us (2 the start, 2 the rows' way through LDS, 4 their stores), since it takes all of a
// CU's LDS and nothing runs beside it. The smallest tile, which
// runs where there are few, has room for four slots; it takes them where the scales' requests,
// one a stage with a TAIL, stand between the codes' (517 rows by 1441 by 2080 columns 10.4 -> 9.8
// us; without a TAIL 64 x 5120 x 2048 5.8 -> 6.2).
template <int WM, int WN, int NW, int NX, bool TAIL>
__global__ __launch_bounds__(kWave * WM * WN) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_mx_linear(
    GemmArgs a) {
  constexpr int BN = 32 * NW * WN, BM = 32 * NX * WM;
  typedef Stage<BN, BM, 8> S;
  typedef ScaleRing<BN, BM, TAIL ? 2 : 4> SC;
  constexpr bool kDeep = TAIL && BN + BM <= 128;
  typedef Slots<S, SC, kDeep ? 4 : 2> R;
  __shared__ S slot0, slot1;
  __shared__ SC scales;
  R ring{&slot0, &slot1, nullptr, nullptr, &scales};
  if constexpr (kDeep) {
    __shared__ S slot2, slot3;
    ring.s2 = &slot2;
    ring.s3 = &slot3;
  }
  const int ntn = (a.N + BN - 1) / BN;
  int mt, nt;
  if (!grid_tile(a, (a.rows + BM - 1) / BM, ntn, mt, nt)) return;
  tile<R, WM, WN, NW, NX, TAIL, kLinear>(ring, a, 0, nt * BN, mt * BM, min(BM, a.rows - mt * BM));
}

// ---------------------------------------------------------------- work list

// Inclusive scan over the workgroup (1024 threads) of two values at once.
__device__ __forceinline__ int2 block_scan(int2 v, int2* wsum) {
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int a = __shfl_up(v.x, off), b = __shfl_up(v.y, off);
    if (lane >= off) v.x += a, v.y += b;
  }
  if (lane == kWave - 1) wsum[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v.x += wsum[w].x, v.y += wsum[w].y;
  __syncthreads();
  return v;
}

// One workgroup of 1024: tiles in expert order, and the XCDs' shares of their cost. A thread finds
// an expert's first tile; then the threads write the tiles, each looking its expert up.
__device__ __forceinline__ void list_tiles(const int32_t* __restrict__ offsets, int E,
                                           int4* __restrict__ tiles, int* __restrict__ xcd_first) {
  __shared__ int2 s_wsum[16];
  __shared__ int s_first[1024], s_cost[1024], s_beg[1025];
  __shared__ int2 s_total;
  const int tid = threadIdx.x;
  const int beg = offsets[min(tid, E)];
  const int m = tid < E ? offsets[tid + 1] - beg : 0;
  const int count = (m + kMxBM - 1) / kMxBM;
  const int2 mine = make_int2(count, mx_tiles_cost(count, m));
  const int2 incl = block_scan(mine, s_wsum);
  s_first[tid] = incl.x - mine.x;
  s_cost[tid] = incl.y - mine.y;
  s_beg[tid] = beg;
  if (tid == 1023) s_total = incl, s_beg[1024] = offsets[E];
  __syncthreads();
  const int ntiles = s_total.x, total = s_total.y;
  for (int j = tid; j < ntiles; j += 1024) {
    int lo = 0, hi = E - 1;  // the last expert whose first tile is not behind j
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (s_first[mid] <= j) lo = mid;
      else hi = mid - 1;
    }
    const int i = j - s_first[lo], g0 = s_beg[lo] + i * kMxBM;
    const int rows = min(kMxBM, s_beg[lo + 1] - g0);
    tiles[j] = make_int4(lo, g0, rows, 0);
    const int cost = s_cost[lo] + mx_tiles_cost(i, i * kMxBM);
    mx_xcd_starts(j, cost, cost + mx_tiles_cost(1, rows), total, xcd_first);
  }
  if (tid <= kXcds && (tid == kXcds || ntiles == 0)) xcd_first[tid] = ntiles;
}

// What the grouped products need first: the first workgroup lists the tiles (5 us, one latency
// after another) while the others quantize the rows.
constexpr int kPrepareThreads = 1024;

template <int DT, bool STRIDED>
__global__ __launch_bounds__(kPrepareThreads) void k_mx_prepare(const char* __restrict__ x, int64_t words,
                                                                int row_words, int64_t row_bytes,
                                                                uint32_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales,
                                                                const int32_t* __restrict__ offsets, int E,
                                                                int4* __restrict__ tiles,
                                                                int* __restrict__ xcd_first) {
  if (blockIdx.x == 0)
    list_tiles(offsets, E, tiles, xcd_first);
  else
    mx_quantize_words<DT, STRIDED, kPrepareThreads>(x, words, row_words, row_bytes, codes, scales,
                                                    (int64_t)blockIdx.x - 1);
}

// ---------------------------------------------------------------- combine

// Reads y once, sixteen slots' words in flight a thread: 5.1 TB/s. y lies in the order of the
// grouped pairs: rows stored to the places of their tokens cost the down product of 8192 tokens 40
// us more, and reading them from there nothing.
constexpr int kCombineBatch = 16;

__global__ __launch_bounds__(1024) void k_mx_combine(const float* __restrict__ y, const int32_t* __restrict__ place,
                                                     const int32_t* __restrict__ ids,
                                                     const float* __restrict__ w, int E, int d, int k,
                                                     const float* residual, float* out) {
  const int t = blockIdx.x, P = gridDim.x * k, lane = threadIdx.x & (kWave - 1);
  // lane j: weight and row of slot j. A pair of no expert has no place and adds nothing.
  const size_t pair = (size_t)t * k + min(lane, k - 1);
  const bool in = (unsigned)ids[pair] < (unsigned)E;
  const int my_row = min((unsigned)place[pair], (unsigned)(P - 1));
  const int row_of = in ? my_row : -1;
  const float my_w = in ? w[pair] : 0.0f;
  // Every lane stays in the loop, since any may hold a slot: lanes past d read its last columns.
  for (int c0 = 0; c0 < d; c0 += 4 * blockDim.x) {
    const int c = min(c0 + 4 * (int)threadIdx.x, d - 4);
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    for (int j0 = 0; j0 < k; j0 += kCombineBatch) {
      mx_f32x4 v[kCombineBatch];
#pragma unroll
      for (int i = 0; i < kCombineBatch; ++i)
        if (j0 + i < k) {
          const int g = __builtin_amdgcn_readlane(row_of, j0 + i);
          v[i] = mx_f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          if (g >= 0)
            v[i] = __builtin_nontemporal_load(reinterpret_cast<const mx_f32x4*>(y + (size_t)g * d + c));
        }
#pragma unroll
      for (int i = 0; i < kCombineBatch; ++i)
        if (j0 + i < k) {
          const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(my_w), j0 + i));
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[q] += (double)wj * (double)v[i][q];
        }
    }
    const size_t at = (size_t)t * d + c;
    mx_f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
    if (residual) r = *reinterpret_cast<const mx_f32x4*>(residual + at);
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = (float)((double)r[q] + acc[q]);
    if (c0 + 4 * (int)threadIdx.x < d) *reinterpret_cast<mx_f32x4*>(out + at) = r;
  }
}

// Splits the tiles over the XCDs: the split that leaves the largest share smallest, of those the
// one whose shares are the most square.
template <int WM, int WN, int NW, int NX>
void linear(GemmArgs g, hipStream_t stream) {
  constexpr int BN = 32 * NW * WN, BM = 32 * NX * WM;
  const int mt = (g.rows + BM - 1) / BM, nt = (g.N + BN - 1) / BN;
  long long best = 0, border = 0;
  for (int m = 1; m <= kXcds; m *= 2) {
    const long long rm = (mt + m - 1) / m, rn = (nt + kXcds / m - 1) / (kXcds / m);
    if (best == 0 || rm * rn < best || (rm * rn == best && rm * BM + rn * BN < border)) {
      best = rm * rn;
      border = rm * BM + rn * BN;
      g.xcd_m = m;
      g.xcd_rm = (int)rm;
      g.xcd_rn = (int)rn;
    }
  }
  // about 32 workgroups of an XCD run at once
  g.panel = std::max(1, std::min(g.xcd_rn, (32 + g.xcd_rm - 1) / g.xcd_rm));
  const dim3 grid((unsigned)(kXcds * best)), block(kWave * WM * WN);
  if (g.K % 512 == 0)
    hipLaunchKernelGGL((k_mx_linear<WM, WN, NW, NX, false>), grid, block, 0, stream, g);
  else
    hipLaunchKernelGGL((k_mx_linear<WM, WN, NW, NX, true>), grid, block, 0, stream, g);
}

}  // namespace

hipError_t launch_mx_linear(const MxLinearArgs& a, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  if (mx_linear_window(a.n, a.N, a.K)) return launch_mx_linear_window(a, stream);
  GemmArgs g{};
  g.w0 = a.w;
  g.s0 = a.ws;
  g.xq = a.xq;
  g.xs = a.xs;
  g.rows = a.n;
  g.wrows = a.N;
  g.xrows = a.n;
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
  // The largest tile that still gives most CUs one: a tile twice as large needs half the loads
  // and LDS reads a product. Measured (us, K = 2048; tiles 64x64, 64x128, 128x128, 128x256,
  // 256x256, rows of x first):  256 x 4096: 6.5 7.6 9.7 12.7 16.4;  1024 x 2048: 8.4 8.4 10.4
  // 12.9 17.0;  2048 x 2048: 14.1 12.4 11.7 14.0 17.9;  1024 x 5120: 18.0 16.0 15.4 14.8 18.8;
  // 4096 x 4096: 50.2 36.6 29.2 30.2 24.1.
  const int most = device_cu_count() * 5 / 8;
  auto tiles = [&](int rows, int cols) { return (long long)((a.n + rows - 1) / rows) * ((a.N + cols - 1) / cols); };
  if (tiles(256, 256) >= most) linear<2, 4, 2, 4>(g, stream);
  else if (tiles(128, 256) >= most) linear<2, 4, 2, 2>(g, stream);
  else if (tiles(128, 128) >= most) linear<2, 2, 2, 2>(g, stream);
  else if (tiles(64, 128) >= most) linear<1, 4, 1, 2>(g, stream);
  else linear<2, 2, 1, 1>(g, stream);
  return hipGetLastError();
}

hipError_t launch_mx_ffn(const MxFfnArgs& a, hipStream_t stream) {
  const moe_mx_layer& L = *a.L;
  const int n = a.n, d = L.d_model, f = L.d_ff, k = L.top_k, E = L.n_experts, P = n * k;
  if (P == 0) return hipSuccess;
  if (mx_window(n, k, d, f, E)) return launch_mx_ffn_window(a, stream);
  const MxFfnWs W = mx_ffn_ws(n, k, d, f, E);
  uint8_t* xq = reinterpret_cast<uint8_t*>(a.work + W.xq);
  uint8_t* xs = reinterpret_cast<uint8_t*>(a.work + W.xs);
  uint8_t* hq = reinterpret_cast<uint8_t*>(a.work + W.hq);
  uint8_t* hs = reinterpret_cast<uint8_t*>(a.work + W.hs);
  float* y = reinterpret_cast<float*>(a.work + W.y);
  int4* tiles = reinterpret_cast<int4*>(a.work + W.tiles);
  int* xcd_first = reinterpret_cast<int*>(a.work + W.xcd_first);
  {
    const int64_t words = (int64_t)n * (d / 8);
    const int share = kPrepareThreads * kMxQuantUnroll;
    const bool strided = n > 1 && a.row_stride != d;
    auto kern = a.dtype == MOE_BF16  ? (strided ? k_mx_prepare<MOE_BF16, true> : k_mx_prepare<MOE_BF16, false>)
                : a.dtype == MOE_F16 ? (strided ? k_mx_prepare<MOE_F16, true> : k_mx_prepare<MOE_F16, false>)
                                     : (strided ? k_mx_prepare<MOE_F32, true> : k_mx_prepare<MOE_F32, false>);
    hipLaunchKernelGGL(kern, dim3((unsigned)((words + share - 1) / share + 1)), dim3(kPrepareThreads), 0, stream,
                       static_cast<const char*>(a.x), words, d / 8, a.row_stride * mx_type_size(a.dtype),
                       reinterpret_cast<uint32_t*>(xq), xs, a.r->expert_offsets, E, tiles, xcd_first);
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;

  const int max_mt = mx_max_mtiles(P, E);
  GemmArgs g{};
  g.pair_index = a.r->pair_index;
  g.place = reinterpret_cast<int32_t*>(a.work + W.place);
  g.tiles = tiles;
  g.xcd_first = xcd_first;
  g.k = k;
  g.w0 = L.gate.codes;
  g.s0 = L.gate.scales;
  g.w1 = L.up.codes;
  g.s1 = L.up.scales;
  g.xq = xq;
  g.xs = xs;
  g.N = f;
  g.K = d;
  g.wrows = (int64_t)E * f;
  g.xrows = n;
  g.hq = hq;
  g.hs = hs;
  const dim3 gu(mx_list_grid(max_mt, (f + 127) / 128));
  if (d % 256 == 0)
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
  g.wrows = (int64_t)E * d;
  g.xrows = P;
  g.out = y;
  const dim3 dn(mx_list_grid(max_mt, (d + 255) / 256));
  if (f % 256 == 0)
    hipLaunchKernelGGL((k_mx_grouped<false, kDown>), dn, dim3(kThreads), 0, stream, g);
  else
    hipLaunchKernelGGL((k_mx_grouped<true, kDown>), dn, dim3(kThreads), 0, stream, g);
  err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int threads = std::min(1024, ((d / 4 + kWave - 1) / kWave) * kWave);
  hipLaunchKernelGGL(k_mx_combine, dim3(n), dim3(threads), 0, stream, y, g.place, a.r->topk_ids, a.r->topk_w, E, d, k, a.residual,
                     a.out);
  return hipGetLastError();
}

}  // namespace qmoe
