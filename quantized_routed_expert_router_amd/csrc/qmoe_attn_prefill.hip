// Causal attention of prompt chunks over the paged cache, with an optional sliding window
// and first keys that stay visible.
//
// The rows of one sequence and one kv head are (token, query head of the group), token
// outermost, so that all heads of a group share each key tile and the causal edge stays
// narrow. A workgroup takes 32 rows a wave; key tiles of KT keys go through LDS, in four
// buffers with 8 waves and two with 4, and every wave runs, on 32x32x16 matrix-core tiles,
//   S^T = K Q^T        A: 8 columns of one key row a lane (LDS rows, 16-byte chunks swizzled
//                      by the row so that 16 rows cover all banks); Q stays in registers
//   O^T += V^T P^T     A: 8 keys of one column a lane, one 16-byte word of the cache's V
//                      layout, copied to LDS as it is
// The key rows of a 32-key half are dealt to the first product's rows (bits 2 and 3
// exchanged) so that its accumulators 8u..8u+7 of a lane are 8 consecutive keys, which is
// the second product's B operand: probabilities never leave the lane. Statistics and sums
// are fp32; probabilities are rounded to the 16-bit type for the matrix cores (in bf16 by up
// to 2^-8 of each, in fp16 by 2^-11, or 2^-36 of the row's largest where that is more: the
// output's own rounding is as large; a second part as in decode would double the products of
// a loop that they bound).
#include <type_traits>

#include "qmoe_attn_plan.h"

namespace qmoe {
namespace {

[[maybe_unused]] constexpr int kTileElems = 8192;  // keys x columns of one LDS tile: 16 KB each of keys and values

struct PrefillParams {
  HeadView q;
  const char* ck;
  const char* cv;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  long long table_stride;
  char* out;
  float* partial;
  float2* stats;
  float scale;  // times log2(e)
  KeyMask mask;
  int num_pages, page_shift, kv_heads, max_pages;
  int n, n_seqs, group, splits, slots;
};

// Sequence s has the row-tile slots floor(q_starts[s] * group / BM) + s up to the next
// sequence's: enough for its own tiles, found without a prefix sum. The values are held
// inside [0, n] whatever the array says.
__device__ __forceinline__ int q_start(const PrefillParams& p, int s) {
  return max(0, min(p.q_starts[s], p.n));
}

template <int BM>
__device__ __forceinline__ int first_slot(const PrefillParams& p, int s) {
  return (int)((long long)q_start(p, s) * p.group / BM) + s;
}

// One row tile: rows row0 .. row0 + BM - 1 of sequence seq (fewer at its end).
struct RowTile {
  int seq, start, rows, row0, first_pos, len;  // first_pos: of the sequence's first token
  TileList keys;
  int per, live;
};

template <int BM, int KT>
__device__ __forceinline__ RowTile row_tile(const PrefillParams& p, int seq, int tile) {
  RowTile t;
  t.seq = seq;
  t.start = q_start(p, seq);
  const int m = max(0, q_start(p, seq + 1) - t.start);
  t.rows = m * p.group;
  t.row0 = tile * BM;
  const long long cap = (long long)p.max_pages << p.page_shift;
  t.len = (int)max(0ll, min((long long)p.kv_lens[seq], cap));
  t.first_pos = t.len - m;
  const int a = t.first_pos + t.row0 / p.group;
  const int b = t.first_pos + (min(t.row0 + BM, t.rows) - 1) / p.group;
  t.keys = visible_tiles<KT>(p.mask, a, b);
  t.per = max(kMinSplitKeys / KT, (t.keys.count + p.splits - 1) / p.splits);
  t.live = (t.keys.count + t.per - 1) / t.per;
  return t;
}

// 8 waves are taken when row tiles fill the card by themselves, so they never split the keys.
template <int NW>
constexpr bool kWhole = NW == 8;

#if defined(__HIP_DEVICE_COMPILE__)

// The last sequence s for which at_or_before(s, q_starts[s]) holds (it does for a first part
// of them), -1 if none: one load by the wave for up to 64 sequences, a binary search beyond.
template <typename F>
__device__ __forceinline__ int find_sequence(const PrefillParams& p, F at_or_before) {
  if (p.n_seqs <= kWave) {
    const int s = min((int)threadIdx.x % kWave, p.n_seqs - 1);
    const uint64_t before = __builtin_amdgcn_ballot_w64(at_or_before(s, q_start(p, s)));
    const uint64_t mine = p.n_seqs == kWave ? before : before & ((1ull << p.n_seqs) - 1);
    return mine == 0 ? -1 : 63 - __builtin_clzll(mine);
  }
  int seq = -1;
  for (int lo = 0, hi = p.n_seqs - 1; lo <= hi;) {
    const int mid = (lo + hi) / 2;
    if (at_or_before(mid, q_start(p, mid))) {
      seq = mid;
      lo = mid + 1;
    } else {
      hi = mid - 1;
    }
  }
  return seq;
}

template <int D>
__device__ __forceinline__ int key_swizzle(int row) {
  return D == 64 ? (row >> 1) & 7 : row & 15;
}

// A thread's part of one key tile on its way from the cache to LDS.
template <typename A, int D, bool F8, int KT, int THREADS>
struct Stage {
  static constexpr int PER_CHUNK = F8 ? 16 : 8;  // elements of a 16-byte chunk
  static constexpr int COLS = D / PER_CHUNK;     // chunks of a key row
  static constexpr int N = KT * D / PER_CHUNK / THREADS;
  static_assert(KT * D / PER_CHUNK % THREADS == 0, "whole chunks");
  static constexpr int BLOCK = F8 ? D / 2 : D;  // chunks of a group of 8 value rows
  u32x4 k[N], v[N];
  int kid[N], vid[N];  // page numbers

  __device__ __forceinline__ int page_of(const PrefillParams& p, const int32_t* table, int key) {
    return table[min(key >> p.page_shift, p.max_pages - 1)];
  }
  __device__ __forceinline__ void ids(const PrefillParams& p, const int32_t* table, int key0,
                                      int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = tid + i * THREADS;
      kid[i] = page_of(p, table, key0 + c / COLS);
      vid[i] = page_of(p, table, key0 + 8 * (c / BLOCK));
    }
  }
  __device__ __forceinline__ long long row_of(const PrefillParams& p, int id, int kvh, int key) {
    const long long page = (unsigned)id < (unsigned)p.num_pages ? id : 0;
    return ((page * p.kv_heads + kvh) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
  }
  __device__ __forceinline__ void load(const PrefillParams& p, int kvh, int key0, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = tid + i * THREADS;
      const long long kr = row_of(p, kid[i], kvh, key0 + c / COLS);
      k[i] = *reinterpret_cast<const u32x4*>(p.ck + kr * (D * (F8 ? 1 : 2)) + 16 * (c % COLS));
      const long long vr = row_of(p, vid[i], kvh, key0 + 8 * (c / BLOCK));
      v[i] = *reinterpret_cast<const u32x4*>(p.cv + vr * (D * (F8 ? 1 : 2)) + 16 * (c % BLOCK));
    }
  }
  // Leaves the non-finite values of the tile out; whether there were any.
  __device__ __forceinline__ bool clear_values() {
    bool any = false;
#pragma unroll
    for (int i = 0; i < N; ++i) any |= clear_word<A, F8>(v[i]);
    return any;
  }
  __device__ __forceinline__ void store(u32x4* lk, u32x4* lv, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = tid + i * THREADS;
      const int row = c / COLS, col = c % COLS, sw = key_swizzle<D>(row);
      if constexpr (F8) {
        lk[row * (D / 8) + ((2 * col) ^ sw)] = bits_as<u32x4>(expand_e4m3<A>(k[i][0], k[i][1]));
        lk[row * (D / 8) + ((2 * col + 1) ^ sw)] =
            bits_as<u32x4>(expand_e4m3<A>(k[i][2], k[i][3]));
        lv[2 * c] = bits_as<u32x4>(expand_e4m3<A>(v[i][0], v[i][1]));
        lv[2 * c + 1] = bits_as<u32x4>(expand_e4m3<A>(v[i][2], v[i][3]));
      } else {
        lk[row * (D / 8) + (col ^ sw)] = k[i];
        lv[c] = v[i];
      }
    }
  }
};

#endif  // __HIP_DEVICE_COMPILE__

// Bound by the matrix cores and the vector unit, which the two waves of a SIMD use in turn: a
// tile's products and its exponentials, maxima and rounding cost about the same. 8192 tokens,
// 32 query and 8 kv heads of 128, bf16: 592-628 us, 875-929 TFLOP/s (a large library product
// reaches 1260); 4096 tokens of 16 heads of 256: 290-317 us, 434-474 TFLOP/s, one wave a SIMD.
template <typename A, int D, bool F8, int NW>
__global__ __launch_bounds__(64 * NW, D == 256 ? 1 : 2) void k_attn_prefill(PrefillParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef typename A::V8 V8;
  constexpr int KT = kTileElems / D, BM = 32 * NW, THREADS = 64 * NW;
  constexpr int KS = D / 16, DT = D / 32, HALVES = KT / 32;
  constexpr int STEP = NW == 8 ? 2 : 1, BUFS = 2 * STEP;  // tiles between barriers
  __shared__ u32x4 lk[BUFS][KT * D / 8], lv[BUFS][KT * D / 8];
  __shared__ int dirty[BUFS][NW];  // an edge tile had non-finite values in a wave's part

  // Workgroups go to the 8 XCDs in turn: with the kv head in the low digits, an XCD's
  // workgroups share few heads' keys in its L2. Later row tiles see more keys: they start
  // first.
  const int kvh = blockIdx.x % p.kv_heads;
  const int slot = p.slots - 1 - blockIdx.x / p.kv_heads;
  const int seq = find_sequence(p, [&](int s, int start) {
    return (int)((long long)start * p.group / BM) + s <= slot;
  });
  if (seq < 0) return;
  const int index = slot - first_slot<BM>(p, seq);
  const RowTile t = row_tile<BM, KT>(p, seq, index);
  if ((long long)index * BM >= t.rows) return;
  const int split = blockIdx.y;
  const bool direct = kWhole<NW> || t.live <= 1;
  if (split >= t.live && !(direct && split == 0)) return;
  const int i0 = split * t.per, i1 = min(i0 + t.per, t.keys.count);

  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int n32 = lane & 31, h = lane >> 5;
  const int32_t* table = p.table + seq * p.table_stride;
  const int hq = p.kv_heads * p.group;

  // this lane's query row
  const int wrow = t.row0 + 32 * wave;  // the wave's first row
  const bool real = wrow + n32 < t.rows;
  const int row = real ? wrow + n32 : t.row0;
  const int token = t.start + row / p.group, head = kvh * p.group + row % p.group;
  const int pos = real ? t.first_pos + row / p.group : -1;
  const bool any = wrow < t.rows;
  const int pos_min = t.first_pos + wrow / p.group;
  const int pos_max = t.first_pos + (min(wrow + 32, t.rows) - 1) / p.group;
  const int first_key = t.first_pos + t.row0 / p.group;  // positions of the workgroup's rows
  const int last_key = t.first_pos + (min(t.row0 + BM, t.rows) - 1) / p.group;
  // the last keys behind the windows of the wave's first and last rows, of the workgroup's last
  const int low_min = behind_window(p.mask, pos_min), low_max = behind_window(p.mask, pos_max);
  const int low_last = behind_window(p.mask, last_key);
  auto visible = [&](int key, bool bad_tile) {
    bool ok = key_visible(p.mask, key, pos);
    if (bad_tile && ok) ok = (unsigned)table[key >> p.page_shift] < (unsigned)p.num_pages;
    return ok;
  };

  const ScaleSplit sc = split_scale(p.scale * (p.k_scale ? p.k_scale[kvh] : 1.0f));
  V8 q[KS];
  {
    const char* src = p.q.data + 2 * ((long long)token * p.q.token_stride +
                                      (long long)head * p.q.head_stride);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      u32x4 w = *reinterpret_cast<const u32x4*>(src + 2 * (16 * ks + 8 * h));
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = real ? (w[i] ^ sc.flip) & sc.keep : 0u;
      q[ks] = bits_as<V8>(w);
    }
  }

  f32x16 o[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[dt][r] = 0.0f;
  float m = kNegInf, l = 0.0f;  // scaled reference maximum; this lane's part of the sum

  Stage<A, D, F8, KT, THREADS> st;
  // An edge tile: not all of the workgroup's rows see all of it.
  auto is_edge = [&](bool bad_tile, int key0) {
    return bad_tile || key0 + KT - 1 > first_key ||
           (key0 <= low_last && key0 + KT - 1 >= p.mask.sinks);
  };
  auto stage_store = [&](int buf, bool edge_tile) {
    if (edge_tile) {
      const bool any = __builtin_amdgcn_ballot_w64(st.clear_values()) != 0;
      if (lane == 0) dirty[buf][wave] = any;
    }
    st.store(lk[buf], lv[buf], tid);
  };
  // Tile i0 + j lies in buffer j % BUFS. While tile j is worked on, tile j + STEP is loaded;
  // it goes to a buffer that was last read before the last barrier.
  int flags = 0;  // bits 2 (j % BUFS), + 1: tile j is bad, an edge tile
  auto note = [&](int j, int key0, int pages) {
    const bool bad_tile =
        __builtin_amdgcn_ballot_w64((unsigned)pages >= (unsigned)p.num_pages) != 0;
    const bool edge_tile = is_edge(bad_tile, key0);
    const int at = 2 * (j & (BUFS - 1));
    flags = (flags & ~(3 << at)) | (bad_tile ? 1 << at : 0) | (edge_tile ? 2 << at : 0);
    return edge_tile;
  };
  // The tile's page numbers up to the last key that any row sees, one a lane. (Scalar loads
  // would share their counter with the LDS reads and wait for both.)
  auto tile_pages = [&](int j) {
    const int first = t.keys.tile(min(i0 + j, i1 - 1)) * KT >> p.page_shift;
    return table[min(first + min(lane, (KT - 1) >> p.page_shift), last_key >> p.page_shift)];
  };
  const int count = i1 - i0;
  int pages = 0;  // of the next tile to load
  if (count > 0) {
    st.ids(p, table, t.keys.tile(i0) * KT, tid);
    pages = tile_pages(0);
  }
#pragma unroll
  for (int j = 0; j < STEP; ++j) {
    if (j >= count) continue;
    const int key0 = t.keys.tile(i0 + j) * KT;
    st.load(p, kvh, key0, tid);
    if (j + 1 < count) st.ids(p, table, t.keys.tile(i0 + j + 1) * KT, tid);
    const bool edge_tile = note(j, key0, pages);
    pages = tile_pages(j + 1);
    stage_store(j, edge_tile);
  }
  lds_barrier();
#pragma unroll 1
  for (int j = 0; j < count; ++j) {
    const int buf = j & (BUFS - 1);
    const int key0 = t.keys.tile(i0 + j) * KT;
    const bool bad = flags >> (2 * buf) & 1, edge = flags >> (2 * buf) & 2;
    const bool more = j + STEP < count;
    bool edge_next = false;
    if (more) {
      const int k1 = t.keys.tile(i0 + j + STEP) * KT;
      st.load(p, kvh, k1, tid);
      edge_next = note(j + STEP, k1, pages);
      pages = tile_pages(j + STEP + 1);
      if (j + STEP + 1 < count) st.ids(p, table, t.keys.tile(i0 + j + STEP + 1) * KT, tid);
    }
    const bool sees = any && key0 <= pos_max &&
                      (key0 + KT - 1 > low_min || key0 < p.mask.sinks);
    if (sees) {
      f32x16 s[HALVES];
      const int krow = (n32 & 19) | ((n32 & 4) << 1) | ((n32 & 8) >> 1);
#pragma unroll
      for (int x = 0; x < HALVES; ++x) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[x][r] = 0.0f;
        const int kr = 32 * x + krow, sw = key_swizzle<D>(kr);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const V8 a = bits_as<V8>(lk[buf][kr * (D / 8) + ((2 * ks + h) ^ sw)]);
          s[x] = A::mfma32(a, q[ks], s[x]);
        }
      }
      // accumulator r of half x is key 32 x + 16 (r / 8) + 8 h + r % 8
      if (edge && (bad || key0 + KT - 1 > pos_min || key0 <= low_max)) {
#pragma unroll
        for (int x = 0; x < HALVES; ++x)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (!visible(key0 + 32 * x + 16 * (r >> 3) + 8 * h + (r & 7), bad)) s[x][r] = kNegInf;
      }
      float top = kNegInf;
#pragma unroll
      for (int x = 0; x < HALVES; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[x][r]);
      top = fmaxf(top, __shfl_xor(top, 32)) * sc.scale;
      const bool moves = top > m + A::kLazy;
      if (__builtin_amdgcn_ballot_w64(moves) != 0) {
        const float now = moves ? top : m;
        const float a = rescale(m - (now == kNegInf ? 0.0f : now));
        l *= a;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[dt] *= a;
        m = now;
      }
      const float base = exponent_base<A>(m);
      V8 pr[2 * HALVES];
#pragma unroll
      for (int x = 0; x < HALVES; ++x) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[x][r] = exp2_fast(__builtin_fmaf(s[x][r], sc.scale, base));
          l += s[x][r];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          f32x8 y;
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = s[x][8 * u + j];
          pr[2 * x + u] = __builtin_convertvector(y, V8);
        }
      }
#pragma unroll
      for (int ks = 0; ks < 2 * HALVES; ++ks)
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
          o[dt] = A::mfma32(bits_as<V8>(lv[buf][(2 * ks + h) * D + 32 * dt + n32]), pr[ks], o[dt]);
      if (edge) {
        int found = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) found |= dirty[buf][w];
        if (found != 0) {
          // the values as the cache has them: what they do to the rows that see them
#pragma unroll 1
          for (int i3 = 0; i3 < 3 * 2 * HALVES; ++i3) {
            const NonFinite kind = non_finite_kind<A>(i3 % 3);
            const int from = key0 + 16 * (i3 / 3) + 8 * h;
            uint32_t seen = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) seen |= (uint32_t)visible(from + j, bad) << j;
            const V8 rows_seen = mask_elements<A>(seen);
            const long long at = st.row_of(p, st.page_of(p, table, from), kvh, from) * D + 8 * n32;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
              V8 a;
              if constexpr (F8) {
                const u32x2 w = *reinterpret_cast<const u32x2*>(p.cv + at + 256 * dt);
                a = expand_e4m3<A>(w[0], w[1]);
              } else {
                a = *reinterpret_cast<const V8*>(p.cv + 2 * (at + 256 * dt));
              }
              f32x16 c;
#pragma unroll
              for (int r = 0; r < 16; ++r) c[r] = 0.0f;
              c = A::mfma32(non_finite<A>(a, kind), rows_seen, c);
#pragma unroll
              for (int r = 0; r < 16; ++r) o[dt][r] += spread(c[r], kind);
            }
          }
        }
      }
    }
    if (more) stage_store((j + STEP) & (BUFS - 1), edge_next);
    if (STEP == 1 || (j & 1)) lds_barrier();
  }

  l += __shfl_xor(l, 32);
  float all = 0.0f;  // NaN where a sum is
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) all += o[dt][r];
  const long long at = (long long)token * hq + head, part = at * p.splits + split;
  const float vs = p.v_scale ? p.v_scale[kvh] : 1.0f;
  const float inv = l == 0.0f ? 0.0f : vs / l;
  if (real && direct) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        f32x4 y;
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = o[dt][4 * r4 + c] * inv;
        *reinterpret_cast<u32x2*>(p.out + 2 * (at * D + 32 * dt + 8 * r4 + 4 * h)) =
            bits_as<u32x2>(__builtin_convertvector(y, typename A::V4));
      }
  } else if (real) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        f32x4 y;
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = o[dt][4 * r4 + c];
        *reinterpret_cast<f32x4*>(p.partial + part * D + 32 * dt + 8 * r4 + 4 * h) = y;
      }
    if (h == 0) p.stats[part] = make_float2(m, l);
  }
  if (__builtin_amdgcn_ballot_w64(real && __builtin_isnan(all)) == 0) return;

  // A value that is not finite takes every row that sees it. But where the 16-bit type holds
  // its key's probability as 0, the products above made NaN of an infinity. So a wave with
  // such sums goes through its values once more, without scores, 32 columns at a time, and
  // writes the columns of the rows that see one again.
#pragma unroll 1
  for (int dt = 0; dt < DT; ++dt) {
    f32x16 c[3];  // counts of each kind
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) c[i][r] = 0.0f;
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
      const int from = t.keys.tile(i0 + j) * KT + 8 * h;
      int id[2 * HALVES];
      u32x4 w[2 * HALVES];
#pragma unroll
      for (int ks = 0; ks < 2 * HALVES; ++ks) id[ks] = st.page_of(p, table, from + 16 * ks);
      bool some = false;
#pragma unroll
      for (int ks = 0; ks < 2 * HALVES; ++ks) {
        const long long word = st.row_of(p, id[ks], kvh, from + 16 * ks) * D + 8 * n32 + 256 * dt;
        if constexpr (F8) {
          const u32x2 x = *reinterpret_cast<const u32x2*>(p.cv + word);
          w[ks] = bits_as<u32x4>(expand_e4m3<A>(x[0], x[1]));
        } else {
          w[ks] = *reinterpret_cast<const u32x4*>(p.cv + 2 * word);
        }
      }
#pragma unroll
      for (int ks = 0; ks < 2 * HALVES; ++ks) {
        V8 finite = bits_as<V8>(w[ks]);
        some |= clear_nonfinite<A>(finite);
      }
      if (__builtin_amdgcn_ballot_w64(some) == 0) continue;
#pragma unroll
      for (int ks = 0; ks < 2 * HALVES; ++ks) {
        uint32_t seen = 0;
        if ((unsigned)id[ks] < (unsigned)p.num_pages) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            seen |= (uint32_t)key_visible(p.mask, from + 16 * ks + k, pos) << k;
        }
        const V8 rows_seen = mask_elements<A>(seen);
#pragma unroll
        for (int i = 0; i < 3; ++i)
          c[i] = A::mfma32(non_finite<A>(bits_as<V8>(w[ks]), non_finite_kind<A>(i)), rows_seen,
                           c[i]);
      }
    }
    if (!real) continue;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float y = 0.0f;
#pragma unroll
      for (int i = 0; i < 3; ++i) y += spread(c[i][r], non_finite_kind<A>(i));
      if (y == 0.0f) continue;
      const int col = 32 * dt + 8 * (r >> 2) + 4 * h + (r & 3);
      if (direct)
        reinterpret_cast<typename A::T*>(p.out)[at * D + col] = (typename A::T)(y * inv);
      else
        p.partial[part * D + col] = y;
    }
  }
#endif
}

// Joins the splits of one (token, query head) row.
template <typename A, int D, int NW>
__global__ __launch_bounds__(kJoinThreads) void k_attn_prefill_join(PrefillParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int KT = kTileElems / D, BM = 32 * NW;
  const int hq = p.kv_heads * p.group;
  const int token = blockIdx.x / hq, head = blockIdx.x % hq;
  const int seq = find_sequence(p, [&](int, int start) { return start <= token; });
  if (seq < 0 || token >= q_start(p, seq + 1)) return;
  const int kvh = head / p.group;
  const int row = (token - q_start(p, seq)) * p.group + head % p.group;
  const RowTile t = row_tile<BM, KT>(p, seq, row / BM);
  if (t.live <= 1) return;  // written by its only split
  join_row<A, D>(p.partial, p.stats, blockIdx.x, p.splits, t.live,
                 p.v_scale ? p.v_scale[kvh] : 1.0f, p.out);
#endif
}

template <typename A, int D, bool F8, int NW>
hipError_t launch_one(const PrefillParams& p, hipStream_t stream) {
  if (kWhole<NW> && p.splits != 1) return hipErrorInvalidValue;
  k_attn_prefill<A, D, F8, NW><<<dim3((unsigned)(p.slots * p.kv_heads), p.splits),
                                 dim3(64 * NW), 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if constexpr (!kWhole<NW>) {
    if (e != hipSuccess || p.splits == 1) return e;
    k_attn_prefill_join<A, D, NW><<<dim3((unsigned)(p.n * p.kv_heads * p.group), D / kJoinCols),
                                    dim3(kJoinThreads), 0, stream>>>(p);
    e = hipGetLastError();
  }
  return e;
}

template <typename A, int D, bool F8>
hipError_t launch_waves(const PrefillParams& p, int nw, hipStream_t stream) {
  if constexpr (D != 256) {
    if (nw == 8) return launch_one<A, D, F8, 8>(p, stream);
  }
  return launch_one<A, D, F8, 4>(p, stream);
}

template <typename A>
hipError_t launch_type(const PrefillParams& p, int D, bool f8, int nw, hipStream_t stream) {
  if (D == 64)
    return f8 ? launch_waves<A, 64, true>(p, nw, stream) : launch_waves<A, 64, false>(p, nw, stream);
  if (D == 128)
    return f8 ? launch_waves<A, 128, true>(p, nw, stream)
              : launch_waves<A, 128, false>(p, nw, stream);
  return f8 ? launch_waves<A, 256, true>(p, nw, stream)
            : launch_waves<A, 256, false>(p, nw, stream);
}

}  // namespace

hipError_t launch_attn_prefill(const AttnArgs& a, const AttnPlan& plan) {
  PrefillParams p{};
  p.q = a.q;
  p.ck = (const char*)a.cache.k;
  p.cv = (const char*)a.cache.v;
  p.k_scale = a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.table = a.pages.table;
  p.kv_lens = a.pages.kv_lens;
  p.q_starts = a.q_starts;
  p.table_stride = a.pages.table_stride;
  p.out = a.out;
  p.partial = (float*)(a.ws + plan.partial);
  p.stats = (float2*)(a.ws + plan.stats);
  p.scale = a.a.scale * kLog2e;
  p.mask = key_mask(a.a);
  p.num_pages = a.cache.num_pages;
  while ((1 << p.page_shift) < a.cache.page_size) ++p.page_shift;
  p.kv_heads = a.cache.kv_heads;
  p.max_pages = a.pages.max_pages;
  p.n = a.n;
  p.n_seqs = a.pages.n_seqs;
  p.group = a.q.heads / a.cache.kv_heads;
  p.splits = plan.splits;
  p.slots = plan.row_tiles;
  const int nw = plan.tile_rows / 32, D = a.cache.head_dim;
  const bool f8 = a.cache.dtype == MOE_E4M3;
  return a.dtype == MOE_BF16 ? launch_type<Bf16>(p, D, f8, nw, a.stream)
                             : launch_type<F16>(p, D, f8, nw, a.stream);
}

}  // namespace qmoe
