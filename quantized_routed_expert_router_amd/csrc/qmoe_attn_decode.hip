// Attention of a decode window (1..16 new tokens a sequence) over the paged cache.
//
// For one sequence and one kv head the window's rows are (token, query head of the group),
// 16 to a matrix-core tile. With 32 keys at a time:
//   S^T = K Q^T        A operand: lane (m, g) holds 8 columns of key row m, straight from
//                      the cache; accumulator: lane (n, g) holds 4 keys of query row n
//   O^T += V^T P^T     A operand: lane (m, g) holds keys 8g..8g+7 of column m, one 16-byte
//                      word of the cache's V layout; B operand: keys 8g..8g+7 of row n
// The key rows of the two 16-key halves are dealt so that lane (n, g)'s 8 scores are keys
// 8g..8g+7: the probabilities leave the first product where the second takes them, and
// nothing goes through LDS until the waves' sums are joined. Softmax statistics and sums
// are fp32; the probabilities enter the second product as a 16-bit value plus the 16-bit
// rest (2^-16 relative and better), which costs matrix-core time that the memory-bound
// loop has to spare.
#include "qmoe_attn_internal.h"

namespace qmoe {
namespace {

constexpr int kThreads = kJoinThreads;
[[maybe_unused]] constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 32;           // keys of one step of a wave
constexpr int kMinSplitTiles = 8;   // 256 keys: below that a split costs more than it saves

struct DecodeParams {
  HeadView q;
  const char* ck;
  const char* cv;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* kv_lens;
  long long table_stride;
  char* out;
  float* partial;  // [token][q head][split][D]
  float2* stats;   // [token][q head][split] (maximum, sum)
  float scale;     // times log2(e)
  KeyMask mask;
  int num_pages, page_shift, kv_heads, max_pages;
  int group, T, splits, row_tiles;
};

// The key tiles of one sequence and how they are dealt to the splits: `per` tiles to each,
// the first `live` of them have any.
struct SeqSplit {
  TileList tiles;
  int len, per, live;
};

__device__ __forceinline__ SeqSplit seq_split(const DecodeParams& p, int seq) {
  SeqSplit s;
  const long long cap = (long long)p.max_pages << p.page_shift;
  s.len = (int)max(0ll, min((long long)p.kv_lens[seq], cap));
  s.tiles = visible_tiles<kTile>(p.mask, s.len - p.T, s.len - 1);
  s.per = max(kMinSplitTiles, (s.tiles.count + p.splits - 1) / p.splits);
  s.live = (s.tiles.count + s.per - 1) / s.per;
  return s;
}

#if defined(__HIP_DEVICE_COMPILE__)

// Where a 32-key tile's two 16-row halves lie: for pages of 32 rows or more both are in
// one page; with 16-row pages each has its own. An entry outside the cache counts as
// invisible (ok false) and reads page 0 instead.
struct TilePages {
  long long base[2];  // row offset (rows of all heads' pages) of each half, head 0
  bool ok[2];
};

__device__ __forceinline__ TilePages tile_pages(const DecodeParams& p, const int32_t* table,
                                                int tile) {
  TilePages t;
  const int row = tile * kTile;
  const int i0 = row >> p.page_shift;
  const int i1 = (row + 16) >> p.page_shift;
  const int id0 = load_uniform(table + i0);
  const int id1 = i1 < p.max_pages ? load_uniform(table + i1) : -1;
  t.ok[0] = (unsigned)id0 < (unsigned)p.num_pages;
  t.ok[1] = (unsigned)id1 < (unsigned)p.num_pages;
  const int in = (1 << p.page_shift) - 1;
  t.base[0] = ((long long)(t.ok[0] ? id0 : 0) * p.kv_heads << p.page_shift) + (row & in);
  t.base[1] = ((long long)(t.ok[1] ? id1 : 0) * p.kv_heads << p.page_shift) + ((row + 16) & in);
  return t;
}

template <typename A, int D, bool F8>
struct KeyRegs {  // one tile of keys: two halves of 16 rows
  static constexpr int N = F8 ? D / 64 : D / 32;
  u32x4 w[2][N];
};
template <typename A, int D, bool F8>
struct ValueRegs {
  static constexpr int N = F8 ? D / 32 : D / 16;
  u32x4 w[N];
};

// Lane (m, g): 8 columns 32 i + 8 g of key row 8 (m / 4) + m % 4 + 4 u; at 8 bits, 16
// columns 64 i + 16 g, two steps of the product.
template <typename A, int D, bool F8>
__device__ __forceinline__ void load_keys(KeyRegs<A, D, F8>& r, const char* ck, const TilePages& t,
                                          long long head, int lane) {
  const int m = lane & 15, g = lane >> 4;
  const int row = 8 * (m >> 2) + (m & 3);
  const long long base = (row & 16 ? t.base[1] : t.base[0]) + head + (row & 15);
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < KeyRegs<A, D, F8>::N; ++i) {
      const long long at = F8 ? (base + 4 * u) * D + 64 * i + 16 * g
                              : ((base + 4 * u) * D + 32 * i + 8 * g) * 2;
      r.w[u][i] = *reinterpret_cast<const u32x4*>(ck + at);
    }
}

// Lane (m, g): keys 8 g .. 8 g + 7 of column 16 i + m; at 8 bits of columns 32 i + 2 m and
// the next.
template <typename A, int D, bool F8>
__device__ __forceinline__ void load_values(ValueRegs<A, D, F8>& r, const char* cv,
                                            const TilePages& t, long long head, int lane) {
  const int m = lane & 15, g = lane >> 4;
  const long long block = (((g & 2 ? t.base[1] : t.base[0]) + head) >> 3) + (g & 1);
#pragma unroll
  for (int i = 0; i < ValueRegs<A, D, F8>::N; ++i) {
    const long long at = F8 ? (block * D + 32 * i + 2 * m) * 8 : (block * D + 16 * i + m) * 16;
    r.w[i] = *reinterpret_cast<const u32x4*>(cv + at);
  }
}

template <typename A, int D, bool F8>
__device__ __forceinline__ typename A::V8 key_step(const KeyRegs<A, D, F8>& r, int u, int ks) {
  if constexpr (F8) {
    const u32x4 w = r.w[u][ks >> 1];
    return ks & 1 ? expand_e4m3<A>(w[2], w[3]) : expand_e4m3<A>(w[0], w[1]);
  } else {
    return bits_as<typename A::V8>(r.w[u][ks]);
  }
}

template <typename A, int D, bool F8>
__device__ __forceinline__ typename A::V8 value_step(const ValueRegs<A, D, F8>& r, int dt) {
  if constexpr (F8) {
    const u32x4 w = r.w[dt >> 1];
    return dt & 1 ? expand_e4m3<A>(w[2], w[3]) : expand_e4m3<A>(w[0], w[1]);
  } else {
    return bits_as<typename A::V8>(r.w[dt]);
  }
}

// Column of accumulator row 4 g + r of column tile dt.
template <bool F8>
__device__ __forceinline__ int out_col(int dt, int row) {
  return F8 ? 32 * (dt >> 1) + 2 * row + (dt & 1) : 16 * dt + row;
}

// Element (key, column) of the tile's values, from the cache.
template <typename A, int D, bool F8>
__device__ __forceinline__ float value_at(const char* cv, const TilePages& t, long long head,
                                          int key, int col) {
  const long long block = (((key & 16 ? t.base[1] : t.base[0]) + head) >> 3) + ((key >> 3) & 1);
  const long long at = (block * D + col) * 8 + (key & 7);
  if constexpr (F8) {
    const uint32_t code = (uint8_t)cv[at];
    return (float)bits_as<typename A::V2>(A::template from_e4m3<false>(code))[0];
  } else {
    return (float)reinterpret_cast<const typename A::T*>(cv)[at];
  }
}

#endif  // __HIP_DEVICE_COMPILE__

template <typename A, int D, bool F8, int NT>
__global__ __launch_bounds__(kThreads) void k_attn_decode(DecodeParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef typename A::V8 V8;
  constexpr int KS = D / 32, DT = D / 16;
  constexpr int DC = D < 128 ? D : 128;  // columns joined at a time
  __shared__ float sums[kWaves][16][DC + 4];
  __shared__ float stat_m[kWaves][16], stat_l[kWaves][16];

  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n16 = lane & 15, g = lane >> 4;
  const int split = blockIdx.x;
  const int kvh = blockIdx.y / p.row_tiles, rt = blockIdx.y % p.row_tiles;
  const int seq = blockIdx.z;
  const SeqSplit sp = seq_split(p, seq);
  const bool direct = sp.live <= 1;
  if (split >= sp.live && !(direct && split == 0)) return;
  const int i0 = split * sp.per, i1 = min(i0 + sp.per, sp.tiles.count);
  const int32_t* table = p.table + seq * p.table_stride;
  const long long head = (long long)kvh << p.page_shift;
  const int first_pos = sp.len - p.T;
  const int rows = p.T * p.group;
  const int hq = p.kv_heads * p.group;

  // this lane's query row of each row tile, as B operand: 8 columns a step
  V8 q[NT][KS];
  int pos[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = (rt * NT + nt) * 16 + n16;
    const int t = row / p.group, h = kvh * p.group + row % p.group;
    const bool real = row < rows;
    pos[nt] = real ? first_pos + t : -1;
    const char* src = p.q.data + 2 * (((long long)seq * p.T + (real ? t : 0)) * p.q.token_stride +
                                      (long long)(real ? h : 0) * p.q.head_stride);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int col = F8 ? 64 * (ks >> 1) + 16 * g + 8 * (ks & 1) : 32 * ks + 8 * g;
      u32x4 w = *reinterpret_cast<const u32x4*>(src + 2 * col);
      if (!real) w = u32x4{0, 0, 0, 0};
      q[nt][ks] = bits_as<V8>(w);
    }
  }
  const float scale = p.scale * (p.k_scale ? p.k_scale[kvh] : 1.0f);

  KeyRegs<A, D, F8> k;
  ValueRegs<A, D, F8> v;
  TilePages here{}, next{};
  f32x4 o[NT][DT];
  float m[NT], l[NT];  // reference maximum of the row; this lane's part of the running sum
  // A second, careful pass runs only where the first one's sums are not all finite: there
  // the split probability's small part would turn a visible infinity into NaN.
  bool careful = false;
again:
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = kNegInf;
    l[nt] = 0.0f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) o[nt][dt] = f32x4{0, 0, 0, 0};
  }

  if (i0 + wave < i1) {
    here = tile_pages(p, table, sp.tiles.tile(i0 + wave));
    load_keys<A, D, F8>(k, p.ck, here, head, lane);
  }
  for (int i = i0 + wave; i < i1; i += kWaves) {
    const int tile = sp.tiles.tile(i);
    load_values<A, D, F8>(v, p.cv, here, head, lane);
    const bool more = i + kWaves < i1;
    if (more) next = tile_pages(p, table, sp.tiles.tile(i + kWaves));

    f32x4 s[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const V8 a = key_step<A, D, F8>(k, u, ks);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][u] = A::mfma16(a, q[nt][ks], s[nt][u]);
      }
    if (more) load_keys<A, D, F8>(k, p.ck, next, head, lane);

    // all keys of the tile visible to all of the window's rows?
    const int key0 = tile * kTile;
    const bool full = !careful && here.ok[0] && here.ok[1] && key0 + kTile - 1 <= first_pos &&
                      (p.mask.window == 0 || key0 > sp.len - 1 - p.mask.window ||
                       key0 + kTile - 1 < p.mask.sinks);
    V8 ph[NT], pl[NT];
    f32x8 pr[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = s[nt][j >> 2][j & 3] * scale;
      if (!full) {
        const bool ok = g & 2 ? here.ok[1] : here.ok[0];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] = ok && key_visible(p.mask, key0 + 8 * g + j, pos[nt]) ? x[j] : kNegInf;
      }
      float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                        fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float now = fmaxf(m[nt], top);
      if (__builtin_amdgcn_ballot_w64(now > m[nt]) != 0) {
        const float a = exp2_fast(m[nt] - (now == kNegInf ? 0.0f : now));
        l[nt] *= a;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[nt][dt] *= a;
        m[nt] = now;
      }
      const float base = m[nt] == kNegInf ? 0.0f : m[nt];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        pr[nt][j] = exp2_fast(x[j] - base);
        l[nt] += pr[nt][j];
      }
      ph[nt] = __builtin_convertvector(pr[nt], V8);
      pl[nt] = __builtin_convertvector(pr[nt] - __builtin_convertvector(ph[nt], f32x8), V8);
    }

    bool dirty = false;  // a masked tile with non-finite values somewhere
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      V8 a = value_step<A, D, F8>(v, dt);
      if (!full) dirty |= clear_nonfinite<A>(a);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        o[nt][dt] = A::mfma16(a, ph[nt], o[nt][dt]);
        o[nt][dt] = A::mfma16(a, pl[nt], o[nt][dt]);
      }
    }
    if (!full && __builtin_amdgcn_ballot_w64(dirty) != 0) {
      // A zero probability times a non-finite value is NaN, so such values of a tile that
      // not all rows see were left out above; here they reach the rows that see them.
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll 1
        for (int key = 0; key < kTile; ++key) {
          const bool seen = (key & 16 ? here.ok[1] : here.ok[0]) &&
                            key_visible(p.mask, key0 + key, pos[nt]);
          if (__builtin_amdgcn_ballot_w64(seen) == 0) continue;
          float w = pr[nt][0];
#pragma unroll
          for (int j = 1; j < 8; ++j) w = (key & 7) == j ? pr[nt][j] : w;
          w = __shfl(w, ((key >> 3) << 4) + n16);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float x = value_at<A, D, F8>(p.cv, here, head, key, out_col<F8>(dt, 4 * g + r));
              if (seen && !__builtin_isfinite(x)) o[nt][dt][r] += w * x;
            }
        }
    }
    here = next;
  }
  if (!careful) {
    bool bad = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int r = 0; r < 4; ++r) bad |= !__builtin_isfinite(o[nt][dt][r]);
    careful = __builtin_amdgcn_ballot_w64(bad) != 0;
    if (careful) goto again;
  }

  // join the waves: one row tile and DC columns at a time
  const float vs = p.v_scale ? p.v_scale[kvh] : 1.0f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float lsum = l[nt];
    lsum += __shfl_xor(lsum, 16);
    lsum += __shfl_xor(lsum, 32);
    if (g == 0) {
      stat_m[wave][n16] = m[nt];
      stat_l[wave][n16] = lsum;
    }
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += DC) {
#pragma unroll
      for (int dt = c0 / 16; dt < (c0 + DC) / 16; ++dt) {
        if constexpr (F8) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            sums[wave][n16][out_col<F8>(dt, 4 * g + r) - c0] = o[nt][dt][r];
        } else {
          *reinterpret_cast<f32x4*>(&sums[wave][n16][16 * dt + 4 * g - c0]) = o[nt][dt];
        }
      }
      __syncthreads();
      constexpr int PER = 16 * DC / kThreads;  // columns a thread: 4 or 8
      const int r = threadIdx.x / 16, col = (threadIdx.x % 16) * PER;
      const int row = (rt * NT + nt) * 16 + r;
      if (row < rows) {
        float top = kNegInf, sum = 0.0f, weight[kWaves], y[PER];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat_m[w][r]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          weight[w] = exp2_fast(stat_m[w][r] - (top == kNegInf ? 0.0f : top));
          sum += weight[w] * stat_l[w][r];
        }
#pragma unroll
        for (int c = 0; c < PER; ++c) {
          y[c] = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) y[c] += weight[w] * sums[w][r][col + c];
        }
        const long long token = (long long)seq * p.T + row / p.group;
        const long long at = token * hq + kvh * p.group + row % p.group;
        if (direct) {
          typename A::T* out = reinterpret_cast<typename A::T*>(p.out) + at * D + c0 + col;
#pragma unroll
          for (int c = 0; c < PER; ++c)
            out[c] = (typename A::T)(sum == 0.0f ? 0.0f : y[c] / sum * vs);
        } else {
          const long long part = at * p.splits + split;
#pragma unroll
          for (int c = 0; c < PER; ++c) p.partial[part * D + c0 + col + c] = y[c];
          if (c0 == 0 && threadIdx.x % 16 == 0) p.stats[part] = make_float2(top, sum);
        }
      }
      __syncthreads();
    }
  }
#endif
}

// Joins the splits of one (token, query head) row.
template <typename A, int D>
__global__ __launch_bounds__(kThreads) void k_attn_decode_join(DecodeParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int hq = p.kv_heads * p.group;
  const long long at = blockIdx.x;
  const SeqSplit sp = seq_split(p, (int)(at / ((long long)p.T * hq)));
  if (sp.live <= 1) return;  // written by its only split
  const int kvh = (int)(at % hq) / p.group;
  join_row<A, D>(p.partial, p.stats, at, p.splits, sp.live, p.v_scale ? p.v_scale[kvh] : 1.0f,
                 p.out);
#endif
}

// Row tiles (of 16 rows) that one workgroup takes: as many as the window has, while their
// accumulators fit beside the tile's keys and values.
int tiles_per_group(int rows, int D) {
  const int most = D == 256 ? 2 : 4;
  int nt = 1;
  while (nt < most && 16 * nt < rows) nt *= 2;
  return nt;
}

template <typename A, int D, bool F8, int NT>
hipError_t launch_one(const DecodeParams& p, int n_seqs, hipStream_t stream) {
  k_attn_decode<A, D, F8, NT><<<dim3(p.splits, p.kv_heads * p.row_tiles, n_seqs),
                                dim3(kThreads), 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  k_attn_decode_join<A, D><<<dim3((unsigned)(n_seqs * p.T * p.kv_heads * p.group)),
                             dim3(kThreads), 0, stream>>>(p);
  return hipGetLastError();
}

template <typename A, int D, bool F8>
hipError_t launch_tiles(const DecodeParams& p, int n_seqs, hipStream_t stream) {
  const int nt = tiles_per_group(p.T * p.group, D);
  if (nt == 1) return launch_one<A, D, F8, 1>(p, n_seqs, stream);
  if (nt == 2) return launch_one<A, D, F8, 2>(p, n_seqs, stream);
  if constexpr (D != 256) return launch_one<A, D, F8, 4>(p, n_seqs, stream);
  return hipErrorInvalidValue;
}

template <typename A>
hipError_t launch_type(const DecodeParams& p, int D, bool f8, int n_seqs, hipStream_t stream) {
  if (D == 64)
    return f8 ? launch_tiles<A, 64, true>(p, n_seqs, stream)
              : launch_tiles<A, 64, false>(p, n_seqs, stream);
  if (D == 128)
    return f8 ? launch_tiles<A, 128, true>(p, n_seqs, stream)
              : launch_tiles<A, 128, false>(p, n_seqs, stream);
  return f8 ? launch_tiles<A, 256, true>(p, n_seqs, stream)
            : launch_tiles<A, 256, false>(p, n_seqs, stream);
}

}  // namespace

AttnPlan decode_plan(int q_heads, int kv_heads, int D, int n_seqs, int window_tokens,
                     int max_pages, int page_size, const moe_attn& a, int num_cus) {
  AttnPlan plan{};
  const int rows = window_tokens * (q_heads / kv_heads);
  plan.tile_rows = 16 * tiles_per_group(rows, D);
  plan.row_tiles = (rows + plan.tile_rows - 1) / plan.tile_rows;
  // tiles of the longest possible sequence (of its visible part)
  long long tiles = ((long long)max_pages * page_size + kTile - 1) / kTile;
  if (a.window > 0)
    tiles = std::min(tiles, ((long long)a.window + window_tokens) / kTile + 2 +
                                ((long long)a.sinks + kTile - 1) / kTile);
  const long long base = (long long)n_seqs * kv_heads * plan.row_tiles;
  const long long fill = (2 * num_cus + base - 1) / base;
  const long long even = (tiles + 63) / 64;  // 2048 keys, so that long sequences share out
  const long long most = std::max(1ll, tiles / kMinSplitTiles);
  plan.splits = (int)std::min<long long>({std::max(fill, even), most, kMaxSplits});
  if (plan.splits > 1) {
    const size_t parts = (size_t)n_seqs * window_tokens * q_heads * plan.splits;
    plan.partial = 0;
    plan.stats = align256(parts * D * sizeof(float));
    plan.total = plan.stats + align256(parts * sizeof(float2));
  }
  return plan;
}

hipError_t launch_attn_decode(const AttnArgs& a, const AttnPlan& plan) {
  DecodeParams p{};
  p.q = a.q;
  p.ck = (const char*)a.cache.k;
  p.cv = (const char*)a.cache.v;
  p.k_scale = a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.table = a.pages.table;
  p.kv_lens = a.pages.kv_lens;
  p.table_stride = a.pages.table_stride;
  p.out = a.out;
  p.partial = (float*)(a.ws + plan.partial);
  p.stats = (float2*)(a.ws + plan.stats);
  p.scale = a.a.scale * kLog2e;
  p.mask = KeyMask{a.a.window, a.a.sinks};
  p.num_pages = a.cache.num_pages;
  while ((1 << p.page_shift) < a.cache.page_size) ++p.page_shift;
  p.kv_heads = a.cache.kv_heads;
  p.max_pages = a.pages.max_pages;
  p.group = a.q.heads / a.cache.kv_heads;
  p.T = a.window_tokens;
  p.splits = plan.splits;
  p.row_tiles = plan.row_tiles;
  return a.dtype == MOE_BF16
             ? launch_type<Bf16>(p, a.cache.head_dim, a.cache.dtype == MOE_E4M3,
                                 a.pages.n_seqs, a.stream)
             : launch_type<F16>(p, a.cache.head_dim, a.cache.dtype == MOE_E4M3, a.pages.n_seqs,
                                a.stream);
}

}  // namespace qmoe
