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
// rest, which costs matrix-core time that the memory-bound loop has to spare. What the two
// parts leave of a probability: 2^-16 of it in bf16; in fp16 2^-22 of it, or 2^-36 of the
// largest one that the wave has seen in the row, where that is more.
#include <type_traits>

#include "qmoe_attn_plan.h"

namespace qmoe {
namespace {

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
  int group, T, splits, fill, row_tiles;
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
  // as many even parts as fill the card, or as cut a long sequence; the table may be far wider
  // than this one is long
  const int parts = max(p.fill, (s.tiles.count + kLongSplitTiles - 1) / kLongSplitTiles);
  const int most = min(parts, p.splits);
  s.per = max(kMinSplitTiles, (s.tiles.count + most - 1) / most);
  s.live = (s.tiles.count + s.per - 1) / s.per;
  return s;
}

#if defined(__HIP_DEVICE_COMPILE__)

// A 32-key tile's two 16-row halves: with pages of 32 rows or more both are in one page,
// with 16-row pages each has its own. The page number of half u, -1 for an entry outside
// the cache: its keys count as invisible, and page 0 is read instead.
__device__ __forceinline__ int half_page(const DecodeParams& p, const int32_t* table, int tile,
                                         int u) {
  const int i = (tile * kTile + 16 * u) >> p.page_shift;
  const int id = i < p.max_pages ? load_uniform(table + i) : -1;
  return (unsigned)id < (unsigned)p.num_pages ? id : -1;
}

// First row of half u in the cache (counting the rows of all heads' pages).
__device__ __forceinline__ long long half_row(const DecodeParams& p, int page, int kvh, int tile,
                                              int u) {
  const long long rows = ((long long)max(page, 0) * p.kv_heads + kvh) << p.page_shift;
  return rows + ((tile * kTile + 16 * u) & ((1 << p.page_shift) - 1));
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

// Each cache line is used once a call (by windows of more rows than a wave takes, once for
// every row tile): non-temporal loads read 7.1 TB/s here, plain ones 6.2.
__device__ __forceinline__ u32x4 stream_load(const char* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}

// Lane (m, g): 8 columns 32 i + 8 g of key row 8 (m / 4) + m % 4 + 4 u; at 8 bits, 16
// columns 64 i + 16 g, two steps of the product.
template <typename A, int D, bool F8>
__device__ __forceinline__ void load_keys(KeyRegs<A, D, F8>& r, const char* ck, long long row0,
                                          long long row1, int lane) {
  const int m = lane & 15, g = lane >> 4;
  const int row = 8 * (m >> 2) + (m & 3);
  constexpr int ROW = F8 ? D : 2 * D;  // bytes
  const char* at = ck + ((row & 16 ? row1 : row0) + (row & 15)) * ROW + 16 * g;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < KeyRegs<A, D, F8>::N; ++i)
      r.w[u][i] = stream_load(at + 4 * u * ROW + 64 * i);
}

// Lane (m, g): keys 8 g .. 8 g + 7 of column 16 i + m; at 8 bits of columns 32 i + 2 m and
// the next.
template <typename A, int D, bool F8>
__device__ __forceinline__ void load_values(ValueRegs<A, D, F8>& r, const char* cv, long long row0,
                                            long long row1, int lane) {
  const int m = lane & 15, g = lane >> 4;
  const long long block = ((g & 2 ? row1 : row0) >> 3) + (g & 1);
  const char* at = cv + block * (D * (F8 ? 8 : 16)) + 16 * m;
#pragma unroll
  for (int i = 0; i < ValueRegs<A, D, F8>::N; ++i)
    r.w[i] = stream_load(at + 256 * i);
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

#endif  // __HIP_DEVICE_COMPILE__

// Wide heads leave no registers for the query fragments: they are read from LDS at each
// tile (1 KB a step of the product, a small part of what LDS can deliver meanwhile).
template <int D, int NT>
constexpr bool kQueriesInLds = D * NT >= 256 && D != 64;

// NT: row tiles of 16 rows; KW: waves, which take the split's key tiles in turn. Bound by
// memory, or by latency where keys are few. 4 tokens over 262144 keys, 16 query and 2 kv heads
// of 256, bf16: 95 us and 5 for the join, 5.7 TB/s of the 7.1 that reading alone reaches; 64
// sequences of 8192 keys, 16 query and 2 kv heads of 128: 90 us, 6.0 TB/s; 517 keys: 10 us.
template <typename A, int D, bool F8, int NT, int KW>
__global__ __launch_bounds__(KW * kWave, decode_waves(NT, D)) void k_attn_decode(DecodeParams p) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef typename A::V8 V8;
  constexpr int KS = D / 32, DT = D / 16, kWaves = KW;
  constexpr int DC = D < 128 ? D : 128;  // columns joined at a time
  __shared__ float sums[kWaves][16][DC + 4];
  __shared__ float stat_m[kWaves][16], stat_l[kWaves][16];
  constexpr bool QLDS = kQueriesInLds<D, NT>;
  __shared__ u32x4 qs[QLDS ? NT * KS : 1][kWave];

  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n16 = lane & 15, g = lane >> 4;
  // Splits outermost: a sequence's live splits are the first ones, and workgroups go to the 8
  // XCDs in turn (64 sequences of 8192 keys with a page table 32 times as wide: 90 us; with
  // the splits innermost, where the live ones share few XCDs, 449).
  const int kvh = blockIdx.x / p.row_tiles, rt = blockIdx.x % p.row_tiles;
  const int seq = blockIdx.y, split = blockIdx.z;
  const SeqSplit sp = seq_split(p, seq);
  const bool direct = sp.live <= 1;
  if (split >= sp.live && !(direct && split == 0)) return;
  const int i0 = split * sp.per, i1 = min(i0 + sp.per, sp.tiles.count);
  const int32_t* table = p.table + seq * p.table_stride;
  const int first_pos = sp.len - p.T;
  const int rows = p.T * p.group;
  const int row0 = rt * NT * 16;  // the workgroup's first row

  KeyRegs<A, D, F8> k;
  ValueRegs<A, D, F8> v;
  int page0 = -1, page1 = -1, next0 = -1, next1 = -1;  // of this tile and the wave's next
  auto first_tile = [&]() {
    const int tile = sp.tiles.tile(i0 + wave);
    page0 = half_page(p, table, tile, 0);
    page1 = half_page(p, table, tile, 1);
    load_keys<A, D, F8>(k, p.ck, half_row(p, page0, kvh, tile, 0),
                        half_row(p, page1, kvh, tile, 1), lane);
  };
  if (i0 + wave < i1) first_tile();

  // this lane's query row of each row tile, as B operand: 8 columns a step
  const ScaleSplit sc = split_scale(p.scale * (p.k_scale ? p.k_scale[kvh] : 1.0f));
  V8 q[NT][QLDS ? 1 : KS];
  int pos[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = row0 + nt * 16 + n16;
    const int t = row / p.group, h = kvh * p.group + row % p.group;
    const bool real = row < rows;
    pos[nt] = real ? first_pos + t : -1;
    const char* src = p.q.data + 2 * (((long long)seq * p.T + (real ? t : 0)) * p.q.token_stride +
                                      (long long)(real ? h : 0) * p.q.head_stride);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (QLDS && (nt * KS + ks) % kWaves != wave) continue;
      const int col = F8 ? 64 * (ks >> 1) + 16 * g + 8 * (ks & 1) : 32 * ks + 8 * g;
      u32x4 w = *reinterpret_cast<const u32x4*>(src + 2 * col);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = real ? (w[i] ^ sc.flip) & sc.keep : 0u;
      if constexpr (QLDS)
        qs[nt * KS + ks][lane] = w;
      else
        q[nt][ks] = bits_as<V8>(w);
    }
  }
  if constexpr (QLDS) __syncthreads();

  f32x4 o[NT][DT];
  float m[NT], l[NT];  // scaled reference maximum of the row; this lane's part of its sum

  // A second, careful pass runs only where the first one's sums are not all finite: there
  // the split probability's small part would turn a visible infinity into NaN. It treats
  // every tile as one that not all rows see.
#pragma unroll 1
  for (bool careful = false;;) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt] = kNegInf;
      l[nt] = 0.0f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[nt][dt] = f32x4{0, 0, 0, 0};
    }
    if (careful) first_tile();
#pragma unroll 1
    for (int i = i0 + wave; i < i1; i += kWaves) {
      const int tile = sp.tiles.tile(i), key0 = tile * kTile;
      load_values<A, D, F8>(v, p.cv, half_row(p, page0, kvh, tile, 0),
                            half_row(p, page1, kvh, tile, 1), lane);
      const bool more = i + kWaves < i1;
      const int tile1 = sp.tiles.tile(i + kWaves);
      if (more) {
        next0 = half_page(p, table, tile1, 0);
        next1 = half_page(p, table, tile1, 1);
      }

      f32x4 s[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        V8 qf[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (QLDS)
            qf[nt] = bits_as<V8>(qs[nt * KS + ks][lane]);
          else
            qf[nt] = q[nt][ks];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const V8 a = key_step<A, D, F8>(k, u, ks);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][u] = A::mfma16(a, qf[nt], s[nt][u]);
        }
      }
      if (more)
        load_keys<A, D, F8>(k, p.ck, half_row(p, next0, kvh, tile1, 0),
                            half_row(p, next1, kvh, tile1, 1), lane);

      // all keys of the tile visible to all of the window's rows?
      const bool full = !careful && (page0 | page1) >= 0 && key0 + kTile - 1 <= first_pos &&
                        (key0 > behind_window(p.mask, sp.len - 1) ||
                         key0 + kTile - 1 < p.mask.sinks);
      bool dirty = false;  // not full, with non-finite values somewhere
      const bool on_page = (g & 2 ? page1 : page0) >= 0;
      if (!full) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (!(on_page && key_visible(p.mask, key0 + 8 * g + j, pos[nt])))
              s[nt][j >> 2][j & 3] = kNegInf;
#pragma unroll
        for (int j = 0; j < ValueRegs<A, D, F8>::N; ++j) dirty |= clear_word<A, F8>(v.w[j]);
      }

      V8 ph[NT], pl[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float top = fmaxf(fmaxf(fmaxf(s[nt][0][0], s[nt][0][1]), fmaxf(s[nt][0][2], s[nt][0][3])),
                          fmaxf(fmaxf(s[nt][1][0], s[nt][1][1]), fmaxf(s[nt][1][2], s[nt][1][3])));
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32)) * sc.scale;
        const bool moves = top > m[nt] + A::kLazy;
        if (__builtin_amdgcn_ballot_w64(moves) != 0) {
          const float now = moves ? top : m[nt];
          const float a = rescale(m[nt] - (now == kNegInf ? 0.0f : now));
          l[nt] *= a;
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) o[nt][dt] *= a;
          m[nt] = now;
        }
        const float base = exponent_base<A>(m[nt]);
        f32x8 pr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          pr[j] = exp2_fast(__builtin_fmaf(s[nt][j >> 2][j & 3], sc.scale, base));
          l[nt] += pr[j];
        }
        ph[nt] = __builtin_convertvector(pr, V8);
        pl[nt] = __builtin_convertvector(pr - __builtin_convertvector(ph[nt], f32x8), V8);
      }
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        const V8 a = value_step<A, D, F8>(v, dt);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[nt][dt] = A::mfma16(a, ph[nt], o[nt][dt]);
          o[nt][dt] = A::mfma16(a, pl[nt], o[nt][dt]);
        }
      }
      if (!full && __builtin_amdgcn_ballot_w64(dirty) != 0) {
        // the values as they are, once more: what they do to the rows that see them
        load_values<A, D, F8>(v, p.cv, half_row(p, page0, kvh, tile, 0),
                              half_row(p, page1, kvh, tile, 1), lane);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t seen = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            seen |= (uint32_t)(on_page && key_visible(p.mask, key0 + 8 * g + j, pos[nt])) << j;
          const V8 rows_seen = mask_elements<A>(seen);
#pragma unroll 1
          for (int i = 0; i < 3; ++i) {
            const NonFinite kind = non_finite_kind<A>(i);
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
              // nothing computed from the values is kept from one kind to the next
              asm volatile("" : "+v"(v.w[dt * ValueRegs<A, D, F8>::N / DT]));
              const f32x4 c = A::mfma16(non_finite<A>(value_step<A, D, F8>(v, dt), kind),
                                        rows_seen, f32x4{0, 0, 0, 0});
#pragma unroll
              for (int r = 0; r < 4; ++r) o[nt][dt][r] += spread(c[r], kind);
            }
          }
        }
      }
      page0 = next0;
      page1 = next1;
    }
    if (careful) break;
    bool bad = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int r = 0; r < 4; ++r) bad |= !__builtin_isfinite(o[nt][dt][r]);
    if (__builtin_amdgcn_ballot_w64(bad) == 0) break;
    careful = true;
  }

  // join the waves: one row tile and DC columns at a time
  const float vs = p.v_scale ? p.v_scale[kvh] : 1.0f;
  const int hq = p.kv_heads * p.group;
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
      constexpr int PER = DC / (4 * kWaves);  // columns a thread: 2, 4 or 8
      const int r = threadIdx.x / (4 * kWaves), col = (threadIdx.x % (4 * kWaves)) * PER;
      const int row = row0 + nt * 16 + r;
      if (row < rows) {
        float top = kNegInf, sum = 0.0f, weight[kWaves];
        typedef float FP __attribute__((ext_vector_type(PER)));
        FP y = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat_m[w][r]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          weight[w] = rescale(stat_m[w][r] - (top == kNegInf ? 0.0f : top));
          sum += weight[w] * stat_l[w][r];
        }
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
          for (int c = 0; c < PER; ++c) y[c] += weight[w] * sums[w][r][col + c];
        const long long token = (long long)seq * p.T + row / p.group;
        const long long at = token * hq + kvh * p.group + row % p.group;
        if (direct) {
          typedef typename A::T TP __attribute__((ext_vector_type(PER)));
#pragma unroll
          for (int c = 0; c < PER; ++c) y[c] = sum == 0.0f ? 0.0f : y[c] / sum * vs;
          *reinterpret_cast<TP*>(p.out + 2 * (at * D + c0 + col)) = __builtin_convertvector(y, TP);
        } else {
          const long long part = at * p.splits + split;
          *reinterpret_cast<FP*>(p.partial + part * D + c0 + col) = y;
          if (c0 == 0 && col == 0) p.stats[part] = make_float2(top, sum);
        }
      }
      __syncthreads();
    }
  }
#endif
}

// Joins the splits of one (token, query head) row.
template <typename A, int D>
__global__ __launch_bounds__(kJoinThreads) void k_attn_decode_join(DecodeParams p) {
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

template <typename A, int D, bool F8, int NT, int KW = 4>
hipError_t launch_one(const DecodeParams& p, int n_seqs, hipStream_t stream) {
  k_attn_decode<A, D, F8, NT, KW><<<dim3(p.kv_heads * p.row_tiles, n_seqs, p.splits),
                                    dim3(KW * kWave), 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  k_attn_decode_join<A, D><<<dim3((unsigned)(n_seqs * p.T * p.kv_heads * p.group),
                                  D / kJoinCols), dim3(kJoinThreads), 0, stream>>>(p);
  return hipGetLastError();
}

template <typename A, int D, bool F8>
hipError_t launch_tiles(const DecodeParams& p, int n_seqs, hipStream_t stream) {
  const int nt = window_tiles(p.T * p.group, D);
  if constexpr (D != 256) {
    if (nt == 4) return launch_one<A, D, F8, 4>(p, n_seqs, stream);
  }
  if (nt == 2) return launch_one<A, D, F8, 2>(p, n_seqs, stream);
  // A short context on few workgroups is a chain of latencies, which twice the waves halve
  // (517 keys: 10.6 us against 7.2 and a joining launch of 3.8); on many, four waves run
  // nearer to the memory's rate (64 sequences at 8 bits: 370 us, with eight 447).
  if constexpr (D != 256) {
    if (p.splits == 1 && (long long)n_seqs * p.kv_heads * p.row_tiles <= device_cu_count())
      return launch_one<A, D, F8, 1, 8>(p, n_seqs, stream);
  }
  return launch_one<A, D, F8, 1>(p, n_seqs, stream);
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
  p.mask = key_mask(a.a);
  p.num_pages = a.cache.num_pages;
  while ((1 << p.page_shift) < a.cache.page_size) ++p.page_shift;
  p.kv_heads = a.cache.kv_heads;
  p.max_pages = a.pages.max_pages;
  p.group = a.q.heads / a.cache.kv_heads;
  p.T = a.window_tokens;
  p.splits = plan.splits;
  p.fill = plan.fill;
  p.row_tiles = plan.row_tiles;
  return a.dtype == MOE_BF16
             ? launch_type<Bf16>(p, a.cache.head_dim, a.cache.dtype == MOE_E4M3,
                                 a.pages.n_seqs, a.stream)
             : launch_type<F16>(p, a.cache.head_dim, a.cache.dtype == MOE_E4M3, a.pages.n_seqs,
                                a.stream);
}

}  // namespace qmoe
