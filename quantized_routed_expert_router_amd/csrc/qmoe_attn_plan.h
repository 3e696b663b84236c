// How an attention call is cut into workgroups: row tiles, splits of the key axis and the
// workspace for joining them. Host code, and the constants that the kernels share with it.
#pragma once

#include "qmoe_attn_internal.h"

namespace qmoe {

// ------------------------------------------------------------------ decode windows

constexpr int kTile = 32;  // keys of one step of a wave
// A context of a few tiles is done sooner than a second launch; below 256 keys a split costs
// more than it saves.
constexpr int kUnsplitTiles = 32;
constexpr int kMinSplitTiles = 8;
// Sequences that fill the card anyway are cut at 4096 keys, so that long ones share out (64
// sequences of 1 to 32768 keys at 8 bits: 367 us, cut at 8192 keys 386).
constexpr int kLongSplitTiles = 128;
// Partial sums of one call, in bytes, at most. The page table's width says how long a sequence
// may be, not how long any is, and every token and head has room for as many splits: without a
// bound 32 sequences behind a table of a million keys asked for 17 GB. Splits that fill the
// card need 17 MB of it at most (512 sequences of 300 keys behind such a table, 64 heads of 128:
// 161 us, unbounded 904; 64 x 8 tokens over 1 to 262144 keys: 3.40 ms, unbounded 3.48).
constexpr size_t kMostPartialBytes = (size_t)256 << 20;

// Row tiles (of 16 query rows) a wave takes: as many as the window has, while accumulators
// (D/4 registers a row tile) fit beside a tile's keys and values (D/2 at 16 bits). More row
// tiles go to workgroups of their own, which read the keys again.
constexpr int kMostAccumulators = 128;
inline int window_tiles(int rows, int D) {
  int tiles = 1;
  while (16 * tiles < rows && tiles < 4 && 2 * tiles * (D / 4) <= kMostAccumulators) tiles *= 2;
  return tiles;
}
// Waves a SIMD that a wave's registers have to allow: two, so that accumulators stay out of
// the accumulation registers, or one where that leaves too few.
constexpr int decode_waves(int tiles, int D) { return D == 256 || tiles * D >= 512 ? 1 : 2; }

inline AttnPlan decode_plan(int q_heads, int kv_heads, int D, int n_seqs, int window_tokens,
                            int max_pages, int page_size, const moe_attn& a, int num_cus) {
  AttnPlan plan{};
  const int rows = window_tokens * (q_heads / kv_heads);
  const int wave_tiles = window_tiles(rows, D);
  plan.tile_rows = 16 * wave_tiles;
  plan.row_tiles = (rows + plan.tile_rows - 1) / plan.tile_rows;
  // tiles of the longest possible sequence (of its visible part)
  long long tiles = ((long long)max_pages * page_size + kTile - 1) / kTile;
  if (a.window > 0)
    tiles = std::min(tiles, ((long long)a.window + window_tokens) / kTile + 2 +
                                ((long long)a.sinks + kTile - 1) / kTile);
  const long long base = (long long)n_seqs * kv_heads * plan.row_tiles;
  // workgroups that run at once: two a CU, one where a wave takes many more than 256 registers
  const long long at_once = (wave_tiles * D >= 512 ? 1 : 2) * num_cus;
  const long long fill = (at_once + base - 1) / base;
  // no more even cuts than fill the card for a sequence alone, or than the workspace holds
  const long long alone = (at_once * n_seqs + base - 1) / base;
  const size_t split_bytes =
      (size_t)n_seqs * window_tokens * q_heads * (D * sizeof(float) + sizeof(float2));
  const long long even = std::min({(tiles + kLongSplitTiles - 1) / kLongSplitTiles, alone,
                                   (long long)(kMostPartialBytes / split_bytes)});
  const long long most = tiles <= kUnsplitTiles ? 1 : std::max(1ll, tiles / kMinSplitTiles);
  plan.splits = (int)std::min<long long>({std::max(fill, even), most, kMaxSplits});
  plan.fill = (int)std::min<long long>(fill, kMaxSplits);
  if (plan.splits > 1) {
    const size_t parts = (size_t)n_seqs * window_tokens * q_heads * plan.splits;
    plan.partial = 0;
    plan.stats = align256(parts * D * sizeof(float));
    plan.total = plan.stats + align256(parts * sizeof(float2));
  }
  return plan;
}

// ------------------------------------------------------------------ prefill chunks

constexpr int kMinSplitKeys = 512;

// Waves of a workgroup (32 rows each): 8 share a key tile among the most rows. Wide heads
// need 128 accumulators a lane and more than 256 registers, one wave a SIMD; and few rows
// fill the card better in halves.
inline int prefill_waves(int q_heads, int D, int n_tokens, int num_cus) {
  if (D == 256) return 4;
  return (long long)n_tokens * q_heads >= 256ll * num_cus ? 8 : 4;
}

inline AttnPlan prefill_plan(int q_heads, int kv_heads, int D, int n_seqs, int n_tokens,
                             int max_pages, int page_size, const moe_attn& a, int num_cus) {
  AttnPlan plan{};
  plan.tile_rows = 32 * prefill_waves(q_heads, D, n_tokens, num_cus);
  const long long rows = (long long)n_tokens * (q_heads / kv_heads);
  plan.row_tiles = (int)(rows / plan.tile_rows) + n_seqs;
  // row tiles that have rows, about; splits fill the card when they do not
  const long long base =
      std::max<long long>((rows + plan.tile_rows - 1) / plan.tile_rows,
                          std::min(n_seqs, n_tokens)) * kv_heads;
  long long keys = (long long)max_pages * page_size;
  if (a.window > 0)
    keys = std::min(keys, (long long)a.window + n_tokens + a.sinks + 128);
  const long long most = std::max(1ll, keys / kMinSplitKeys);
  const long long fill = (plan.tile_rows == 128 && D != 256 ? 2 : 1) * num_cus / base;
  plan.splits = (int)std::max(1ll, std::min<long long>({fill, most, kMaxSplits}));
  if (plan.splits > 1) {
    const size_t parts = (size_t)n_tokens * q_heads * plan.splits;
    plan.partial = 0;
    plan.stats = align256(parts * D * sizeof(float));
    plan.total = plan.stats + align256(parts * sizeof(float2));
  }
  return plan;
}

}  // namespace qmoe
