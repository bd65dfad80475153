// Definitions shared by the attention translation units: the per-pass workspace header, the prefill
// work-item record and the prefill launch entry.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv_internal.cuh"

namespace pkv {

constexpr int kBS = 16;          // tokens per cache block
constexpr int kHeadsTile = 8;    // query heads per KV head handled by one decode MMA tile (G <= 8)
// On a 4-bit cache split_blocks may be up to 256 and is 128 by default.  A task costs its SM about 3.6 us beside its blocks, so
// large batches run faster in longer splits and single rows slower (d 128, 12 / 2 heads, us a call with 128 and 256 blocks a
// split: 256 rows of up to 8192 tokens 75.5 and 66.0, 64 rows of 32000 132 and 116, of 8000 42.5 and 38.8; 16 rows of 8000
// 17.6 and 22.6, one row of 8000 15.7 and 21.9).
constexpr int kMaxSplitBlocksInt4 = 256;

// Rows with at least this many new tokens (a prefill chunk) go to the tensor-core tile kernel; shorter
// rows (decode, short chunks) to the split-K decode kernel.  The choice depends on the row alone, so a
// row's result does not depend on the rest of the batch.
constexpr int kPrefillMinQlen = 16;
constexpr int kPrefillRows = 128;  // MMA rows of a prefill Q tile: (query position, query head) pairs
constexpr int kPrefillKeys = 128;  // keys per K/V tile (64 at head_dim 256, prefill_tile_keys)
constexpr int kPrefillBuckets = 1024;
// An item whose keys span more K/V tiles than this runs as two chunks of keys (split-KV) that the
// second chunk to finish merges, when its row alone cannot keep every CTA busy for the item's length; the
// split depends on the row (and the SM count) alone.
constexpr int kPrefillSplitTiles = 24;

// Query positions per prefill Q tile: the G query heads of a KV head are packed into the MMA rows.
__host__ __device__ constexpr int prefill_positions(int group) { return kPrefillRows / group; }
// Keys per prefill K/V tile: at head_dim 256 a Q tile's output takes 256 tensor memory columns, its scores the
// next 64 (a 128-key tile's would not fit beside them), and 64-key tiles keep the K/V rings in shared memory.
__host__ __device__ constexpr int prefill_tile_keys(int head_dim) { return head_dim == 256 ? 64 : kPrefillKeys; }

// What a query at position p sees of its row: every key k <= p with k > p - window, and the row's first `sinks`
// keys whatever the window.  kNoWindow: all of them.
constexpr int kNoWindow = 0x7FFFFFFF;
struct KeyWindow {
  int window = kNoWindow;
  int sinks = 0;
  int split = 0;  // blocks per split of a token that the window cuts (make_window)
};

// A windowed plan's tokens mostly see the same number of blocks, a little more than a power of two of them: full splits
// of 32 would leave each token a last split of a few blocks, whose cost is that of a task and not of its blocks.  So a
// token cut by its window runs in equal splits, rounded up to eight blocks (two for each streaming warp, a pair on the
// 8-bit d 256 path): 66 blocks as 24 + 24 + 18 take 51.2 us, as 32 + 32 + 2 54.4 (256 rows, 12 / 2 heads, d 128); 34 as
// 24 + 10 33.0 against 36.2; 261 stay at 32 (103 us on the 8-bit cache at d 256, 120 in splits of 28).  At head_dim 64,
// whose warps go in pairs of blocks, the 66 would be faster as 32 + 32 + 2 (8 / 2 heads: 41.0 us, 45.6 so).  The window
// alone decides, and a token whose whole context is visible keeps the unwindowed partition.  (On a 4-bit cache a split
// may be a quarter longer than split_blocks, `slack`: 130 blocks, a window of 2048 tokens, as one take 30.7 us, as 72 + 58 39.8;
// 200 rows, 12 / 2 heads, d 128.  Rounding up to 24 blocks, a pair for each of twelve warps, or to 16 at d 256, gained
// nothing over eight there: windows of 1000 to 4096 within 1 %, of 8000 at d 256 1.5 % longer.)
__host__ __device__ constexpr int window_blocks_at_most(int window, int sinks) {
  return (sinks + kBS - 1) / kBS + (window > kNoWindow - kBS ? kNoWindow / kBS : (window + kBS - 2) / kBS) + 1;
}
__host__ constexpr KeyWindow make_window(int window, int sinks, int split_blocks, int slack = 0) {
  const int seen = window_blocks_at_most(window, sinks < kNoWindow - kBS ? sinks : kNoWindow - kBS), most = split_blocks + slack;
  const int n = (seen + most - 1) / most, even = ((seen + n - 1) / n + 7) / 8 * 8;
  return KeyWindow{window, sinks, even < most ? even : most};
}
// Blocks per split of a token that sees ctx keys without the window.
__host__ __device__ constexpr int token_split(int ctx, int split_blocks, const KeyWindow& win) {
  return ctx > win.window ? win.split : split_blocks;
}

// First key of the window of the query that sees `ctx` keys without one (position ctx - 1).
__host__ __device__ constexpr int window_low(int ctx, int window) { return ctx > window ? ctx - window : 0; }

// The units (blocks of 16 keys, or K/V tiles) that queries with windows from key `low` on and `kend` keys in all see:
// the first `head` ones (the sinks'), then those from unit head + skip on; n of them.  Unit j of the n is unit
// j of the row below `head` and unit j + skip above; without a gap between sinks and window skip is 0.
struct VisibleUnits {
  int head, skip, n;
  __host__ __device__ int row_unit(int j) const { return j < head ? j : j + skip; }
};
__host__ __device__ constexpr VisibleUnits visible_units(int kend, int low, int sinks, int unit) {
  const int all = (kend + unit - 1) / unit, first = low / unit;
  const int head = ((sinks < kend ? sinks : kend) + unit - 1) / unit;
  const int skip = first > head ? first - head : 0;
  return VisibleUnits{head, skip, all - skip};
}
__host__ __device__ constexpr VisibleUnits visible_blocks(int ctx, int window, int sinks) {
  return visible_units(ctx, window_low(ctx, window), sinks, kBS);
}

struct WsHeader {
  int32_t n_tasks;   // decode tasks of the pass
  int32_t work;      // dynamic decode tasks handed out so far (each CTA's first two are static)
  int32_t done;      // decode CTAs of the current launch that have finished
  int32_t n_items;   // prefill items of the pass
  int32_t pwork;     // dynamic prefill items handed out so far (each CTA's first is static)
  int32_t pdone;     // prefill CTAs of the current launch that have finished
  int32_t pad[58];
};
static_assert(sizeof(WsHeader) == 256, "header is one 256-byte line");

// A prefill work entry: one KV head, up to prefill_item_positions(G, d) consecutive query positions of one
// row, all of its keys or one of two chunks of them.
//   x: row (block-table row)
//   y: KV head | positions << 8 | chunk << 20 | split << 21
//   z: first query token (packed)     w: keys visible to the item's first position, minus one
// Position i of the item attends causally to keys 0 .. w + i.  A split item's two entries share a slot
// (the partial results and the merge handshake).
__host__ __device__ constexpr int prefill_rec_y(int g, int npos, int chunk, int split) {
  return g | (npos << 8) | (chunk << 20) | (split << 21);
}

struct PrefillArgs {
  const CUtensorMap* kv_map;  // device copy is passed by value below; this one is host-side
  const void* q;
  void* out;
  const int32_t* block_tables;
  const int4* items;
  const int32_t* items_slot;  // per work entry: the split item's slot, or -1
  int2* pf_sync;              // per slot: {chunks finished, first chunk's partial published}
  float2* pf_ml;              // per slot: [256 rows] (running max, running sum) of the first chunk
  float* pf_o;                // per slot and Q tile: [head_dim][128 rows] unnormalised output of the first chunk
  WsHeader* hdr;
  int32_t* err;
  int layer_row0_k, layer_row0_v;
  int max_blocks, num_q_heads, num_kv_heads, num_blocks, head_dim;
  pkv_pool* pool;
  int64_t max_items;
  KeyWindow win;
};

// Launch the prefill tile kernel for one layer (programmatic dependent launch on `stream`).
cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream);
// The same with a.win's window (its instances live in prefill_window.cu).
cudaError_t launch_prefill_window(const PrefillArgs& a, cudaStream_t stream);
// Whether the tile kernel serves this head shape (otherwise every row takes the decode path).
bool prefill_supported(int head_dim, int group);
// Query positions per prefill item (the Q tiles of one item share their K/V tiles).
int prefill_item_positions(int group, int head_dim);

}  // namespace pkv
