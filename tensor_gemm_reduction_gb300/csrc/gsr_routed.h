// gsr_routed.h -- launch parameters of the routed projections (internal to the
// library): products grouped by expert, the gated form, the K-sharded
// projection with per-row adapters, the route and the combine.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gsr_params.h"

namespace gsr {

constexpr int kMaxGroups = 1024;
constexpr int kMaxTopk = 128;
constexpr int kMaxRank = 128;       // columns of an adapter
constexpr int kMaxAdapters = 65536;

// kGrouped: Y = X . W[group]^T. kGated: Y = silu(X . Wg^T) * (X . Wu^T), gate and
// up rows in one W. kLora: the K-sharded projection plus the adapters' products.
enum RoutedKind : int { kGrouped = 0, kGated = 1, kLora = 2 };

// Workspace of the routed calls (bytes): [0, 256) header (status word at 0);
// [256, 256 + kRoutedCounterBytes) arrival counters of cut tiles; then the
// fp32 partials of cut tiles; then the adapters' low-rank rows and lists.
constexpr size_t kRoutedCounterBytes = 8192;
constexpr int kRoutedTileRows = 256;        // weight rows of a CTA pair's tile
constexpr int kRoutedMaxTokens = 256;       // tokens of a tile, at most (kLora)
// One adapter list per token tile: a count, then the tile's adapters ascending.
constexpr int kAdapterListStride = kRoutedMaxTokens + 8;

struct RoutedParams {  // 128-byte aligned through its CUtensorMap members
  // Weights. Grouped: tmap_w[0] = W as {K, rows, E}, boxes of 64 x 128 rows (64
  // rows when gated). Lora: tmap_w[r] = W_r, boxes of 64 x w_rows.
  CUtensorMap tmap_w[kMaxShards];
  // Tokens. Grouped: tmap_x[i] = X in boxes of 64 x 8 (i + 1) rows (none when the
  // rows are gathered). Lora: tmap_x[r] = X_r in boxes of 64 x tile_tokens / 2.
  CUtensorMap tmap_x[kMaxShards];
  CUtensorMap tmap_b;               // lora: B as {rank, N, L}, boxes of unit_cols x w_rows

  const int32_t* offsets;           // grouped: E + 1 row offsets
  const int32_t* rows;              // grouped: row of X of each row of Y (gathered)
  const uint16_t* x;                // gathered: X, T x K
  const int32_t* adapter;           // lora: the adapter of each row
  const int32_t* lists;             // lora: adapter lists of the token tiles
  const uint16_t* low;              // lora: M x rank_pad, the scaled low-rank rows
  const uint16_t* b;                // lora: L x N x rank
  const uint16_t *x_r[kMaxShards], *a_r[kMaxShards];   // lora, self_rows: the operands of the
  int k_r[kMaxShards];                                 // low-rank rows
  const float* scale;
  int self_rows;                    // lora: the product computes the low-rank rows itself
  uint16_t* y;                      // M x N
  uint32_t* status;
  uint32_t* counters;
  float* partials;
  uint64_t timeout_ns;

  int E, M, N, K, T, R, L, rank;       // T: rows of X (grouped)
  int n_tiles;                      // tiles of output columns
  int cta_cols, w_rows;             // output columns and weight rows of a CTA's part of a tile
  int stages_per_tile;              // ring stages of a whole tile (the base product)
  int m_tiles, tile_tokens;         // lora: token tiles and their width
  int stages;                       // lora, half tiles: of the ring
  int whole_boxes;                  // lora, half tiles: tmap_w and tmap_x are {64, rows, k-blocks}
                                    // views with boxes of a stage's k-blocks
  int max_pieces;                   // of a cut tile
  // Remaining tiles are cut when a piece is shorter than the tile by more stages than
  // this: when no whole tiles follow, and when they do and hide the sum.
  int cut_alone, cut_ahead;
  int unit_cols, units_per_adapter; // lora: columns of one step over an adapter
  int rank_pad;                     // lora: unit_cols * units_per_adapter
  int policy_w, policy_x;
  int shard_st_begin[kMaxShards + 1];  // lora: first stage of shard r
};

// Calls of this few rows and padded columns (M * rank_pad, one or two rows) compute the
// low-rank rows in the product. Measured in the product / by the kernel before it (us, N =
// K = 7168): one row of rank 8 24.8 / 29.7, 16 25.3 / 29.7, 32 29.0 / 30.6, two of rank 16
// 27.4 / 30.0.
constexpr int kSelfRows = 2, kSelfElements = 32;

// The low-rank rows: low[m, :] = scale[a] * sum_r X_r[m] . A_r[a]^T, a = adapter[m],
// in bf16, and the adapter lists of the token tiles.
struct LowRankParams {
  const uint16_t* x[kMaxShards];    // M x K_r
  const uint16_t* a[kMaxShards];    // L x rank x K_r
  int64_t k[kMaxShards];
  const int32_t* adapter;
  const float* scale;               // NULL: 1
  uint16_t* low;
  int32_t* lists;
  int M, R, L, rank, rank_pad;
  int tile_tokens, m_tiles;         // of the product that reads the lists
};

struct RouteParams {
  const void* ids;                  // T x topk
  int32_t* offsets;
  int32_t* source;
  int32_t* position;
  int n, topk, E, wide;             // wide: 64-bit ids
  // Set by the launcher. The entries in parts, one per CTA: of units + 1 times 32 entries
  // the first `longer`, of units times 32 the others (the last may be short of 32).
  int parts, units, longer;
  uint32_t topk_magic;              // 0: divide
};

struct CombineParams {
  const uint16_t* z;
  const int32_t* position;
  const float* weights;
  const uint16_t* base;             // or NULL
  uint16_t* y;
  int64_t T, z_rows;
  int topk, vecs;                   // 16-byte vectors of a row
};

// Token capacities of the routed product's instances.
constexpr int kRoutedSmall = 64, kRoutedMid = 128, kRoutedWide = 256, kRoutedDouble = 512;
// k-blocks of 64 in one ring stage. A stage costs its barriers' fixed time (about
// 200 ns), so it should carry many bytes: with one k-block per stage the 256-token
// tiles are 10 to 20 % slower. The half tiles carry few weight rows, so four.
constexpr int routed_kblocks(bool half, int tokens) {
  return tokens == kRoutedDouble ? 1 : half && tokens <= kRoutedMid ? 4 : 2;
}

// The half tiles' ring: bytes, and stages at most.
constexpr int kHalfRing = 196608, kHalfSlots = 16;

cudaError_t prepare_routed_kernels();
cudaError_t prepare_lowrank_kernels();
cudaError_t prepare_route_kernels();
// half: tiles of at most 128 weight rows (kLora).
cudaError_t launch_routed(const RoutedParams& p, int kind, bool gather, bool half, int tokens, int ctas,
                          cudaStream_t stream);
cudaError_t launch_low_rank(const LowRankParams& p, cudaStream_t stream);
cudaError_t launch_route(const RouteParams& p, cudaStream_t stream);
cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream);

}  // namespace gsr
