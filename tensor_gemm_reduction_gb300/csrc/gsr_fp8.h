// gsr_fp8.h -- launch parameters of the 8-bit projections and of what feeds them
// (internal to the library): the residual sum with RMS norm, the quantisation, and
// the products of e4m3 operands with a scale per block of 128.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gsr_params.h"

namespace gsr {

constexpr int kScaleBlock = 128;        // columns (and weight rows) of one scale
constexpr int kMaxNormColumns = 32768;  // a row in one CTA's registers

struct NormParams {
  const uint16_t* x;          // M x H
  const uint16_t* residual;   // M x H, or NULL
  const uint16_t* gamma;      // H, or NULL (1)
  uint16_t* sum;              // M x H, or NULL
  uint16_t* y;                // M x H, or NULL
  uint8_t* q;                 // M x H, or NULL (with scale)
  float* scale;               // ceil(H / 128) x M
  int64_t M;
  int H;
  float eps;
};

struct QuantParams {
  const uint16_t* x;
  uint8_t* q;
  float* scale;
  int64_t rows;
  int cols;
  int block_rows;             // 1: scale is ceil(cols / 128) x rows; 128: blocks, row-major
};

struct Fp8Params {  // 128-byte aligned through its CUtensorMap members
  // AR: X_r and W_r. AG: A_r, and W in tmap_w[0]. Boxes of 128 columns x box_rows
  // (tile_n / 2) rows; with whole_boxes of a stage's k-blocks of them.
  CUtensorMap tmap_x[kMaxShards];
  CUtensorMap tmap_w[kMaxShards];
  // The rows of Y of M-shard r, in boxes of fp8_store_cols x 32 rows (wide, with tma_store).
  CUtensorMap tmap_y[kMaxShards];
  const float* sx[kMaxShards];   // scales of X_r / A_r: k-blocks x rows
  const float* sw[kMaxShards];   // of W_r, or [0]: row blocks x k-blocks
  uint16_t* y;
  uint32_t* status;
  uint64_t timeout_ns;

  int ag;
  int N;
  int k_shards;                     // AR: R; AG: 1
  int m_shards;                     // AR: 1; AG: R
  int tile_n, n_tiles, m_tiles, tiles;
  int group_m;                      // raster: token tiles that run before the next weight tile
  int box_rows, boxes;              // a CTA's tokens: `boxes` boxes of box_rows rows, each of one shard
  int pad_shard;                    // AG: a shard with rows, read out of range (zeros) past the last box
  int ring;                         // stages of the shared-memory ring
  int whole_boxes;
  int tma_store;                    // every warp's 32 rows are of one box
  int policy_x, policy_w;
  int stages_per_tile;
  int shard_kb[kMaxShards];         // k-blocks of 128 of K-shard r
  int shard_st_begin[kMaxShards + 1];  // first stage of K-shard r
  int box_begin[kMaxShards + 1];    // first box of M-shard r
  int shard_rows[kMaxShards];       // rows of M-shard r
  int64_t shard_row_begin[kMaxShards];  // its first row of Y
};

// The instances. kFp8Wide: 256 token rows per CTA pair, weight tiles of 64, 128, 192 or 256
// rows; kFp8Narrow: up to 128 token rows, weight tiles of 32, 64, 96 or 128. k-blocks of a
// ring stage: a stage costs the barriers' fixed time, so as many as have an accumulator
// each, twice.
enum Fp8Form : int { kFp8Wide = 0, kFp8Narrow = 1 };
__host__ __device__ constexpr int fp8_kblocks(int form, int tile_n) {
  return form == kFp8Narrow ? 4 : tile_n <= 128 ? 2 : 1;
}
constexpr int fp8_max_tile_n(int form) { return form == kFp8Wide ? 256 : 128; }
constexpr int fp8_cta_rows(int form) { return form == kFp8Wide ? 128 : 64; }
constexpr int kFp8MaxRing = 16;
constexpr int kFp8ScaleRing = 2;      // of the scales' products, four k-blocks a stage
constexpr int kFp8RawRing = 4;        // of the scales
// Shared memory of what the epilogue stores from (wide: 32 rows of a warp's tile_n / 2 columns,
// or of 64 at a time), and of the ring.
__host__ __device__ constexpr int fp8_staged_cols(int tile_n) { return tile_n == 256 ? 64 : tile_n / 2; }
__host__ __device__ constexpr uint32_t fp8_staging_bytes(int form, int tile_n) {
  return form == kFp8Wide ? 8 * 32 * 2 * static_cast<uint32_t>(fp8_staged_cols(tile_n)) : 0;
}
__host__ __device__ constexpr uint32_t fp8_ring_bytes(int form, int tile_n) {
  return 206 * 1024 - fp8_staging_bytes(form, tile_n);
}
// Columns of a copy to Y (a warp's are tile_n / 2).
__host__ __device__ constexpr int fp8_store_cols(int tile_n) { return tile_n / 2 % 64 == 0 ? 64 : 32; }
constexpr uint32_t fp8_stage_bytes(int form, int tile_n, int token_rows) {
  return fp8_kblocks(form, tile_n) * kScaleBlock * static_cast<uint32_t>(tile_n / 2 + token_rows);
}
// Stages that fit. The MMAs read fp8_cta_rows rows of the tokens from a stage whatever it
// holds, in the last one past its end.
constexpr int fp8_ring(int form, int tile_n, int token_rows) {
  const uint32_t past = kScaleBlock * static_cast<uint32_t>(fp8_cta_rows(form) - token_rows);
  const uint32_t fit = (fp8_ring_bytes(form, tile_n) - past) / fp8_stage_bytes(form, tile_n, token_rows);
  return static_cast<int>(fit < kFp8MaxRing ? fit : kFp8MaxRing);
}

cudaError_t prepare_fp8_kernels();
cudaError_t launch_fp8(const Fp8Params& p, int form, int ctas, cudaStream_t stream);
cudaError_t launch_norm(const NormParams& p, int sm_count, cudaStream_t stream);
cudaError_t launch_quantize(const QuantParams& p, cudaStream_t stream);

}  // namespace gsr
