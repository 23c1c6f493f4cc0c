// gsr_fp8_api.cu -- host side of the 8-bit projections, the norm and the quantisation
// (include/gsr.h): argument checks, choice of the kernel instance, tensor maps and
// launches. Nothing here allocates device memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "gsr.h"
#include "gsr_fp8.h"
#include "gsr_host.h"

using gsr::aligned16;
using gsr::cdiv;
using gsr::check_plan;
using gsr::cuda_fail;
using gsr::DeviceScope;
using gsr::encode_fn;
using gsr::fail;
using gsr::kMaxShards;
using gsr::kScaleBlock;
using gsr::ok;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Rows of e4m3 in boxes of 128 columns x box_rows; with kblocks > 0 (cols a multiple of
// 128) as {128 columns, rows, k-blocks} in boxes of that many k-blocks. L2 fetches 256 bytes
// at once, but 128 where rows start inside a sector (cols a multiple of 16 alone): such rows
// are slower to copy with 256 (M = 1367, N = 6288, 3 shards of 1008: 35.5 us against 32.0; of
// 1040 38.8 against 35.1), others as fast or up to 1.5 % faster.
CUresult encode(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, int box_rows, int kblocks) {
  const bool deep = kblocks > 0;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(deep ? kScaleBlock : cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(cols / kScaleBlock)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(kScaleBlock)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(kScaleBlock), static_cast<cuuint32_t>(box_rows),
                       static_cast<cuuint32_t>(kblocks)};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, deep ? 3 : 2, const_cast<void*>(ptr), dims, strides, box,
                     estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     cols % 32 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Rows of Y in boxes of `width` (64 or 32) columns x 32 rows.
CUresult encode_y(CUtensorMap* m, void* ptr, int64_t rows, int64_t cols, int width) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(width), 32};
  cuuint32_t estr[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE,
                     width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

int64_t pairs_of(const gemm_shard_plan* P) {
  const int cap = P->opt_max_ctas ? std::min(P->opt_max_ctas, P->sm_count) : P->sm_count;
  return std::max<int64_t>(1, std::min<int64_t>(cap / 2, P->pair_clusters));
}

// Of rows and columns: 32-bit coordinates, and one past every shard's rows.
constexpr int64_t kMostRows = (int64_t(1) << 30) - 256;

struct Shape {
  int form, box_rows, boxes, tile_n;
  int64_t m_tiles, n_tiles;
};

// Token tiles if a CTA's `cta_rows` rows are cut into boxes of `box` rows of one shard each.
int64_t token_tiles(int cta_rows, int box, int shards, const int64_t* rows) {
  int64_t boxes = 0;
  for (int r = 0; r < shards; ++r) boxes += cdiv(rows[r], box);
  return cdiv(boxes, 2 * (cta_rows / box));
}

// The token tiles of the best box: the fewest, where a box more in a CTA counts as 5 % of a
// tile (a copy more per k-block) and, in the wide form, boxes that are not of whole warps'
// rows as 12 % (their tiles are not stored by copies); of equal ones the largest.
int64_t best_box(int form, int shards, const int64_t* rows, int* box) {
  const int cta_rows = gsr::fp8_cta_rows(form);
  int64_t best = INT64_MAX, tiles = 0;
  for (int b = cta_rows; b >= 8; b -= 8) {
    const int64_t t = token_tiles(cta_rows, b, shards, rows);
    const int64_t cost = t * (100 + 5 * (cta_rows / b - 1) + (form == gsr::kFp8Wide && b % 32 ? 12 : 0));
    if (cost < best) {
      best = cost;
      tiles = t;
      *box = b;
    }
  }
  return tiles;
}

Shape choose(const gemm_shard_plan* P, int64_t N, int64_t kblocks, int shards, const int64_t* rows) {
  Shape s;
  const int64_t pairs = pairs_of(P);
  const int narrow = gsr::fp8_cta_rows(gsr::kFp8Narrow), wide = gsr::fp8_cta_rows(gsr::kFp8Wide);
  s.form = gsr::kFp8Narrow;
  s.m_tiles = best_box(s.form, shards, rows, &s.box_rows);
  if (s.m_tiles == 1) {
    // One row shard is split evenly over the pair.
    if (shards == 1) s.box_rows = static_cast<int>(cdiv(cdiv(rows[0], 2), 8) * 8);
    s.boxes = shards == 1 ? 1 : narrow / s.box_rows;
    // As few weight rows as spread N over the pairs in the fewest waves.
    const int64_t waves = cdiv(N, 128 * pairs);
    s.tile_n = static_cast<int>(std::min<int64_t>(128, std::max<int64_t>(32, cdiv(cdiv(N, waves * pairs), 32) * 32)));
    s.n_tiles = cdiv(N, s.tile_n);
    return s;
  }
  s.form = gsr::kFp8Wide;
  s.m_tiles = best_box(s.form, shards, rows, &s.box_rows);
  s.boxes = wide / s.box_rows;
  // One row shard in one tile is split evenly here too, in whole warps' rows. (Boxes that hold
  // a few rows of 128 and end inside a shard's k-blocks are slow to copy: 136 rows, 8 K-shards
  // of 7 k-blocks, 25 us against 19.)
  if (shards == 1 && s.m_tiles == 1) s.box_rows = static_cast<int>(cdiv(cdiv(rows[0], 2), 32) * 32);
  // The tile width by the cycles that its waves take: a k-block of 256, 192, 128 or 64 weight
  // rows takes 800, 680, 450 and 320 (the epilogue's chain of waits and reads, and for the
  // narrower ones the copies), a tile's start and store some 2500. Measured with all tiles
  // of 256 / 192 / 128 / 64 (us, N = K = 7168): M = 256 28 / 26 / 20 / 26, 512 29 / 27 / 31 /
  // 37, 1000 51 / 47 / 49 / 68, 4096 148 / 168 / 173 / 253.
  constexpr struct { int n, cycles; } kWidths[] = {{256, 800}, {192, 680}, {128, 450}, {64, 320}};
  int64_t best = INT64_MAX;
  for (const auto& w : kWidths) {
    const int64_t cost = cdiv(s.m_tiles * cdiv(N, w.n), pairs) * (kblocks * w.cycles + 2500);
    if (cost < best) {
      best = cost;
      s.tile_n = w.n;
      s.n_tiles = cdiv(N, w.n);
    }
  }
  return s;
}

// What both products share, from the shards on: K-shards (AR) or row shards (AG).
gsr_status run_fp8(const gemm_shard_plan* P, bool ag, int64_t N, int R, const int64_t* K_r, const int64_t* M_r,
                   const void* const* X, const float* const* SX, const void* const* W, const float* const* SW,
                   void* Y, void* ws, gsr_stream_t stream) {
  const int m_shards = ag ? R : 1, k_shards = ag ? 1 : R;
  int64_t kblocks = 0, k_total = 0;
  for (int r = 0; r < k_shards; ++r) {
    kblocks += cdiv(K_r[r], kScaleBlock);
    k_total += K_r[r];
  }
  if (N > kMostRows || k_total > kMostRows) return fail(GSR_ERR_INVALID_VALUE, "N or K is too large");
  const Shape s = choose(P, N, kblocks, m_shards, M_r);
  const int kz = gsr::fp8_kblocks(s.form, s.tile_n);
  int64_t stages = 0;
  for (int r = 0; r < k_shards; ++r) stages += cdiv(cdiv(K_r[r], kScaleBlock), kz);
  if (s.m_tiles * s.n_tiles > INT32_MAX / 2 || stages > INT32_MAX / 2)
    return fail(GSR_ERR_INVALID_VALUE, "M, N and K give too many tiles");
  const int64_t tiles = s.m_tiles * s.n_tiles;
  const int ctas = static_cast<int>(2 * std::min(pairs_of(P), tiles));
  if (gsr::log_config_enabled())
    std::fprintf(stderr, "gsr: %s_fp8 N=%lld K=%lld R=%d kernel=fp8 form=%s tile_n=%d boxes=%dx%d tiles=%lld ctas=%d\n",
                 ag ? "ag" : "ar", (long long)N, (long long)k_total, R,
                 s.form == gsr::kFp8Wide ? "wide" : "narrow", s.tile_n, s.boxes, s.box_rows, (long long)tiles, ctas);
  if (P->device < 0) return fail(GSR_ERR_UNSUPPORTED, "host plan: arguments are valid, nothing launched");
  if (!encode_fn()) return fail(GSR_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is unavailable");

  gsr::Fp8Params p;
  std::memset(&p, 0, sizeof p);
  p.y = static_cast<uint16_t*>(Y);
  p.status = static_cast<uint32_t*>(ws);
  p.timeout_ns = P->timeout_ns;
  p.ag = ag;
  p.N = static_cast<int>(N);
  p.k_shards = k_shards;
  p.m_shards = m_shards;
  p.tile_n = s.tile_n;
  p.n_tiles = static_cast<int>(s.n_tiles);
  p.m_tiles = static_cast<int>(s.m_tiles);
  p.tiles = static_cast<int>(tiles);
  p.group_m = static_cast<int>(std::min<int64_t>(8, s.m_tiles));
  p.box_rows = s.box_rows;
  p.boxes = s.boxes;
  p.ring = gsr::fp8_ring(s.form, s.tile_n, s.boxes * s.box_rows);
  // One token tile: the weights are read once and stream by.
  p.policy_w = s.m_tiles == 1 ? gsr::kPolicyEvictFirst : gsr::kPolicyNormal;
  p.policy_x = s.m_tiles == 1 ? gsr::kPolicyEvictLast : gsr::kPolicyNormal;
  p.stages_per_tile = static_cast<int>(stages);
  // A stage in one copy per operand, where no shard ends inside a block.
  p.whole_boxes = kz > 1;
  for (int r = 0; r < k_shards; ++r) p.whole_boxes = p.whole_boxes && K_r[r] % kScaleBlock == 0;
  const int w_kb = p.whole_boxes ? kz : 0, x_kb = !p.whole_boxes ? 0 : s.boxes == 1 ? kz : 1;
  CUresult cr = CUDA_SUCCESS;
  int st = 0;
  for (int r = 0; r < k_shards; ++r) {
    p.shard_kb[r] = static_cast<int>(cdiv(K_r[r], kScaleBlock));
    p.shard_st_begin[r] = st;
    st += static_cast<int>(cdiv(p.shard_kb[r], kz));
    p.sw[r] = SW[r];
    if (cr == CUDA_SUCCESS) cr = encode(&p.tmap_w[r], W[r], N, K_r[r], s.tile_n / 2, w_kb);
  }
  for (int r = k_shards; r <= kMaxShards; ++r) p.shard_st_begin[r] = st;
  int box = 0;
  int64_t row = 0;
  for (int r = 0; r < m_shards; ++r) {
    p.box_begin[r] = box;
    box += static_cast<int>(cdiv(M_r[r], s.box_rows));
    p.shard_rows[r] = static_cast<int>(M_r[r]);
    p.shard_row_begin[r] = row;
    row += M_r[r];
    if (M_r[r] > 0) p.pad_shard = r;
  }
  for (int r = m_shards; r <= kMaxShards; ++r) p.box_begin[r] = box;
  for (int r = 0; r < R; ++r) {
    const int64_t rows = ag ? M_r[r] : M_r[0];
    p.sx[r] = SX[r];
    if (rows > 0 && cr == CUDA_SUCCESS) cr = encode(&p.tmap_x[r], X[r], rows, ag ? K_r[0] : K_r[r], s.box_rows, x_kb);
  }
  // A warp's 32 rows lie in one box: the tile's rows are stored by copies, which leave out
  // what a shard does not have.
  p.tma_store = s.form == gsr::kFp8Wide && s.box_rows % 32 == 0;
  if (p.tma_store)
    for (int r = 0; r < m_shards && cr == CUDA_SUCCESS; ++r)
      if (M_r[r] > 0) cr = encode_y(&p.tmap_y[r], p.y + p.shard_row_begin[r] * N, M_r[r], N, gsr::fp8_store_cols(s.tile_n));
  if (cr != CUDA_SUCCESS) return fail(GSR_ERR_CUDA, "encoding the operands' descriptors failed (%d)", (int)cr);
  DeviceScope scope(P->device);
  if (scope.err != cudaSuccess) return cuda_fail(scope.err, "selecting the plan's device");
  const cudaError_t e = gsr::launch_fp8(p, s.form, ctas, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
  return ok();
}

gsr_status check_status_ws(const void* ws, size_t ws_bytes) {
  if (!ws) return fail(GSR_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) & 255u)
    return fail(GSR_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < gsr::kWsHeader)
    return fail(GSR_ERR_WORKSPACE, "workspace too small: %zu bytes given, %zu needed", ws_bytes, gsr::kWsHeader);
  return ok();
}

}  // namespace

extern "C" {

gsr_status gemm_shard_rms_norm(const gemm_shard_plan* P, int64_t M, int64_t H, const void* X, const void* residual,
                               const void* gamma, float eps, void* sum, void* Y, void* Q, float* scale,
                               gsr_stream_t stream) {
  gsr_status s = check_plan(P);
  if (s) return s;
  if (M < 0 || M > P->max_M)
    return fail(GSR_ERR_INVALID_VALUE, "M=%lld outside 0..%lld (the plan's max_M)", (long long)M, (long long)P->max_M);
  const int64_t most = std::min<int64_t>(std::max(P->max_N, P->max_K), gsr::kMaxNormColumns);
  if (H < 8 || H % 8 || H > most)
    return fail(GSR_ERR_INVALID_VALUE, "H=%lld must be a positive multiple of 8, at most %lld", (long long)H,
                (long long)most);
  if (Q && H % 16) return fail(GSR_ERR_INVALID_VALUE, "H=%lld must be a multiple of 16 for Q", (long long)H);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(GSR_ERR_INVALID_VALUE, "eps must be finite and >= 0");
  if (M > 0 && !X) return fail(GSR_ERR_INVALID_VALUE, "X must not be NULL");
  if (M > 0 && !sum && !Y && !Q) return fail(GSR_ERR_INVALID_VALUE, "no output: sum, Y and Q are NULL");
  if (M > 0 && (Q != nullptr) != (scale != nullptr))
    return fail(GSR_ERR_INVALID_VALUE, "Q and scale come together");
  if (!aligned16(X) || !aligned16(residual) || !aligned16(gamma) || !aligned16(sum) || !aligned16(Y) || !aligned16(Q))
    return fail(GSR_ERR_INVALID_VALUE, "X, residual, gamma, sum, Y and Q must be 16-byte aligned");
  if (!aligned4(scale)) return fail(GSR_ERR_INVALID_VALUE, "scale must be 4-byte aligned");
  if (M == 0) return ok();
  if (P->device < 0) return fail(GSR_ERR_UNSUPPORTED, "host plan: arguments are valid, nothing launched");
  gsr::NormParams p = {};
  p.x = static_cast<const uint16_t*>(X);
  p.residual = static_cast<const uint16_t*>(residual);
  p.gamma = static_cast<const uint16_t*>(gamma);
  p.sum = static_cast<uint16_t*>(sum);
  p.y = static_cast<uint16_t*>(Y);
  p.q = static_cast<uint8_t*>(Q);
  p.scale = scale;
  p.M = M;
  p.H = static_cast<int>(H);
  p.eps = eps;
  DeviceScope scope(P->device);
  if (scope.err != cudaSuccess) return cuda_fail(scope.err, "selecting the plan's device");
  const cudaError_t e = gsr::launch_norm(p, P->sm_count, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
  return ok();
}

gsr_status gemm_shard_quantize(const gemm_shard_plan* P, int64_t rows, int64_t cols, int block_rows, const void* X,
                               void* Q, float* scale, gsr_stream_t stream) {
  gsr_status s = check_plan(P);
  if (s) return s;
  if (block_rows != 1 && block_rows != kScaleBlock)
    return fail(GSR_ERR_INVALID_VALUE, "block_rows must be 1 or %d (got %d)", kScaleBlock, block_rows);
  const int64_t most_rows = block_rows == 1 ? P->max_M : P->max_N;
  if (rows < 0 || rows > most_rows)
    return fail(GSR_ERR_INVALID_VALUE, "rows=%lld outside 0..%lld (the plan's %s)", (long long)rows,
                (long long)most_rows, block_rows == 1 ? "max_M" : "max_N");
  if (cols < 16 || cols % 16 || cols > P->max_K || cols > INT32_MAX - 256)
    return fail(GSR_ERR_INVALID_VALUE, "cols=%lld must be a positive multiple of 16, at most the plan's max_K=%lld",
                (long long)cols, (long long)P->max_K);
  if (cdiv(rows, 16) * cdiv(cols, kScaleBlock) > INT32_MAX)   // (a grid of fewer CTAs in either form)
    return fail(GSR_ERR_INVALID_VALUE, "rows and cols give too many groups");
  if (rows > 0 && (!X || !Q || !scale)) return fail(GSR_ERR_INVALID_VALUE, "X, Q and scale must not be NULL");
  if (!aligned16(X) || !aligned16(Q) || !aligned4(scale))
    return fail(GSR_ERR_INVALID_VALUE, "X and Q must be 16-byte aligned, scale 4-byte aligned");
  if (rows == 0) return ok();
  if (P->device < 0) return fail(GSR_ERR_UNSUPPORTED, "host plan: arguments are valid, nothing launched");
  gsr::QuantParams p = {};
  p.x = static_cast<const uint16_t*>(X);
  p.q = static_cast<uint8_t*>(Q);
  p.scale = scale;
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  p.block_rows = block_rows;
  DeviceScope scope(P->device);
  if (scope.err != cudaSuccess) return cuda_fail(scope.err, "selecting the plan's device");
  const cudaError_t e = gsr::launch_quantize(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
  return ok();
}

gsr_status gemm_ar_fp8(const gemm_shard_plan* P, int64_t M, int64_t N, int R, const int64_t* K_r,
                       const void* const* X_r, const float* const* SX_r, const void* const* W_r,
                       const float* const* SW_r, void* Y, void* ws, size_t ws_bytes, gsr_stream_t stream) {
  gsr_status s = check_plan(P);
  if (s) return s;
  s = gsr::check_ksharded(P, M, N, R, K_r, X_r, W_r);
  if (s) return s;
  if (M > kMostRows) return fail(GSR_ERR_INVALID_VALUE, "M=%lld is too large", (long long)M);
  if (!SX_r || !SW_r) return fail(GSR_ERR_INVALID_VALUE, "SX_r and SW_r must not be NULL");
  for (int r = 0; r < R; ++r) {
    if (K_r[r] % 16)
      return fail(GSR_ERR_INVALID_VALUE, "K_r[%d]=%lld must be a multiple of 16", r, (long long)K_r[r]);
    if ((M > 0 && !SX_r[r]) || !SW_r[r] || !aligned4(SX_r[r]) || !aligned4(SW_r[r]))
      return fail(GSR_ERR_INVALID_VALUE, "SX_r[%d] and SW_r[%d] must be non-NULL and 4-byte aligned", r, r);
  }
  if ((M > 0 && !Y) || !aligned16(Y))
    return fail(GSR_ERR_INVALID_VALUE, "Y must be non-NULL and 16-byte aligned");
  s = check_status_ws(ws, ws_bytes);
  if (s) return s;
  if (M == 0) return ok();
  return run_fp8(P, false, N, R, K_r, &M, X_r, SX_r, W_r, SW_r, Y, ws, stream);
}

gsr_status gemm_ag_fp8(const gemm_shard_plan* P, int64_t N, int64_t K, int R, const int64_t* M_r,
                       const void* const* A_r, const float* const* SA_r, const void* W, const float* SW, void* Y,
                       void* ws, size_t ws_bytes, gsr_stream_t stream) {
  gsr_status s = check_plan(P);
  if (s) return s;
  if (R < 1 || R > P->max_R) return fail(GSR_ERR_INVALID_VALUE, "R=%d outside 1..%d", R, P->max_R);
  if (!M_r || !A_r || !SA_r) return fail(GSR_ERR_INVALID_VALUE, "M_r, A_r and SA_r must not be NULL");
  int64_t M = 0;
  for (int r = 0; r < R; ++r) {
    if (M_r[r] < 0 || M_r[r] > P->max_M || (M += M_r[r]) > P->max_M)
      return fail(GSR_ERR_INVALID_VALUE, "M_r[%d]=%lld: rows outside 0..%lld in total (the plan's max_M)", r,
                  (long long)M_r[r], (long long)P->max_M);
    if (M_r[r] > 0 && (!A_r[r] || !aligned16(A_r[r]) || !SA_r[r] || !aligned4(SA_r[r])))
      return fail(GSR_ERR_INVALID_VALUE, "A_r[%d] must be non-NULL and 16-byte aligned, SA_r[%d] 4-byte aligned", r, r);
  }
  if (M > kMostRows) return fail(GSR_ERR_INVALID_VALUE, "M=%lld is too large", (long long)M);
  if (N < 8 || N % 8 || N > P->max_N)
    return fail(GSR_ERR_INVALID_VALUE, "N=%lld must be a positive multiple of 8, at most the plan's max_N=%lld",
                (long long)N, (long long)P->max_N);
  if (K < 16 || K % 16 || K > P->max_K)
    return fail(GSR_ERR_INVALID_VALUE, "K=%lld must be a positive multiple of 16, at most the plan's max_K=%lld",
                (long long)K, (long long)P->max_K);
  if (!W || !aligned16(W) || !SW || !aligned4(SW))
    return fail(GSR_ERR_INVALID_VALUE, "W must be non-NULL and 16-byte aligned, SW 4-byte aligned");
  if ((M > 0 && !Y) || !aligned16(Y))
    return fail(GSR_ERR_INVALID_VALUE, "Y must be non-NULL and 16-byte aligned");
  s = check_status_ws(ws, ws_bytes);
  if (s) return s;
  if (M == 0) return ok();
  return run_fp8(P, true, N, R, &K, M_r, A_r, SA_r, &W, &SW, Y, ws, stream);
}

}  // extern "C"
