// gsr_routed_api.cu -- host side of the routed projections' entry points
// (include/gsr.h): argument checks, choice of the kernel instance, tensor maps
// and launches. Nothing here allocates device memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstring>

#include "gsr.h"
#include "gsr_host.h"
#include "gsr_layer.h"
#include "gsr_routed.h"

using gsr::aligned16;
using gsr::BK;
using gsr::cdiv;
using gsr::check_plan;
using gsr::cuda_fail;
using gsr::DeviceScope;
using gsr::encode_fn;
using gsr::fail;
using gsr::ok;
using gsr::round256;

namespace {

// k of one ring stage.
int stage_k(bool half, int tokens) { return gsr::routed_kblocks(half, tokens) * BK; }

// CTA pairs a launch may use.
int64_t pairs_of(const gemm_shard_plan* P) {
  const int cap = P->opt_max_ctas ? std::min(P->opt_max_ctas, P->sm_count) : P->sm_count;
  return std::max<int64_t>(1, std::min<int64_t>(cap / 2, P->pair_clusters));
}

// Workspace regions after the header and the counters.
size_t partial_bytes(const gemm_shard_plan* P) {
  // A pair has one piece at most: a slot per pair, one half per CTA.
  const size_t pairs = static_cast<size_t>(std::max(1, P->sm_count / 2));
  return pairs * 2 * gsr::kRoutedDouble * 128 * sizeof(float);
}
size_t low_bytes(const gemm_shard_plan* P) {
  return round256(static_cast<size_t>(P->max_M) * gsr::kMaxRank * 2);
}
int64_t max_lists(const gemm_shard_plan* P) { return P->max_M / 128 + 2; }
size_t list_bytes(const gemm_shard_plan* P) {
  return round256(static_cast<size_t>(max_lists(P)) * gsr::kAdapterListStride * sizeof(int32_t));
}
// The expert layer's rows between its products and after them, and its route.
size_t layer_rows_bytes(const gemm_shard_plan* P) {
  return round256(static_cast<size_t>(std::min<int64_t>(P->max_M, gsr::kLayerMost)) * P->max_N * 2);
}
constexpr size_t kLayerRouteBytes = 4 * (gsr::kMaxGroups + 64 + 2 * gsr::kLayerMost);
size_t layer_bytes(const gemm_shard_plan* P) { return 2 * layer_rows_bytes(P) + kLayerRouteBytes; }
constexpr size_t kPartialsAt = gsr::kWsHeader + gsr::kRoutedCounterBytes;

size_t workspace_bytes(const gemm_shard_plan* P) {
  return kPartialsAt + partial_bytes(P) + low_bytes(P) + list_bytes(P) + layer_bytes(P);
}

gsr_status check_routed_ws(const gemm_shard_plan* P, const void* ws, size_t ws_bytes) {
  if (!ws) return fail(GSR_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) & 255u)
    return fail(GSR_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  const size_t need = workspace_bytes(P);
  if (ws_bytes < need)
    return fail(GSR_ERR_WORKSPACE, "workspace too small: %zu bytes given, %zu needed", ws_bytes, need);
  // Two counters per cut tile, fewer cut tiles than pairs.
  if (static_cast<size_t>(P->sm_count) * sizeof(uint32_t) > gsr::kRoutedCounterBytes)
    return fail(GSR_ERR_UNSUPPORTED, "more than %zu SMs", gsr::kRoutedCounterBytes / sizeof(uint32_t));
  return ok();
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

CUresult encode_2d(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, int box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(BK), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// The same rows as {64 columns, rows, k-blocks} (cols a multiple of 64), in boxes of
// kblocks k-blocks, which land one after the other.
CUresult encode_kblocks(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, int box_rows,
                        int kblocks) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(BK), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(cols / BK)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(BK) * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(BK), static_cast<cuuint32_t>(box_rows),
                       static_cast<cuuint32_t>(kblocks)};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// count matrices of rows x cols, one after the other; boxes of box_cols (16, 32 or
// 64, the swizzle's width) x box_rows.
CUresult encode_stack(CUtensorMap* m, const void* ptr, int64_t count, int64_t rows, int64_t cols,
                      int box_cols, int box_rows) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(count)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(cols) * rows * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapSwizzle swizzle = box_cols == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                      : CU_TENSOR_MAP_SWIZZLE_32B;
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Fields that every kind shares. `tokens`: the instance's capacity, `kblocks`: of a stage.
void fill_routed(gsr::RoutedParams& p, const gemm_shard_plan* P, int64_t M, int64_t N, int stages,
                 int kblocks, int tokens, void* ws) {
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.stages_per_tile = stages;
  // How finely a remainder of tiles is cut: narrow tiles are streams of weights
  // with small partials, wide ones pay 128 KB of partial per piece and CTA.
  // Cutting costs the partials' way through L2 and the last arrival's sum. Measured
  // in whole tiles / cut ones (us, K = 7168): 8 tiles of 64 tokens 21.9 / 16.9 in 9
  // pieces, 24 23.5 / 23.4 in 3, 36 27.7 / 28.9 in 2; of 256 tokens, 16 41.3 / 32.5, 36
  // 44.1 / 43.0; after one more wave, 36 of 64 tokens 67.4 / 66.0, of 256 91.1 / 83.6.
  // K = 2048: 16 tiles of 256 tokens 17.3 / 23.3, 12 of 64 tokens after a wave 22.9 /
  // 23.4. So a cut has to save some 60 k-blocks (narrow) or 52, or 40 after a wave.
  p.max_pieces = tokens == gsr::kRoutedSmall ? 32 : tokens == gsr::kRoutedMid ? 8 : 4;
  p.cut_alone = (tokens <= gsr::kRoutedMid ? 60 : 52) / kblocks;
  p.cut_ahead = 40 / kblocks;
  p.timeout_ns = P->timeout_ns;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.status = reinterpret_cast<uint32_t*>(w);
  p.counters = reinterpret_cast<uint32_t*>(w + gsr::kWsHeader);
  p.partials = reinterpret_cast<float*>(w + kPartialsAt);
}

// A grouped product's tiles along N, and the limits of its tiles and of a group's matrix.
int64_t grouped_n_tiles(int kind, int64_t N) { return cdiv(N, kind == gsr::kGated ? 128 : 256); }
gsr_status check_grouped_size(int kind, int E, int64_t M, int64_t N, int64_t K) {
  const int64_t wide = kind == gsr::kGated ? 2 * N : N;
  if (wide * K >= (int64_t(1) << 38) || (cdiv(M, 64) + E) * grouped_n_tiles(kind, N) > INT32_MAX / 2)
    return fail(GSR_ERR_INVALID_VALUE, "M, N, K and E give too many tiles or too large a matrix");
  return ok();
}

gsr_status run_grouped(const gemm_shard_plan* P, int kind, int E, int64_t M, int64_t N, int64_t K,
                       const int32_t* offsets, int64_t T, const void* X, const int32_t* rows,
                       const void* W, void* Y, void* ws, size_t ws_bytes, gsr_stream_t stream) {
  gsr_status s = check_plan(P);
  if (s) return s;
  if (E < 1 || E > gsr::kMaxGroups)
    return fail(GSR_ERR_INVALID_VALUE, "E=%d outside 1..%d", E, gsr::kMaxGroups);
  if (M < 0 || M > P->max_M)
    return fail(GSR_ERR_INVALID_VALUE, "M=%lld outside 0..%lld (the plan's max_M)", (long long)M,
                (long long)P->max_M);
  if (N < 8 || N % 8 || N > P->max_N)
    return fail(GSR_ERR_INVALID_VALUE, "N=%lld must be a positive multiple of 8, at most the plan's max_N=%lld",
                (long long)N, (long long)P->max_N);
  if (K < 8 || K % 8 || K > P->max_K)
    return fail(GSR_ERR_INVALID_VALUE, "K=%lld must be a positive multiple of 8, at most the plan's max_K=%lld",
                (long long)K, (long long)P->max_K);
  if (T < 0 || T > INT32_MAX - 256 || (!rows && T < M) || (M > 0 && T < 1))
    return fail(GSR_ERR_INVALID_VALUE, "T=%lld: X needs at least %s", (long long)T,
                rows ? "one row" : "M rows");
  if (!offsets || !aligned_to(offsets, 4) || !aligned_to(rows, 4))
    return fail(GSR_ERR_INVALID_VALUE, "offsets must be non-NULL, offsets and rows 4-byte aligned");
  if (!W || !aligned16(W)) return fail(GSR_ERR_INVALID_VALUE, "W must be non-NULL and 16-byte aligned");
  if ((M > 0 && (!X || !Y)) || !aligned16(X) || !aligned16(Y))
    return fail(GSR_ERR_INVALID_VALUE, "X and Y must be non-NULL and 16-byte aligned");
  s = check_grouped_size(kind, E, M, N, K);
  if (s) return s;
  const int64_t wide = kind == gsr::kGated ? 2 * N : N, n_tiles = grouped_n_tiles(kind, N);
  s = check_routed_ws(P, ws, ws_bytes);
  if (s) return s;
  if (M == 0) return ok();

  // The instance by the mean group: the rows of a group are few where the
  // weights are the traffic, and a capacity near them leaves shared memory for a
  // deeper ring; but groups differ in size, and one larger than the capacity reads its
  // weights again. Any instance is right for any sizes. Measured with 64 groups of
  // uneven sizes (64 / 128 / 256 tokens, us): grouped N = 7168, K = 896, mean 16 128 / 126
  // / 130, 32 133 / 130 / 132, 64 146 / 137 / 137, 96 168 / 149 / 143, 128 192 / 159 / 150;
  // gated N = 896, K = 7168, gathered, 16 239 / 243 / 256, 32 243 / 245 / 259, 64 258 / 255
  // / 267, 96 302 / 270 / 280, 128 334 / 285 / 293.
  // Large groups: tiles of 512 tokens read the weights half as often from L2, but have
  // one accumulator, so nothing hides the epilogue, and fewer sizes between them. Rows
  // that do not start on 128-byte lines take two lines per 128 bytes of k: L2 then
  // bounds the product and the larger tiles pay. Measured with 16 groups or fewer, N =
  // 4096 (256 / 512 tokens, us), 384 rows per group: K = 264 34 / 33, 520 47 / 43, 1000 71 /
  // 62, but 1024 49 / 55, 4096 152 / 151; 2048 rows: 264 129 / 113, 520 186 / 148, 1000
  // 290 / 230, but 1024 168 / 205, 2048 159 / 175, 4096 154 / 159, 7168 146 / 132.
  // With gathered rows the copies' latency eats the gain (567 / 622, K = 7168).
  // The mean counts the empty groups, so rows that meet few of many groups get narrower
  // tiles: 1024 rows in 4 of 64 groups (64 tokens) / in 4 of 4 (256): N = 7168, K = 896 22.6 /
  // 22.7 us, gated, N = 896, K = 7168, 40.9 / 51.7 (narrow tiles fill more pairs); in one of
  // 64 22.4 / in one of one (256) 16.5.
  const int64_t mean = cdiv(M, E);
  const int tokens = mean <= 24   ? gsr::kRoutedSmall
                     : mean <= 96 ? gsr::kRoutedMid
                     : mean <= gsr::kRoutedWide || K % BK == 0 || rows ? gsr::kRoutedWide
                                                                      : gsr::kRoutedDouble;
  const int64_t ctas = 2 * std::min<int64_t>(pairs_of(P), (cdiv(M, tokens) + E) * n_tiles *
                                                              cdiv(K, 2 * stage_k(false, tokens)));
  if (gsr::log_config_enabled())
    std::fprintf(stderr, "gsr: %s M=%lld N=%lld K=%lld E=%d gather=%d kernel=routed tokens=%d ctas=%lld\n",
                 kind == gsr::kGated ? "grouped_gated" : "grouped", (long long)M, (long long)N,
                 (long long)K, E, rows ? 1 : 0, tokens, (long long)ctas);
  if (P->device < 0) return fail(GSR_ERR_UNSUPPORTED, "host plan: arguments are valid, nothing launched");
  if (!encode_fn()) return fail(GSR_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is unavailable");

  gsr::RoutedParams p;
  std::memset(&p, 0, sizeof p);
  fill_routed(p, P, M, N, static_cast<int>(cdiv(K, stage_k(false, tokens))),
              gsr::routed_kblocks(false, tokens), tokens, ws);
  p.E = E;
  p.T = static_cast<int>(T);
  p.K = static_cast<int>(K);
  p.x = static_cast<const uint16_t*>(X);
  p.offsets = offsets;
  p.rows = rows;
  p.y = static_cast<uint16_t*>(Y);
  p.n_tiles = static_cast<int>(n_tiles);
  p.cta_cols = kind == gsr::kGated ? 64 : 128;
  p.w_rows = 128;
  p.policy_w = tokens >= gsr::kRoutedWide ? gsr::kPolicyNormal : gsr::kPolicyEvictFirst;
  p.policy_x = tokens >= gsr::kRoutedWide ? gsr::kPolicyNormal : gsr::kPolicyEvictLast;
  CUresult cr = encode_stack(&p.tmap_w[0], W, E, wide, K, BK, kind == gsr::kGated ? 64 : 128);
  if (cr != CUDA_SUCCESS) return fail(GSR_ERR_CUDA, "encoding the W descriptor failed (%d)", (int)cr);
  if (!rows)
    for (int i = 0; i < std::min(tokens, 256) / 16 && cr == CUDA_SUCCESS; ++i)
      cr = encode_2d(&p.tmap_x[i], X, M, K, 8 * (i + 1));
  if (cr != CUDA_SUCCESS) return fail(GSR_ERR_CUDA, "encoding the X descriptor failed (%d)", (int)cr);
  DeviceScope scope(P->device);
  if (scope.err != cudaSuccess) return cuda_fail(scope.err, "selecting the plan's device");
  cudaError_t e = gsr::launch_routed(p, kind, rows != nullptr, false, tokens, static_cast<int>(ctas),
                                     reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
  return ok();
}

}  // namespace

extern "C" {

size_t gemm_routed_workspace_size(const gemm_shard_plan* P) { return P ? workspace_bytes(P) : 0; }

gsr_status gemm_routed_workspace_init(const gemm_shard_plan* P, void* ws, size_t ws_bytes,
                                      gsr_stream_t stream) {
  gsr_status s = check_plan(P);
  if (s) return s;
  s = check_routed_ws(P, ws, ws_bytes);
  if (s) return s;
  if (P->device < 0) return fail(GSR_ERR_UNSUPPORTED, "host plan: nothing to initialise");
  DeviceScope scope(P->device);
  if (scope.err != cudaSuccess) return cuda_fail(scope.err, "selecting the plan's device");
  cudaError_t e = cudaMemsetAsync(ws, 0, kPartialsAt, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  return ok();
}

gsr_status gemm_group_route(const gemm_shard_plan* P, int64_t T, int topk, int E, const void* ids,
                            int id_bytes, int32_t* offsets, int32_t* source, int32_t* position,
                            gsr_stream_t stream) {
  gsr_status s = check_plan(P);
  if (s) return s;
  if (E < 1 || E > gsr::kMaxGroups)
    return fail(GSR_ERR_INVALID_VALUE, "E=%d outside 1..%d", E, gsr::kMaxGroups);
  if (topk < 1 || topk > gsr::kMaxTopk)
    return fail(GSR_ERR_INVALID_VALUE, "topk=%d outside 1..%d", topk, gsr::kMaxTopk);
  if (T < 0 || T > P->max_M || T * topk > P->max_M)
    return fail(GSR_ERR_INVALID_VALUE, "T=%lld: T * topk outside 0..%lld (the plan's max_M)",
                (long long)T, (long long)P->max_M);
  if (T * topk > (int64_t(1) << 30))
    return fail(GSR_ERR_INVALID_VALUE, "T * topk exceeds 2^30");
  if (id_bytes != 4 && id_bytes != 8)
    return fail(GSR_ERR_INVALID_VALUE, "id_bytes must be 4 or 8 (got %d)", id_bytes);
  if (!offsets || !aligned_to(offsets, 4))
    return fail(GSR_ERR_INVALID_VALUE, "offsets must be non-NULL and 4-byte aligned");
  if (T > 0 && (!ids || !source || !position))
    return fail(GSR_ERR_INVALID_VALUE, "ids, source and position must not be NULL");
  if (!aligned_to(ids, id_bytes) || !aligned_to(source, 4) || !aligned_to(position, 4))
    return fail(GSR_ERR_INVALID_VALUE, "ids, source and position must be aligned to their elements");
  if (P->device < 0) return fail(GSR_ERR_UNSUPPORTED, "host plan: arguments are valid, nothing launched");
  gsr::RouteParams p = {};
  p.ids = ids;
  p.offsets = offsets;
  p.source = source;
  p.position = position;
  p.n = static_cast<int>(T * topk);
  p.topk = topk;
  p.E = E;
  p.wide = id_bytes == 8;
  DeviceScope scope(P->device);
  if (scope.err != cudaSuccess) return cuda_fail(scope.err, "selecting the plan's device");
  cudaError_t e = gsr::launch_route(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
  return ok();
}

gsr_status gemm_grouped(const gemm_shard_plan* P, int E, int64_t M, int64_t N, int64_t K,
                        const int32_t* offsets, int64_t T, const void* X, const int32_t* rows,
                        const void* W, void* Y, void* ws, size_t ws_bytes, gsr_stream_t stream) {
  return run_grouped(P, gsr::kGrouped, E, M, N, K, offsets, T, X, rows, W, Y, ws, ws_bytes, stream);
}

gsr_status gemm_grouped_gated(const gemm_shard_plan* P, int E, int64_t M, int64_t N, int64_t K,
                              const int32_t* offsets, int64_t T, const void* X, const int32_t* rows,
                              const void* W, void* Y, void* ws, size_t ws_bytes, gsr_stream_t stream) {
  return run_grouped(P, gsr::kGated, E, M, N, K, offsets, T, X, rows, W, Y, ws, ws_bytes, stream);
}

gsr_status gemm_group_combine(const gemm_shard_plan* P, int64_t T, int topk, int64_t H,
                              int64_t z_rows, const void* Z, const int32_t* position,
                              const float* weights, const void* base, void* Y, gsr_stream_t stream) {
  gsr_status s = check_plan(P);
  if (s) return s;
  if (topk < 1 || topk > gsr::kMaxTopk)
    return fail(GSR_ERR_INVALID_VALUE, "topk=%d outside 1..%d", topk, gsr::kMaxTopk);
  if (T < 0 || T > P->max_M)
    return fail(GSR_ERR_INVALID_VALUE, "T=%lld outside 0..%lld (the plan's max_M)", (long long)T,
                (long long)P->max_M);
  if (H < 8 || H % 8 || H > P->max_N)
    return fail(GSR_ERR_INVALID_VALUE, "H=%lld must be a positive multiple of 8, at most the plan's max_N=%lld",
                (long long)H, (long long)P->max_N);
  if (z_rows < 0 || z_rows > INT32_MAX)
    return fail(GSR_ERR_INVALID_VALUE, "z_rows=%lld must be >= 0 and below 2^31", (long long)z_rows);
  if (T > 0 && (!position || !weights || !Y || (z_rows > 0 && !Z)))
    return fail(GSR_ERR_INVALID_VALUE, "Z, position, weights and Y must not be NULL");
  if (!aligned16(Z) || !aligned16(base) || !aligned16(Y))
    return fail(GSR_ERR_INVALID_VALUE, "Z, base and Y must be 16-byte aligned");
  if (!aligned_to(position, 4) || !aligned_to(weights, 4))
    return fail(GSR_ERR_INVALID_VALUE, "position and weights must be 4-byte aligned");
  if (T == 0) return ok();
  if (P->device < 0) return fail(GSR_ERR_UNSUPPORTED, "host plan: arguments are valid, nothing launched");
  gsr::CombineParams p = {};
  p.z = static_cast<const uint16_t*>(Z);
  p.position = position;
  p.weights = weights;
  p.base = static_cast<const uint16_t*>(base);
  p.y = static_cast<uint16_t*>(Y);
  p.T = T;
  p.z_rows = z_rows;
  p.topk = topk;
  p.vecs = static_cast<int>(H / 8);
  DeviceScope scope(P->device);
  if (scope.err != cudaSuccess) return cuda_fail(scope.err, "selecting the plan's device");
  cudaError_t e = gsr::launch_combine(p, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
  return ok();
}

gsr_status gemm_expert_layer(const gemm_shard_plan* P, int64_t T, int topk, int E, int64_t N, int64_t K,
                             const void* ids, int id_bytes, const float* weights, const void* X, const void* W_up,
                             const void* W_down, const void* base, void* Y, void* ws, size_t ws_bytes,
                             gsr_stream_t stream) {
  gsr_status s = check_plan(P);
  if (s) return s;
  if (E < 1 || E > gsr::kMaxGroups)
    return fail(GSR_ERR_INVALID_VALUE, "E=%d outside 1..%d", E, gsr::kMaxGroups);
  if (topk < 1 || topk > gsr::kMaxTopk)
    return fail(GSR_ERR_INVALID_VALUE, "topk=%d outside 1..%d", topk, gsr::kMaxTopk);
  if (T < 0 || T > gsr::kLayerTokens || T * topk > gsr::kLayerMost || T * topk > P->max_M)
    return fail(GSR_ERR_INVALID_VALUE, "T=%lld outside 0..%d, or T * topk above %d or the plan's max_M=%lld",
                (long long)T, gsr::kLayerTokens, gsr::kLayerMost, (long long)P->max_M);
  // Either width is an output's and a reduction's.
  const int64_t widest = std::min<int64_t>(std::min(P->max_N, P->max_K), 1 << 20);
  if (N < 8 || N % 8 || N > widest)
    return fail(GSR_ERR_INVALID_VALUE, "N=%lld must be a positive multiple of 8, at most the plan's max_N and max_K (%lld)",
                (long long)N, (long long)widest);
  if (K < 8 || K % 8 || K > widest)
    return fail(GSR_ERR_INVALID_VALUE, "K=%lld must be a positive multiple of 8, at most the plan's max_N and max_K (%lld)",
                (long long)K, (long long)widest);
  if (id_bytes != 4 && id_bytes != 8)
    return fail(GSR_ERR_INVALID_VALUE, "id_bytes must be 4 or 8 (got %d)", id_bytes);
  if (T > 0 && (!ids || !weights || !X || !Y))
    return fail(GSR_ERR_INVALID_VALUE, "ids, weights, X and Y must not be NULL");
  if (!aligned_to(ids, id_bytes) || !aligned_to(weights, 4))
    return fail(GSR_ERR_INVALID_VALUE, "ids and weights must be aligned to their elements");
  if (!W_up || !W_down || !aligned16(W_up) || !aligned16(W_down))
    return fail(GSR_ERR_INVALID_VALUE, "W_up and W_down must be non-NULL and 16-byte aligned");
  if (!aligned16(X) || !aligned16(base) || !aligned16(Y))
    return fail(GSR_ERR_INVALID_VALUE, "X, base and Y must be 16-byte aligned");
  // Both products' limits, before the first launch, and for either form alike.
  s = check_grouped_size(gsr::kGated, E, T * topk, N, K);
  if (!s) s = check_grouped_size(gsr::kGrouped, E, T * topk, K, N);
  if (s) return s;
  s = check_routed_ws(P, ws, ws_bytes);
  if (s) return s;
  if (T == 0) return ok();
  if (gsr::log_config_enabled())
    std::fprintf(stderr, "gsr: expert_layer T=%lld topk=%d E=%d N=%lld K=%lld kernel=%s\n", (long long)T, topk, E,
                 (long long)N, (long long)K, gsr::layer_in_two(T * topk, E) ? "layer" : "routed");
  if (P->device < 0) return fail(GSR_ERR_UNSUPPORTED, "host plan: arguments are valid, nothing launched");
  uint8_t* rows = static_cast<uint8_t*>(ws) + workspace_bytes(P) - layer_bytes(P);
  if (!gsr::layer_in_two(T * topk, E)) {
    void* z = rows + layer_rows_bytes(P);
    int32_t* offsets = reinterpret_cast<int32_t*>(rows + 2 * layer_rows_bytes(P));
    int32_t *source = offsets + gsr::kMaxGroups + 64, *position = source + gsr::kLayerMost;
    const int64_t M = T * topk;
    s = gemm_group_route(P, T, topk, E, ids, id_bytes, offsets, source, position, stream);
    if (!s) s = run_grouped(P, gsr::kGated, E, M, N, K, offsets, T, X, source, W_up, rows, ws, ws_bytes, stream);
    if (!s) s = run_grouped(P, gsr::kGrouped, E, M, K, N, offsets, M, rows, nullptr, W_down, z, ws, ws_bytes, stream);
    if (!s) s = gemm_group_combine(P, T, topk, K, M, z, position, weights, base, Y, stream);
    return s;
  }
  gsr::LayerParams p = {};
  p.ids = ids;
  p.weights = weights;
  p.x = static_cast<const uint16_t*>(X);
  p.up = static_cast<const uint16_t*>(W_up);
  p.down = static_cast<const uint16_t*>(W_down);
  p.base = static_cast<const uint16_t*>(base);
  p.h = reinterpret_cast<uint16_t*>(rows);
  p.y = static_cast<uint16_t*>(Y);
  p.T = static_cast<int>(T);
  p.topk = topk;
  p.E = E;
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.wide = id_bytes == 8;
  DeviceScope scope(P->device);
  if (scope.err != cudaSuccess) return cuda_fail(scope.err, "selecting the plan's device");
  cudaError_t e = gsr::launch_layer(p, P->sm_count, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
  return ok();
}

gsr_status gemm_ar_lora(const gemm_shard_plan* P, int64_t M, int64_t N, int R, const int64_t* K_r,
                        const void* const* X_r, const void* const* W_r, int L, int rank,
                        const void* const* A_r, const void* B, const int32_t* adapter,
                        const float* scale, void* Y, void* ws, size_t ws_bytes, gsr_stream_t stream) {
  gsr_status s = check_plan(P);
  if (s) return s;
  s = gsr::check_ksharded(P, M, N, R, K_r, X_r, W_r);
  if (s) return s;
  if (L < 1 || L > gsr::kMaxAdapters)
    return fail(GSR_ERR_INVALID_VALUE, "L=%d outside 1..%d", L, gsr::kMaxAdapters);
  if (rank < 8 || rank % 8 || rank > gsr::kMaxRank)
    return fail(GSR_ERR_INVALID_VALUE, "rank=%d must be a multiple of 8 in 8..%d", rank, gsr::kMaxRank);
  if (!A_r) return fail(GSR_ERR_INVALID_VALUE, "A_r must not be NULL");
  for (int r = 0; r < R; ++r)
    if (!A_r[r] || !aligned16(A_r[r]))
      return fail(GSR_ERR_INVALID_VALUE, "A_r[%d] must be non-NULL and 16-byte aligned", r);
  if (!B || !aligned16(B)) return fail(GSR_ERR_INVALID_VALUE, "B must be non-NULL and 16-byte aligned");
  if ((M > 0 && !adapter) || !aligned_to(adapter, 4) || !aligned_to(scale, 4))
    return fail(GSR_ERR_INVALID_VALUE, "adapter must be non-NULL, adapter and scale 4-byte aligned");
  if ((M > 0 && !Y) || !aligned16(Y))
    return fail(GSR_ERR_INVALID_VALUE, "Y must be non-NULL and 16-byte aligned");
  s = check_routed_ws(P, ws, ws_bytes);
  if (s) return s;
  if (M == 0) return ok();

  // Up to 256 rows run as one token tile, a stream of weights: tiles of at most
  // 128 weight rows, as few as spread N over the pairs in the fewest waves (N = 7168
  // on 76 pairs: 96 rows, 75 tiles, none cut; at M = 128, cutting 256-row tiles
  // instead spent 10 us of 40 on the partials). Fewer than 64 rows make the copies
  // too small: then tiles are cut.
  const bool half = M <= gsr::kRoutedWide;
  const int tokens = M <= gsr::kRoutedSmall ? gsr::kRoutedSmall
                     : M <= gsr::kRoutedMid ? gsr::kRoutedMid
                                            : gsr::kRoutedWide;
  const int64_t m_tiles = cdiv(M, tokens);
  const int64_t width = cdiv(cdiv(M, m_tiles), 16) * 16;
  int64_t tile_rows = gsr::kRoutedTileRows;
  if (half) {
    const int64_t waves = cdiv(N, 128 * pairs_of(P));
    tile_rows = std::min<int64_t>(128, std::max<int64_t>(64, cdiv(cdiv(N, waves * pairs_of(P)), 16) * 16));
  }
  const int64_t n_tiles = cdiv(N, tile_rows);
  if (m_tiles * n_tiles > INT32_MAX / 2) return fail(GSR_ERR_INVALID_VALUE, "M and N give too many tiles");
  const int kStageK = stage_k(half, tokens);
  int64_t stages = 0;
  for (int r = 0; r < R; ++r) stages += cdiv(K_r[r], kStageK);
  const int64_t ctas = 2 * std::min(pairs_of(P), m_tiles * n_tiles * cdiv(stages, 2));
  if (gsr::log_config_enabled())
    std::fprintf(stderr, "gsr: ar_lora M=%lld N=%lld R=%d L=%d rank=%d kernel=routed tokens=%d ctas=%lld\n",
                 (long long)M, (long long)N, R, L, rank, tokens, (long long)ctas);
  if (P->device < 0) return fail(GSR_ERR_UNSUPPORTED, "host plan: arguments are valid, nothing launched");
  if (!encode_fn()) return fail(GSR_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is unavailable");

  uint8_t* w = static_cast<uint8_t*>(ws);
  uint16_t* low = reinterpret_cast<uint16_t*>(w + kPartialsAt + partial_bytes(P));
  int32_t* lists = reinterpret_cast<int32_t*>(w + kPartialsAt + partial_bytes(P) + low_bytes(P));

  gsr::RoutedParams p;
  std::memset(&p, 0, sizeof p);
  fill_routed(p, P, M, N, static_cast<int>(stages), gsr::routed_kblocks(half, tokens), tokens, ws);
  p.R = R;
  p.L = L;
  p.adapter = adapter;
  p.low = low;
  p.b = static_cast<const uint16_t*>(B);
  p.rank = rank;
  p.lists = lists;
  p.y = static_cast<uint16_t*>(Y);
  p.n_tiles = static_cast<int>(n_tiles);
  p.cta_cols = p.w_rows = static_cast<int>(tile_rows / 2);
  if (half) {
    const int64_t stage = kStageK / BK * (128 * p.w_rows + 64 * width);
    p.stages = static_cast<int>(std::min<int64_t>(gsr::kHalfSlots, gsr::kHalfRing / stage));
  }
  p.m_tiles = static_cast<int>(m_tiles);
  p.tile_tokens = static_cast<int>(width);
  p.unit_cols = rank <= 16 ? 16 : rank <= 32 ? 32 : 64;
  p.units_per_adapter = rank <= 64 ? 1 : 2;
  p.rank_pad = p.unit_cols * p.units_per_adapter;
  p.scale = scale;
  // A row or a few of low rank: the product computes their low-rank rows itself, and
  // is the call's only kernel.
  p.self_rows = M <= gsr::kSelfRows && M * p.rank_pad <= gsr::kSelfElements;
  p.policy_w = m_tiles == 1 ? gsr::kPolicyEvictFirst : gsr::kPolicyNormal;
  p.policy_x = m_tiles == 1 ? gsr::kPolicyEvictLast : gsr::kPolicyNormal;
  // One copy per operand and stage where no shard ends inside a k-block (a view by
  // k-blocks would read the next row there). One row without an adapter: 22.6 us, with
  // a copy per k-block 24.3.
  p.whole_boxes = half;
  for (int r = 0; r < R; ++r) p.whole_boxes = p.whole_boxes && K_r[r] % BK == 0;
  gsr::LowRankParams q;
  std::memset(&q, 0, sizeof q);
  int st = 0;
  for (int r = 0; r < R; ++r) {
    p.shard_st_begin[r] = st;
    st += static_cast<int>(cdiv(K_r[r], kStageK));
    q.x[r] = static_cast<const uint16_t*>(X_r[r]);
    q.a[r] = static_cast<const uint16_t*>(A_r[r]);
    q.k[r] = K_r[r];
    p.x_r[r] = q.x[r];
    p.a_r[r] = q.a[r];
    p.k_r[r] = static_cast<int>(K_r[r]);
    const int x_rows = static_cast<int>(width / 2), kb = kStageK / BK;
    CUresult cr = p.whole_boxes ? encode_kblocks(&p.tmap_w[r], W_r[r], N, K_r[r], p.w_rows, kb)
                                : encode_2d(&p.tmap_w[r], W_r[r], N, K_r[r], p.w_rows);
    if (cr == CUDA_SUCCESS)
      cr = p.whole_boxes ? encode_kblocks(&p.tmap_x[r], X_r[r], M, K_r[r], x_rows, kb)
                         : encode_2d(&p.tmap_x[r], X_r[r], M, K_r[r], x_rows);
    if (cr != CUDA_SUCCESS) return fail(GSR_ERR_CUDA, "encoding shard %d's descriptors failed (%d)", r, (int)cr);
  }
  for (int r = R; r <= gsr::kMaxShards; ++r) p.shard_st_begin[r] = st;
  CUresult cr = encode_stack(&p.tmap_b, B, L, N, rank, p.unit_cols, p.w_rows);
  if (cr != CUDA_SUCCESS) return fail(GSR_ERR_CUDA, "encoding the B descriptor failed (%d)", (int)cr);
  q.adapter = adapter;
  q.scale = scale;
  q.low = low;
  q.lists = lists;
  q.M = static_cast<int>(M);
  q.R = R;
  q.L = L;
  q.rank = rank;
  q.rank_pad = p.rank_pad;
  q.tile_tokens = p.tile_tokens;
  q.m_tiles = p.m_tiles;
  DeviceScope scope(P->device);
  if (scope.err != cudaSuccess) return cuda_fail(scope.err, "selecting the plan's device");
  cudaStream_t st_ = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = p.self_rows ? cudaSuccess : gsr::launch_low_rank(q, st_);
  if (e == cudaSuccess) e = gsr::launch_routed(p, gsr::kLora, false, half, tokens, static_cast<int>(ctas), st_);
  if (e != cudaSuccess) return cuda_fail(e, "kernel launch");
  return ok();
}

}  // extern "C"
