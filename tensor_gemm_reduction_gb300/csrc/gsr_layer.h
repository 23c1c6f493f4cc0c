// gsr_layer.h -- launch parameters of the few-token expert layer (internal to the
// library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gsr {

constexpr int kLayerTokens = 64;        // T, at most
constexpr int kLayerMost = 1024;        // T * topk, at most
// T * topk up to which the two kernels run, and the same per expert. Beyond them the entries'
// rows, which are read for every 8 or 16 columns, are the traffic, and the routed
// products, with up to 256 tokens a tile, are faster. Measured, the two kernels / the four
// routed ones (us): one entry of one expert, N = 896, K = 7168, 18 / 29; 4 of 128, N = 256, K =
// 7168, 17 / 31; 8 of 64, N = 896, K = 7168, 50 / 65, 128 325 / 323, 256 452 / 358, 512 604 / 365;
// 64 of 8, same widths, 58 / 66, N = 1024, K = 4096, 53 / 50; 64 of 16, 78 / 79; 64 of 4, N =
// K = 2048, 46 / 34; 128 of 32, N = 512, K = 2048, 61 / 49; 183 of 7, N = 1000, K = 1832, 47 / 34.
// (Sizes alone do not tell the sides apart everywhere: 64 of 8 at the smaller widths lose 3 us.)
// The routed form's down products leave their kernel as rows of bf16, as every product's
// rows do, before the combine weights them in fp32: one rounding more. Relative error
// against 64 bits 0.0017 to 0.0018 in two kernels, 0.0018 to 0.0019 in the routed ones.
constexpr int kLayerEntries = 64, kLayerPerExpert = 8;
inline bool layer_in_two(int64_t entries, int E) {
  return entries <= kLayerEntries && entries <= static_cast<int64_t>(kLayerPerExpert) * E;
}

struct LayerParams {
  const void* ids;          // T x topk
  const float* weights;     // T x topk
  const uint16_t* x;        // T x K
  const uint16_t* up;       // E x 2 N x K
  const uint16_t* down;     // E x K x N
  const uint16_t* base;     // T x K, or NULL
  uint16_t* h;              // workspace: T * topk x N
  uint16_t* y;              // T x K
  int T, topk, E, N, K;
  int wide;                 // 64-bit ids
};

cudaError_t launch_layer(const LayerParams& p, int sm_count, cudaStream_t stream);

}  // namespace gsr
