// gsr_layer.h -- launch parameters of the few-token expert layer (internal to the
// library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gsr {

constexpr int kLayerTokens = 64;      // T, at most
constexpr int kLayerEntries = 1024;   // T * topk, at most

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
