// gsr_host.h -- host-side pieces shared by the translation units that implement
// the C ABI (internal to the library): the plan object, error recording, the
// driver's tensor-map encoder and small helpers. Defined in gsr_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gsr.h"

struct gemm_shard_plan {
  int device;
  int sm_count;
  int64_t max_M, max_N, max_K;
  int max_R;
  int opt_split;       // 0 = heuristic
  int opt_block_n;     // 0 = heuristic
  int opt_max_ctas;    // 0 = one per SM
  int opt_raster_m;    // 0 = heuristic
  int opt_raster_n;    // 0 = raster by m-tile groups
  int opt_l2_hints;    // 0 = heuristic
  int opt_cta_group;   // 0 = heuristic
  int opt_schedule;    // 0 = heuristic, 1 = uniform, 2 = stream-K over the last one or two
                       // waves, 3/4 = stream-K over a partial last wave (its range first /
                       // last), 5 = split tail (GSR_OPT_SCHEDULE in gsr.h)
  int opt_small;       // 0 = heuristic, 1 = never use the small-M kernel, 2 = always when it applies
  int opt_small_rows;  // small-M kernel: W rows per tile (0 = heuristic)
  int opt_small_kz;    // small-M kernel: k-blocks per copy (0 = heuristic)
  int64_t l2_bytes;    // the device's L2 size
  int pair_clusters;   // CTA pairs that can be resident at once
  int quad_clusters;   // clusters of two CTA pairs that can be resident at once
  uint64_t timeout_ns;
};

namespace gsr {

// Records the message that gsr_last_error_string() returns on this thread.
gsr_status fail(gsr_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gsr_status cuda_fail(cudaError_t e, const char* what);
inline gsr_status ok() { return GSR_OK; }

// cuTensorMapEncodeTiled through the runtime's driver entry point, so that the
// library itself has no link-time dependency on the driver library. NULL when
// the driver has none.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();

// Restores the caller's current device on scope exit.
struct DeviceScope {
  int prev = -1;
  bool switched = false;
  cudaError_t err = cudaSuccess;
  explicit DeviceScope(int dev) {
    err = cudaGetDevice(&prev);
    if (err == cudaSuccess && prev != dev) {
      err = cudaSetDevice(dev);
      switched = (err == cudaSuccess);
    }
  }
  ~DeviceScope() {
    if (switched) cudaSetDevice(prev);
  }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

gsr_status check_plan(const gemm_shard_plan* P);
// Shared validation of the K-sharded (AR/RS) argument lists.
gsr_status check_ksharded(const gemm_shard_plan* P, int64_t M, int64_t N, int R, const int64_t* K_r,
                          const void* const* X_r, const void* const* W_r);
bool log_config_enabled();

}  // namespace gsr
