// gsr_quant.cu -- the residual sum with its RMS norm, and the quantisation to 8
// bits, for GB300: what runs between two projections.
//
//   h = x + residual,  y = h * (mean(h^2) + eps)^-1/2 * gamma
//   scale = max(max|v| / 448, 2^-126) over a group,  q = e4m3(v * (1 / scale))
//
// A group is 128 columns of a row, or a block of 128 x 128. All of it in fp32; sum and
// y are rounded to bf16 once, and q comes from the unrounded y. The maximum keeps NaN,
// so a group that holds NaN or infinity has such a scale, and its products are NaN as
// they would be without the scale.
//
// Both are bound by memory. Norm: a CTA holds a row in registers, 8 columns per vector
// and thread, so that 16 lanes are a group; it loads its next row before it reduces this
// one. Every element is read once and written once. 32768 rows of 7168 with every output
// 340 us (0.92 of the copy bandwidth; 10 of it are the scales, 4 bytes at a time), without
// the row ahead 374; 16 rows 2.7, a launch. Quantisation: 16384 rows of 7168 55 us (0.95),
// weights of 6288 x 7168 22.6 (0.88).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gsr_fp8.h"

namespace gsr {
namespace {

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The larger, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

__device__ __forceinline__ float largest(const float (&f)[8]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
  return m;
}

__device__ __forceinline__ float scale_of(float most) { return max_nan(most / 448.f, 0x1p-126f); }

// 8 values times `inv` in e4m3, to nearest even, at most 448 in magnitude.
__device__ __forceinline__ uint2 to_e4m3(const float (&f)[8], float inv) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(f[2 * i + 1] * inv), "f"(f[2 * i] * inv));
  return make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
}

__device__ __forceinline__ float max_of_16(float m) {
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// Read once by this kernel and by nothing soon after.
__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}

// ------------------------------------------------------------ norm

// VECS 4 (rows of more than 8192 columns) has no registers for the next row, and with a
// residual spills (96 bytes stored and 172 loaded a thread).
template <int VECS>
constexpr int kNormThreads = VECS == 2 ? 512 : 1024;

template <int VECS, bool RES>
__global__ void __launch_bounds__(kNormThreads<VECS>, VECS == 2 ? 2 : 1) gsr_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sums[2][32];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int threads = static_cast<int>(blockDim.x), warps = threads >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int vecs = p.H >> 3;
  uint4 gamma[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int v = tid + i * threads;
    gamma[i] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    if (p.gamma && v < vecs) gamma[i] = *reinterpret_cast<const uint4*>(p.gamma + 8 * v);
  }
  uint4 x[VECS], r[VECS];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int v = tid + i * threads;
      if (v < vecs) {
        x[i] = load_once(p.x + row * p.H + 8 * v);
        if constexpr (RES) r[i] = load_once(p.residual + row * p.H + 8 * v);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < VECS; ++i) x[i] = r[i] = make_uint4(0, 0, 0, 0);
  int64_t row = blockIdx.x;
  constexpr bool kAhead = VECS <= 2;
  if constexpr (kAhead) load(row);   // the grid has no more CTAs than rows
  for (int turn = 0; row < p.M; turn ^= 1) {
    if constexpr (!kAhead) load(row);
    float h[VECS][8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      unpack(x[i], h[i]);
      if constexpr (RES) {
        float f[8];
        unpack(r[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += f[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(h[i][j], h[i][j], sum);
    }
    const int64_t next = row + gridDim.x;
    // Every thread has read its own part of its row alone, and writes it alone: the
    // next row's loads cannot meet this row's stores where sum or Y is X or residual. (Q is
    // none of them: its rows are half as long and would lie on other CTAs' rows.)
    if constexpr (kAhead)
      if (next < p.M) load(next);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) sums[turn][warp] = sum;
    __syncthreads();
    sum = lane < warps ? sums[turn][lane] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const float norm = 1.f / sqrtf(sum / static_cast<float>(p.H) + p.eps);
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int v = tid + i * threads;
      const bool in = v < vecs;
      const size_t at = static_cast<size_t>(row) * p.H + 8 * v;
      if (p.sum && in) *reinterpret_cast<uint4*>(p.sum + at) = pack(h[i]);
      float g[8];
      unpack(gamma[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * norm * g[j];
      if (p.y && in) *reinterpret_cast<uint4*>(p.y + at) = pack(h[i]);
      if (p.q) {
        // (Lanes past the row hold zeros, but a norm that is not finite makes them NaN.)
        const float scale = scale_of(max_of_16(in ? largest(h[i]) : 0.f));
        if (in) *reinterpret_cast<uint2*>(p.q + at) = to_e4m3(h[i], 1.f / scale);
        if (in && (v & 15) == 0) p.scale[static_cast<size_t>(v >> 4) * p.M + row] = scale;
      }
    }
    row = next;
  }
}

// ------------------------------------------------------------ quantisation

constexpr int kQuantThreads = 256;
constexpr int kRowUnits = 4;   // groups of a row that 16 lanes hold

// 16 rows x 4 groups of 128 columns per CTA: 16 lanes hold a row's four groups, 1 KB of it.
// The scales leave together, 64 bytes of a column block at a time (4 bytes at a time from
// wherever a group was, 16384 rows of 7168 took 76 us).
__global__ void __launch_bounds__(kQuantThreads) gsr_quantize_rows_kernel(const __grid_constant__ QuantParams p) {
  constexpr int kRows = kQuantThreads / 16;
  __shared__ float scales[kRowUnits][kRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = static_cast<int>(threadIdx.x), team = tid >> 4;
  const int groups = (p.cols + kScaleBlock - 1) / kScaleBlock;
  const uint32_t parts = static_cast<uint32_t>((groups + kRowUnits - 1) / kRowUnits);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / parts) * kRows, row = row0 + team;
  const int group0 = static_cast<int>(blockIdx.x % parts) * kRowUnits;
  const int col0 = group0 * kScaleBlock + 8 * (tid & 15);
  const int64_t at = row * p.cols + col0;
  uint4 v[kRowUnits];
#pragma unroll
  for (int i = 0; i < kRowUnits; ++i) {
    v[i] = make_uint4(0, 0, 0, 0);
    if (row < p.rows && col0 + i * kScaleBlock < p.cols) v[i] = load_once(p.x + at + i * kScaleBlock);
  }
#pragma unroll
  for (int i = 0; i < kRowUnits; ++i) {
    float f[8];
    unpack(v[i], f);
    const float scale = scale_of(max_of_16(largest(f)));
    if (row < p.rows && col0 + i * kScaleBlock < p.cols)
      *reinterpret_cast<uint2*>(p.q + at + i * kScaleBlock) = to_e4m3(f, 1.f / scale);
    if ((tid & 15) == 0) scales[i][team] = scale;
  }
  __syncthreads();
  if (tid < kRowUnits * kRows) {
    const int i = tid / kRows, r = tid % kRows;
    if (row0 + r < p.rows && group0 + i < groups) p.scale[(group0 + i) * p.rows + row0 + r] = scales[i][r];
  }
}

// A block of 128 x 128 per CTA: 16 lanes a row, 8 rows per thread.
__global__ void __launch_bounds__(kQuantThreads) gsr_quantize_blocks_kernel(const __grid_constant__ QuantParams p) {
  __shared__ float most[kQuantThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kHeld = kScaleBlock * 16 / kQuantThreads;
  const int tid = static_cast<int>(threadIdx.x);
  const uint32_t groups = static_cast<uint32_t>((p.cols + kScaleBlock - 1) / kScaleBlock);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / groups) * kScaleBlock + (tid >> 4);
  const int col = static_cast<int>(blockIdx.x % groups) * kScaleBlock + 8 * (tid & 15);
  uint4 v[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int64_t row = row0 + i * (kQuantThreads / 16);
    v[i] = make_uint4(0, 0, 0, 0);
    if (row < p.rows && col < p.cols) v[i] = load_once(p.x + row * p.cols + col);
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    float f[8];
    unpack(v[i], f);
    m = max_nan(m, largest(f));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((tid & 31) == 0) most[tid >> 5] = m;
  __syncthreads();
  m = most[0];
#pragma unroll
  for (int i = 1; i < kQuantThreads / 32; ++i) m = max_nan(m, most[i]);
  const float scale = scale_of(m), inv = 1.f / scale;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int64_t row = row0 + i * (kQuantThreads / 16);
    float f[8];
    unpack(v[i], f);
    if (row < p.rows && col < p.cols) *reinterpret_cast<uint2*>(p.q + row * p.cols + col) = to_e4m3(f, inv);
  }
  if (tid == 0) p.scale[blockIdx.x] = scale;
}

template <class P>
cudaError_t launch_one(void (*kernel)(const P), const P& p, dim3 grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int VECS>
cudaError_t launch_norm_as(const NormParams& p, int sm_count, cudaStream_t stream) {
  const int threads = (p.H / 8 + 32 * VECS - 1) / (32 * VECS) * 32;
  const int64_t resident = static_cast<int64_t>(sm_count) * std::max(1, 1024 / threads);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(p.M, resident)));
  return p.residual ? launch_one(gsr_norm_kernel<VECS, true>, p, grid, threads, stream)
                    : launch_one(gsr_norm_kernel<VECS, false>, p, grid, threads, stream);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int sm_count, cudaStream_t stream) {
  const int vecs = p.H / 8;
  if (vecs > 1024) return launch_norm_as<4>(p, sm_count, stream);
  if (p.M <= sm_count) return launch_norm_as<1>(p, sm_count, stream);
  return launch_norm_as<2>(p, sm_count, stream);
}

cudaError_t launch_quantize(const QuantParams& p, cudaStream_t stream) {
  const int64_t groups = (p.cols + kScaleBlock - 1) / kScaleBlock;
  if (p.block_rows == 1) {
    const int64_t ctas = (groups + kRowUnits - 1) / kRowUnits * ((p.rows + kQuantThreads / 16 - 1) / (kQuantThreads / 16));
    return launch_one(gsr_quantize_rows_kernel, p, dim3(static_cast<unsigned>(ctas)), kQuantThreads, stream);
  }
  const dim3 grid(static_cast<unsigned>(groups * ((p.rows + kScaleBlock - 1) / kScaleBlock)));
  return launch_one(gsr_quantize_blocks_kernel, p, grid, kQuantThreads, stream);
}

}  // namespace gsr
