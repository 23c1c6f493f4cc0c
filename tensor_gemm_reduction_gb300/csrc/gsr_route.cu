// gsr_route.cu -- the route (a stable counting sort of expert ids) and the
// combine (the experts' rows weighted and added back per token), for GB300.
//
// Route. n ids, E groups: offsets[e] = ids below e that are in 0..E-1, position[i]
// = offsets[id] + earlier entries with the same id, source[position[i]] = i /
// topk. One cluster, one launch: every warp owns a run of entries and a row of
// counts in shared memory; 32 entries at a time are matched by id, so counts
// need no atomics and the order is the entries'. Warps' counts are summed per
// CTA, CTAs' totals are read through distributed shared memory, and every CTA
// scans the groups itself. The second pass over the ids (L2) places them.
//
// Combine. Y[t] = base[t] + sum_j weight[t, j] * Z[position[t, j]], fp32, j
// ascending, rounded once. Bound by reading Z: each thread owns 16 bytes of a
// row and keeps the loads of eight rows in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gsr_routed.h"

namespace gsr {
namespace {

constexpr int kRouteWarps = 32;
constexpr int kRouteThreads = 32 * kRouteWarps;
constexpr int kRouteCluster = 16;       // CTAs, for many entries
static_assert(kMaxGroups <= kRouteThreads, "one thread per group in the scan");

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(a), "r"(rank));
  return out;
}

__device__ __forceinline__ int load_id(const RouteParams& p, int i) {
  if (i >= p.n) return -1;
  if (p.wide) {
    const long long v = __ldg(reinterpret_cast<const long long*>(p.ids) + i);
    return v >= 0 && v < p.E ? static_cast<int>(v) : -1;
  }
  const int v = __ldg(reinterpret_cast<const int*>(p.ids) + i);
  return v >= 0 && v < p.E ? v : -1;
}

__global__ void __launch_bounds__(kRouteThreads, 1) gsr_route_kernel(const RouteParams p) {
  extern __shared__ int counts[];                       // [kRouteWarps][E]
  __shared__ int totals[kMaxGroups], base[kMaxGroups], sums[32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  const int per = ((p.n + ctas * kRouteWarps - 1) / (ctas * kRouteWarps) + 31) & ~31;
  const long long run = static_cast<long long>(cta * kRouteWarps + warp) * per;
  const int i0 = static_cast<int>(run < p.n ? run : p.n);
  const int i1 = static_cast<int>(run + per < p.n ? run + per : p.n);
  int* mine = counts + warp * p.E;
  for (int e = lane; e < p.E; e += 32) mine[e] = 0;
  __syncwarp();

  for (int i = i0; i < i1; i += 32) {
    const int id = load_id(p, i + lane < i1 ? i + lane : p.n);
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    if (id >= 0 && lane == __ffs(same) - 1) mine[id] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // Per group: each warp's count becomes the sum of the warps before it.
  if (tid < p.E) {
    int at = 0;
    for (int w = 0; w < kRouteWarps; ++w) {
      const int c = counts[w * p.E + tid];
      counts[w * p.E + tid] = at;
      at += c;
    }
    totals[tid] = at;
  }
  __syncwarp();   // .aligned: whole warps arrive
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
  int before = 0, all = 0;
  if (tid < p.E) {
    for (int c = 0; c < ctas; ++c) {
      int v;
      asm volatile("ld.shared::cluster.s32 %0, [%1];"
                   : "=r"(v)
                   : "r"(remote(totals + tid, static_cast<uint32_t>(c))));
      if (c < cta) before += v;
      all += v;
    }
  }
  int incl = all;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int start = incl - all, kept = 0;
  for (int w = 0; w < kRouteWarps; ++w) {
    if (w < warp) start += sums[w];
    kept += sums[w];
  }
  if (tid < p.E) {
    base[tid] = start + before;
    if (cta == 0) {
      p.offsets[tid] = start;
      if (tid == p.E - 1) p.offsets[p.E] = kept;
    }
  }
  __syncthreads();

  for (int i = i0; i < i1; i += 32) {
    const int at = i + lane;
    const int id = load_id(p, at < i1 ? at : p.n);
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    int position = -1;
    if (id >= 0) position = base[id] + mine[id] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (id >= 0 && lane == __ffs(same) - 1) mine[id] += __popc(same);
    __syncwarp();
    if (at < i1) {
      p.position[at] = position;
      if (position >= 0) p.source[position] = at / p.topk;
    }
  }
  for (int i = kept + cta * kRouteThreads + tid; i < p.n; i += ctas * kRouteThreads) p.source[i] = -1;
  // No CTA leaves while another may still read its totals.
  __syncwarp();   // .aligned: whole warps arrive
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

__device__ __forceinline__ void add_row(float (&acc)[8], uint4 v, float w) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(w, __uint_as_float(u[i] << 16), acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, __uint_as_float(u[i] & 0xffff0000u), acc[2 * i + 1]);
  }
}

__global__ void __launch_bounds__(256) gsr_combine_kernel(const CombineParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t total = p.T * p.vecs, step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += step) {
    const int64_t t = i / p.vecs;
    const int c = static_cast<int>(i - t * p.vecs);
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    if (p.base) add_row(acc, __ldg(reinterpret_cast<const uint4*>(p.base) + i), 1.f);
    const int32_t* pos = p.position + t * p.topk;
    const float* wts = p.weights + t * p.topk;
    for (int j0 = 0; j0 < p.topk; j0 += 8) {
      uint4 v[8];
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = j0 + j < p.topk ? __ldg(pos + j0 + j) : -1;
        const bool live = at >= 0 && at < p.z_rows;
        // An absent entry adds nothing, whatever its weight is.
        w[j] = live ? __ldg(wts + j0 + j) : 0.f;
        v[j] = live ? __ldg(reinterpret_cast<const uint4*>(p.z) + static_cast<int64_t>(at) * p.vecs + c)
                    : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) add_row(acc, v[j], w[j]);
    }
    uint4 out;
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * j], acc[2 * j + 1]);
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    out = make_uint4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<uint4*>(p.y)[i] = out;
  }
}

cudaError_t launch_pdl(const void* kernel, dim3 grid, int threads, size_t smem, int cluster,
                       void** args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace

cudaError_t prepare_route_kernels() {
  cudaError_t e = cudaFuncSetAttribute(gsr_route_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kRouteWarps * kMaxGroups * static_cast<int>(sizeof(int)));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(gsr_route_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
  const int ctas = p.n <= 4096 ? 1 : kRouteCluster;
  RouteParams q = p;
  void* args[] = {&q};
  return launch_pdl(reinterpret_cast<const void*>(gsr_route_kernel), dim3(ctas), kRouteThreads,
                    static_cast<size_t>(kRouteWarps) * p.E * sizeof(int), ctas, args, stream);
}

cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream) {
  const int64_t blocks = (p.T * p.vecs + 255) / 256;
  const unsigned grid = static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30));
  CombineParams q = p;
  void* args[] = {&q};
  return launch_pdl(reinterpret_cast<const void*>(gsr_combine_kernel), dim3(grid), 256, 0, 0, args, stream);
}

}  // namespace gsr
