// gsr_route.cu -- the route (a stable counting sort of expert ids) and the
// combine (the experts' rows weighted and added back per token), for GB300.
//
// Route. n ids, E groups: offsets[e] = ids below e that are in 0..E-1, position[i]
// = offsets[id] + earlier entries with the same id, source[position[i]] = i /
// topk. One cluster, one launch: every warp owns a run of entries and a row of
// counts in shared memory; 32 entries at a time are matched by id, so counts
// need no atomics and the order is the entries'. Warps' counts are summed per
// CTA, CTAs' totals are read through distributed shared memory, and every CTA
// scans the groups itself. Up to 16384 entries per CTA stay in registers with their
// places, and are ordered in shared memory first, so that source is written in
// runs (scattered, 262144 entries took 37 us, most of it 32 sectors per store);
// more are read and matched a second time and written where they belong.
//
// Combine. Y[t] = base[t] + sum_j weight[t, j] * Z[position[t, j]], fp32, j
// ascending, rounded once. Bound by reading Z: each thread owns 16 bytes of a
// row and keeps the loads of eight rows in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gsr_routed.h"

namespace gsr {
namespace {

constexpr int kRouteWarps = 32;         // at most
constexpr int kRouteThreads = 32 * kRouteWarps;
constexpr int kRouteCluster = 16;       // CTAs, for many entries
constexpr int kHeld = 16;               // entries per thread that stay in registers
constexpr int kHeldMax = kRouteThreads * kHeld;   // per CTA

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(a), "r"(rank));
  return out;
}

// The lanes with this lane's id (-1 .. 2^bits - 2). A ballot per bit takes a few
// issue slots; the match instruction took about 50 cycles per warp on an SM.
__device__ __forceinline__ uint32_t same_id(int id, int bits) {
  uint32_t same = 0xffffffffu;
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = __ballot_sync(0xffffffffu, (id + 1) >> b & 1);
    same &= (id + 1) >> b & 1 ? set : ~set;
  }
  return same;
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

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();   // .aligned: whole warps arrive
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// HELD: every thread's entries (at most kHeld) stay in registers.
template <bool HELD>
__global__ void __launch_bounds__(kRouteThreads, 1) gsr_route_kernel(const RouteParams p) {
  extern __shared__ int counts[];        // [warps][E], then (HELD) the CTA's entries in order
  __shared__ int totals[kMaxGroups];     // this CTA's entries of each group
  __shared__ int base[kMaxGroups];       // first sorted row of the CTA's entries of the group
  __shared__ int begin[kMaxGroups];      // its first place among the CTA's entries
  __shared__ int sums[kRouteWarps], local_sums[kRouteWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int threads = static_cast<int>(blockDim.x), warps = threads >> 5;
  const int ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  const int per = ((p.n + ctas * warps - 1) / (ctas * warps) + 31) & ~31;   // entries of a warp
  const long long run = static_cast<long long>(cta * warps + warp) * per;
  const int i0 = static_cast<int>(run < p.n ? run : p.n);
  const int i1 = static_cast<int>(run + per < p.n ? run + per : p.n);
  const int bits = 32 - __clz(p.E);   // of id + 1, 0 .. E
  int* mine = counts + warp * p.E;
  int held[kHeld];   // the entry's id, then also its place among the warp's: id << 16 | place
  if constexpr (HELD) {
    // All loads at once: a branch on the ids' width between them would have each
    // wait for the one before.
    if (p.wide) {
      long long v[kHeld];
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const int i = i0 + 32 * j + lane;
        v[j] = i < i1 ? __ldg(reinterpret_cast<const long long*>(p.ids) + i) : -1;
      }
#pragma unroll
      for (int j = 0; j < kHeld; ++j) held[j] = v[j] >= 0 && v[j] < p.E ? static_cast<int>(v[j]) : -1;
    } else {
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        const int i = i0 + 32 * j + lane;
        held[j] = i < i1 ? __ldg(reinterpret_cast<const int*>(p.ids) + i) : -1;
      }
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        if (held[j] < 0 || held[j] >= p.E) held[j] = -1;
    }
  }
  for (int e = lane; e < p.E; e += 32) mine[e] = 0;
  __syncwarp();

  // Counts the group's entries of the warp; the place of this one among them.
  auto count = [&](int id) {
    const uint32_t same = same_id(id, bits);
    const int before = id >= 0 ? mine[id] : 0;
    __syncwarp();
    if (id >= 0 && lane == __ffs(same) - 1) mine[id] = before + __popc(same);
    __syncwarp();
    return before + __popc(same & ((1u << lane) - 1u));
  };
  if constexpr (HELD) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (i0 + 32 * j >= i1) break;
      const int place = count(held[j]);
      if (held[j] >= 0) held[j] = held[j] << 16 | place;
    }
  } else {
    for (int i = i0; i < i1; i += 32) count(load_id(p, i + lane < i1 ? i + lane : p.n));
  }
  __syncthreads();
  // Each thread a run of groups. Per group, each warp's count becomes the sum of
  // the warps before it.
  const int eper = (p.E + threads - 1) / threads, e0 = min(tid * eper, p.E), e1 = min(e0 + eper, p.E);
  for (int e = e0; e < e1; ++e) {
    int at = 0;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const int c = counts[w * p.E + e];
      counts[w * p.E + e] = at;
      at += c;
    }
    totals[e] = at;
  }
  if (ctas > 1)
    cluster_sync();
  else
    __syncthreads();
  // Group totals over the cluster, and the scans over the groups.
  int all = 0, local = 0;
  for (int e = e0; e < e1; ++e) {
    int v[kRouteCluster], before = 0, sum = 0;
#pragma unroll
    for (int c = 0; c < kRouteCluster; ++c) {
      v[c] = 0;
      if (c < ctas)
        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                     : "=r"(v[c])
                     : "r"(remote(totals + e, static_cast<uint32_t>(c))));
    }
#pragma unroll
    for (int c = 0; c < kRouteCluster; ++c) {
      if (c < cta) before += v[c];
      sum += v[c];
    }
    base[e] = before + all;   // all, local: of this thread's groups before e
    begin[e] = local;
    if (cta == 0) p.offsets[e] = all;
    all += sum;
    local += totals[e];
  }
  int incl = all, local_incl = local;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d), u = __shfl_up_sync(0xffffffffu, local_incl, d);
    if (lane >= d) {
      incl += v;
      local_incl += u;
    }
  }
  if (lane == 31) {
    sums[warp] = incl;
    local_sums[warp] = local_incl;
  }
  __syncthreads();
  int start = incl - all, local_start = local_incl - local, kept = 0, local_kept = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) {
      start += sums[w];
      local_start += local_sums[w];
    }
    kept += sums[w];
    local_kept += local_sums[w];
  }
  for (int e = e0; e < e1; ++e) {
    base[e] += start;
    begin[e] += local_start;
    if (cta == 0) p.offsets[e] += start;   // written above by this thread
  }
  if (cta == 0 && tid == 0) p.offsets[p.E] = kept;
  __syncthreads();

  if constexpr (HELD) {
    int* ordered = counts + warps * p.E;   // id << 16 | place among the CTA's entries
    const int first = cta * warps * per;   // the CTA's first entry (HELD: n is small)
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int i = i0 + 32 * j + lane;
      if (i0 + 32 * j >= i1) break;
      int position = -1;
      if (held[j] >= 0) {
        const int id = held[j] >> 16, place = (held[j] & 0xffff) + mine[id];
        position = base[id] + place;
        ordered[begin[id] + place] = id << 16 | (i - first);
      }
      if (i < i1) p.position[i] = position;
    }
    __syncthreads();
    for (int j = tid; j < local_kept; j += threads) {
      const int id = ordered[j] >> 16;
      const uint32_t i = static_cast<uint32_t>(first + (ordered[j] & 0xffff));
      p.source[base[id] + j - begin[id]] = static_cast<int>(p.topk == 1 ? i : __umulhi(i, p.topk_magic));
    }
  } else {
    for (int i = i0; i < i1; i += 32) {
      const int at = i + lane;
      const int id = load_id(p, at < i1 ? at : p.n);
      const int place = count(id);
      const int position = id >= 0 ? base[id] + place : -1;
      if (at < i1) {
        p.position[at] = position;
        if (position >= 0) p.source[position] = at / p.topk;
      }
    }
  }
  for (int i = kept + cta * threads + tid; i < p.n; i += ctas * threads) p.source[i] = -1;
  if (ctas > 1) cluster_sync();   // no CTA leaves while another may still read its totals
}

__device__ __forceinline__ void add_row(float (&acc)[8], uint4 v, float w) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(w, __uint_as_float(u[i] << 16), acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, __uint_as_float(u[i] & 0xffff0000u), acc[2 * i + 1]);
  }
}

// A read that is not kept in L1 (each row of Z is read once).
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// ITEMS 16-byte vectors of Y per thread, 256 apart. Registers for three blocks per
// SM keep 16 rows' reads in flight per thread: 8192 tokens x 8 rows of 7168 in 160 us
// (0.96 of the copy bandwidth), against 184 with the 64 registers that the compiler
// takes by itself and 179 with one vector per thread.
template <int ITEMS>
__global__ void __launch_bounds__(256, ITEMS == 2 ? 3 : 4) gsr_combine_kernel(const CombineParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t total = p.T * p.vecs, step = static_cast<int64_t>(gridDim.x) * (256 * ITEMS);
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * (256 * ITEMS) + threadIdx.x; i0 < total; i0 += step) {
    float acc[ITEMS][8];
    int64_t t[ITEMS];
    const uint4* z[ITEMS];
#pragma unroll
    for (int q = 0; q < ITEMS; ++q) {
      const int64_t i = i0 + 256 * q;
      t[q] = i < total ? i / p.vecs : 0;
      z[q] = reinterpret_cast<const uint4*>(p.z) + (i - t[q] * p.vecs);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[q][j] = 0.f;
      if (p.base && i < total) add_row(acc[q], __ldg(reinterpret_cast<const uint4*>(p.base) + i), 1.f);
    }
    for (int j0 = 0; j0 < p.topk; j0 += 8) {
      uint4 v[ITEMS][8];
      float w[ITEMS][8];
#pragma unroll
      for (int q = 0; q < ITEMS; ++q) {
        const int32_t* pos = p.position + t[q] * p.topk + j0;
        const float* wts = p.weights + t[q] * p.topk + j0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = j0 + j < p.topk && i0 + 256 * q < total ? __ldg(pos + j) : -1;
          const bool live = at >= 0 && at < p.z_rows;
          // An absent entry adds nothing, whatever its weight is.
          w[q][j] = live ? __ldg(wts + j) : 0.f;
          v[q][j] = live ? load_once(z[q] + static_cast<int64_t>(at) * p.vecs) : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int q = 0; q < ITEMS; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) add_row(acc[q], v[q][j], w[q][j]);
    }
#pragma unroll
    for (int q = 0; q < ITEMS; ++q) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(acc[q][2 * j], acc[q][2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if (i0 + 256 * q < total)
        __stcs(reinterpret_cast<uint4*>(p.y) + i0 + 256 * q, make_uint4(o[0], o[1], o[2], o[3]));
    }
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
  cudaError_t e = cudaSuccess;
  const void* kernels[] = {reinterpret_cast<const void*>(gsr_route_kernel<true>),
                           reinterpret_cast<const void*>(gsr_route_kernel<false>)};
  for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
    const int bytes = kRouteWarps * kMaxGroups * 4 + (i == 0 ? kHeldMax * 4 : 0);
    e = cudaFuncSetAttribute(kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kernels[i], cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  }
  return e;
}

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
  // Few entries: one CTA, with warps for 128 entries each. Many: the cluster.
  const int ctas = p.n <= 4096 ? 1 : kRouteCluster;
  const int threads = p.n <= 1024 ? 256 : kRouteThreads;
  const bool held = p.n <= ctas * threads * kHeld;
  const size_t smem = static_cast<size_t>(threads / 32) * p.E * sizeof(int) +
                      (held ? static_cast<size_t>(threads) * kHeld * sizeof(int) : 0);
  RouteParams q = p;
  // i / topk = (i * magic) >> 32 while i * (magic * topk - 2^32) < 2^32, that is for i <
  // 2^25: held entries are at most 2^18.
  q.topk_magic = static_cast<uint32_t>(((1ull << 32) + p.topk - 1) / p.topk);
  void* args[] = {&q};
  return launch_pdl(held ? reinterpret_cast<const void*>(gsr_route_kernel<true>)
                         : reinterpret_cast<const void*>(gsr_route_kernel<false>),
                    dim3(ctas), threads, smem, ctas, args, stream);
}

cudaError_t launch_combine(const CombineParams& p, cudaStream_t stream) {
  const int64_t total = p.T * p.vecs;
  const bool two = total > 152 * 2048;   // more than the SMs' threads at once
  const int64_t blocks = (total + (two ? 511 : 255)) / (two ? 512 : 256);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(blocks, 1 << 30));
  CombineParams q = p;
  void* args[] = {&q};
  return launch_pdl(two ? reinterpret_cast<const void*>(gsr_combine_kernel<2>)
                        : reinterpret_cast<const void*>(gsr_combine_kernel<1>),
                    dim3(grid), 256, 0, 0, args, stream);
}

}  // namespace gsr
