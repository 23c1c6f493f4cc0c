// gsr_route.cu -- the route (a stable counting sort of expert ids) and the
// combine (the experts' rows weighted and added back per token), for GB300.
//
// Route. n ids, E groups: offsets[e] = ids below e that are in 0..E-1, position[i]
// = offsets[id] + earlier entries with the same id, source[position[i]] = i /
// topk. Every warp owns a run of entries, kept in registers, and a row of counts in
// shared memory; 32 entries at a time are matched by id, so counts need no atomics
// and the order is the entries'. The CTA's entries are ordered in shared memory
// first, so that source is written in runs (scattered, 262144 entries took 37 us,
// most of it 32 sectors per store).
//
// One launch of one CTA or of a cluster, whose CTAs read one another's group totals
// through distributed shared memory, is bound by its latencies (64 groups: 2048
// entries 4.8 us, 16384 6.0, 32768 7.0) until the work of 16 SMs takes longer
// (262144 entries of 256 groups: 21.5 us). Beyond: three launches over every SM. The
// first counts each CTA's ids; the second, one cluster, turns the counts into the
// sorted row at which each CTA's entries of each group begin; the third is the kernel
// above with those beginnings in place of its own. It starts beside the first two and
// waits for them only after it has matched and ordered its own entries. A CTA's
// counts and beginnings live in its own part of position, at least E entries, which
// that CTA alone reads back before it writes positions there: no workspace. 11.5 us
// for those 262144, three quarters of it the chain of launches.
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
constexpr int kHeld = 16;               // entries per thread, at most
constexpr int kHeldMax = kRouteThreads * kHeld;   // per CTA
constexpr int kScanCtas = 16;           // the cluster of the second launch
constexpr int kScanThreads = 512;       // of them each, at most
constexpr int kScanRows = 8;            // CTAs' counts that a thread keeps in registers
enum RouteForm : int { kAlone = 0, kCluster = 1, kChain = 2 };
constexpr int kRouteCluster = 16;       // CTAs of kCluster

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

// First entry of CTA c's part.
__device__ __forceinline__ int part_begin(const RouteParams& p, int c) {
  const long long first = 32ll * (static_cast<long long>(c) * p.units + min(c, p.longer));
  return first < p.n ? static_cast<int>(first) : p.n;
}

// Entries i, i + step, ... below end; -1 for an id outside 0..E-1. All loads at once:
// a branch on the ids' width between them would have each wait for the one before.
__device__ __forceinline__ void load_ids(const RouteParams& p, int i, int step, int end, int (&id)[kHeld]) {
  if (p.wide) {
    long long v[kHeld];
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      v[j] = i + step * j < end ? reinterpret_cast<const long long*>(p.ids)[i + step * j] : -1;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) id[j] = v[j] >= 0 && v[j] < p.E ? static_cast<int>(v[j]) : -1;
  } else {
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      id[j] = i + step * j < end ? reinterpret_cast<const int*>(p.ids)[i + step * j] : -1;
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (id[j] < 0 || id[j] >= p.E) id[j] = -1;
  }
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();   // .aligned: whole warps arrive
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// Many entries, first launch: how often each id occurs in the CTA's part.
__global__ void __launch_bounds__(kRouteThreads, 1) gsr_route_count_kernel(const RouteParams p) {
  __shared__ int counts[kMaxGroups];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x);
  const int first = part_begin(p, blockIdx.x), end = part_begin(p, blockIdx.x + 1);
  const int bits = 32 - __clz(p.E);
  int id[kHeld];
  load_ids(p, first + tid, threads, end, id);
  for (int e = tid; e < p.E; e += threads) counts[e] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    if (first + threads * j >= end) break;
    const uint32_t same = same_id(id[j], bits);
    if (id[j] >= 0 && (tid & 31) == __ffs(same) - 1) atomicAdd(counts + id[j], __popc(same));
  }
  __syncthreads();
  for (int e = tid; e < p.E; e += threads) p.position[first + e] = counts[e];
}

// Second launch: the counts c[part][e] become the sorted rows at which they begin. A
// CTA of the cluster has a run of groups; its threads are a grid of groups times runs
// of parts.
__global__ void __launch_bounds__(kScanThreads, 1) gsr_route_scan_kernel(const RouteParams p) {
  __shared__ int sums[kScanThreads], groups[kMaxGroups / kScanCtas];
  __shared__ int total;
  // The third launch may start: the first has begun, so every kernel before it is done.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x);
  const int cta = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
  const int own = (p.E + ctas - 1) / ctas, e0 = cta * own, width = min(own, max(p.E - e0, 0));
  const int shift = 32 - __clz(own - 1);   // 2^shift >= own
  const int columns = 1 << shift;
  const int x = tid & (columns - 1), y = tid >> shift;
  const int per = (p.parts + (threads >> shift) - 1) / (threads >> shift);
  const int r0 = min(y * per, p.parts), r1 = x < width ? min(r0 + per, p.parts) : r0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto load = [&](int r, int (&v)[kScanRows]) {
#pragma unroll
    for (int j = 0; j < kScanRows; ++j) v[j] = r + j < r1 ? p.position[part_begin(p, r + j) + e0 + x] : 0;
  };
  int head[kScanRows], sum = 0;
  load(r0, head);
#pragma unroll
  for (int j = 0; j < kScanRows; ++j) sum += head[j];
  for (int r = r0 + kScanRows; r < r1; r += kScanRows) {
    int v[kScanRows];
    load(r, v);
#pragma unroll
    for (int j = 0; j < kScanRows; ++j) sum += v[j];
  }
  // Inclusive sums down a group's runs of parts, then over the CTA's groups.
  sums[tid] = sum;
  __syncthreads();
  for (int d = columns; d < threads; d *= 2) {
    const int v = tid >= d ? sums[tid - d] : 0;
    __syncthreads();
    sums[tid] += v;
    __syncthreads();
  }
  const int of_group = sums[threads - columns + x];
  if (y == 0) groups[x] = of_group;
  __syncthreads();
  for (int d = 1; d < columns; d *= 2) {
    const int v = tid < columns && tid >= d ? groups[tid - d] : 0;
    __syncthreads();
    if (tid < columns) groups[tid] += v;
    __syncthreads();
  }
  if (tid == 0) total = groups[columns - 1];
  cluster_sync();
  int before = 0, all = 0;
#pragma unroll
  for (int c = 0; c < kScanCtas; ++c) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];"
                 : "=r"(v)
                 : "r"(remote(&total, static_cast<uint32_t>(c))));
    if (c < cta) before += v;
    all += v;
  }
  const int begin = before + groups[x] - of_group;
  if (y == 0 && x < width) p.offsets[e0 + x] = begin;
  if (cta == 0 && tid == 0) p.offsets[p.E] = all;
  int at = begin + sums[tid] - sum;
  for (int r = r0; r < r1; r += kScanRows) {
    if (r != r0) load(r, head);
#pragma unroll
    for (int j = 0; j < kScanRows; ++j) {
      if (r + j < r1) p.position[part_begin(p, r + j) + e0 + x] = at;
      at += head[j];
    }
  }
  cluster_sync();   // no CTA leaves while another may still read its total
}

// Everything by one CTA or one cluster; kChain: the third launch.
template <int FORM>
__global__ void __launch_bounds__(kRouteThreads, 1) gsr_route_kernel(const RouteParams p) {
  extern __shared__ int counts[];        // [warps][E], then the CTA's entries in order
  __shared__ int base[kMaxGroups];       // first sorted row of the CTA's entries of the group
  __shared__ int begin[kMaxGroups];      // its first place among the CTA's entries
  __shared__ int totals[kMaxGroups];     // kCluster: this CTA's entries of each group
  __shared__ int sums[kRouteWarps], all_sums[kRouteWarps];
  if constexpr (FORM != kChain) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int threads = static_cast<int>(blockDim.x), warps = threads >> 5;
  const int ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  const int first = part_begin(p, cta), end = part_begin(p, cta + 1);
  const int per = ((end - first + warps - 1) / warps + 31) & ~31;   // entries of a warp
  const int i0 = min(first + warp * per, end), i1 = min(i0 + per, end);
  const int bits = 32 - __clz(p.E);   // of id + 1, 0 .. E
  int* mine = counts + warp * p.E;
  int held[kHeld];   // the entry's id, then also its place among the warp's: id << 16 | place
  load_ids(p, i0 + lane, 32, i1, held);
  for (int e = lane; e < p.E; e += 32) mine[e] = 0;
  __syncwarp();

#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    if (i0 + 32 * j >= i1) break;
    // Counts the group's entries of the warp; the place of this one among them.
    const int id = held[j];
    const uint32_t same = same_id(id, bits);
    const int before = id >= 0 ? mine[id] : 0;
    __syncwarp();
    if (id >= 0 && lane == __ffs(same) - 1) mine[id] = before + __popc(same);
    __syncwarp();
    if (id >= 0) held[j] = id << 16 | (before + __popc(same & ((1u << lane) - 1u)));
  }
  __syncthreads();
  // Each thread a run of groups. Per group, each warp's count becomes the sum of
  // the warps before it; then the scan over the groups.
  const int eper = (p.E + threads - 1) / threads, e0 = min(tid * eper, p.E), e1 = min(e0 + eper, p.E);
  int all = 0;
  for (int e = e0; e < e1; ++e) {
    int at = 0;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const int c = counts[w * p.E + e];
      counts[w * p.E + e] = at;
      at += c;
    }
    begin[e] = all;   // of this thread's groups before e
    all += at;
    if constexpr (FORM == kCluster) totals[e] = at;
  }
  int incl = all;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int start = incl - all, kept = 0;   // of the CTA's entries
  for (int w = 0; w < warps; ++w) {
    if (w < warp) start += sums[w];
    kept += sums[w];
  }
  for (int e = e0; e < e1; ++e) begin[e] += start;
  __syncthreads();

  int* ordered = counts + warps * p.E;   // id << 16 | place among the CTA's entries
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    if (i0 + 32 * j >= i1) break;
    if (held[j] >= 0) {
      const int id = held[j] >> 16, place = (held[j] & 0xffff) + mine[id];
      held[j] = id << 16 | place;   // now among the CTA's
      ordered[begin[id] + place] = id << 16 | (i0 + 32 * j + lane - first);
    }
  }
  int dropped = kept;   // the first row of no entry
  if constexpr (FORM == kChain) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int e = tid; e < p.E; e += threads) base[e] = p.position[first + e];
    dropped = p.offsets[p.E];
  } else if constexpr (FORM == kCluster) {
    cluster_sync();
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
      int v[kRouteCluster], before = 0, of_group = 0;
#pragma unroll
      for (int c = 0; c < kRouteCluster; ++c)
        asm volatile("ld.shared::cluster.s32 %0, [%1];"
                     : "=r"(v[c])
                     : "r"(remote(totals + e, static_cast<uint32_t>(c))));
#pragma unroll
      for (int c = 0; c < kRouteCluster; ++c) {
        if (c < cta) before += v[c];
        of_group += v[c];
      }
      base[e] = before + sum;
      if (cta == 0) p.offsets[e] = sum;
      sum += of_group;
    }
    int through = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, through, d);
      if (lane >= d) through += v;
    }
    if (lane == 31) all_sums[warp] = through;
    __syncthreads();
    int from = through - sum;
    dropped = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) from += all_sums[w];
      dropped += all_sums[w];
    }
    for (int e = e0; e < e1; ++e) {
      base[e] += from;
      if (cta == 0) p.offsets[e] += from;   // written above by this thread
    }
    if (cta == 0 && tid == 0) p.offsets[p.E] = dropped;
  } else {
    for (int e = e0; e < e1; ++e) base[e] = p.offsets[e] = begin[e];
    if (tid == 0) p.offsets[p.E] = kept;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int i = i0 + 32 * j + lane;
    if (i0 + 32 * j >= i1) break;
    if (i < i1) p.position[i] = held[j] >= 0 ? base[held[j] >> 16] + (held[j] & 0xffff) : -1;
  }
  for (int j = tid; j < kept; j += threads) {
    const int id = ordered[j] >> 16;
    const uint32_t i = static_cast<uint32_t>(first + (ordered[j] & 0xffff));
    p.source[base[id] + j - begin[id]] =
        static_cast<int>(p.topk_magic ? __umulhi(i, p.topk_magic) : i / static_cast<uint32_t>(p.topk));
  }
  for (int i = dropped + cta * threads + tid; i < p.n; i += ctas * threads) p.source[i] = -1;
  if constexpr (FORM == kCluster) cluster_sync();   // no CTA leaves while another may still read its totals
}

__device__ __forceinline__ void add_row(float (&acc)[8], uint4 v, float w) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(w, __uint_as_float(u[i] << 16), acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, __uint_as_float(u[i] & 0xffff0000u), acc[2 * i + 1]);
  }
}

// A read that is not kept in L1 (each row of Z is read once). No load here is a
// non-coherent one: those are for memory that nothing writes while the kernel runs, and
// this one may be resident while its predecessor writes, and base may be Y.
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
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
      if (p.base && i < total) add_row(acc[q], reinterpret_cast<const uint4*>(p.base)[i], 1.f);
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
          const int at = j0 + j < p.topk && i0 + 256 * q < total ? pos[j] : -1;
          const bool live = at >= 0 && at < p.z_rows;
          // An absent entry adds nothing, whatever its weight is.
          w[q][j] = live ? wts[j] : 0.f;
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
  const int bytes = (kRouteWarps * kMaxGroups + kHeldMax) * 4;
  cudaError_t e = cudaFuncSetAttribute(gsr_route_kernel<kAlone>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(gsr_route_kernel<kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(gsr_route_kernel<kCluster>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(gsr_route_kernel<kChain>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(gsr_route_scan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return e;
}

cudaError_t launch_route(const RouteParams& p, cudaStream_t stream) {
  RouteParams q = p;
  const int64_t units = (static_cast<int64_t>(p.n) + 31) / 32;
  // One CTA, the cluster, or three launches, measured side by side in loops of calls
  // (us, 64 groups): 1024 entries 4.0 / 4.2 / -, 2048 4.8 / 4.4, 4096 7.2 / 4.6 / 10, 16384
  // - / 6.0 / 10.4, 32768 7.0 / 9.5, 65536 10.4 / 9.5, 131072 13.4 / 9.7, 262144 19.5 /
  // 11; with 1000 groups 2048 6.3 / 11, 4096 8.9 / 11.2, 32768 - / 13.2 / 11.
  const RouteForm form = p.n <= 2048 ? kAlone : p.n <= 49152 ? kCluster : kChain;
  // kChain: parts of some 2048 entries, on every SM twice, or, if those are too few, of a
  // CTA's capacity; never fewer entries than kMaxGroups.
  int64_t parts = form == kAlone ? 1 : kRouteCluster;
  if (form == kChain)
    parts = std::max<int64_t>(std::min<int64_t>(units / 64, 304), (units + kHeldMax / 32 - 1) / (kHeldMax / 32));
  q.parts = static_cast<int>(parts);
  q.units = static_cast<int>(units / parts);
  q.longer = static_cast<int>(units % parts);
  const int most = 32 * (q.units + (q.longer ? 1 : 0));      // entries of a part
  // Warps of 128 entries, where that does not take more than a CTA has; in the cluster a
  // thread per group at least (a thread with four of 1000 groups: 14.9 us for 1024
  // entries).
  const int least = std::max(form == kCluster ? p.E : 256, most / 4);
  const int threads = std::min(kRouteThreads, std::max(256, (least + 31) / 32 * 32));
  const size_t smem = (static_cast<size_t>(threads / 32) * p.E + most) * sizeof(int);
  // i / topk = (i * magic) >> 32 while i * (magic * topk - 2^32) < 2^32, that is for i < 2^25.
  q.topk_magic = p.topk > 1 && p.n <= 1 << 25
                     ? static_cast<uint32_t>(((1ull << 32) + p.topk - 1) / p.topk) : 0;
  void* args[] = {&q};
  const dim3 grid(static_cast<unsigned>(parts));
  auto launch = [&](auto kernel, dim3 ctas, int block, size_t bytes, int cluster) {
    return launch_pdl(reinterpret_cast<const void*>(kernel), ctas, block, bytes, cluster, args, stream);
  };
  if (form == kAlone) return launch(gsr_route_kernel<kAlone>, grid, threads, smem, 0);
  if (form == kCluster) return launch(gsr_route_kernel<kCluster>, grid, threads, smem, kRouteCluster);
  // The scan: threads for its groups times runs of parts, few for cheap barriers (262144
  // entries of 256 groups, 256 / 512 threads 11.5 / 12.6 us, of 1000 groups 17.6 / 16.2).
  cudaError_t e = launch(gsr_route_count_kernel, grid, threads, 0, 0);
  if (e == cudaSuccess) e = launch(gsr_route_scan_kernel, dim3(kScanCtas), p.E <= 512 ? 256 : kScanThreads, 0, kScanCtas);
  if (e == cudaSuccess) e = launch(gsr_route_kernel<kChain>, grid, threads, smem, 0);
  return e;
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
