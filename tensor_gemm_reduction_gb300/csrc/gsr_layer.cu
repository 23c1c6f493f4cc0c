// gsr_layer.cu -- a layer of experts for a few tokens in two kernels, for GB300.
//
//   Y[t] = base[t] + sum_j weight[t, j] * D[e] . (silu(G[e] . x_t) * (U[e] . x_t)),  e = ids[t, j]
//
// With few tokens the layer is a stream of the named experts' weights, each used by a
// row or a few, and what matters is that every SM streams all the time and that little
// else happens. So the weights go from memory straight into registers, where they are
// the A operand of mma.sync (16 weight rows x 16 k, bf16, fp32 sums): at the memory's
// rate an SM receives 11 weights per clock, far below what the tensor cores of either
// kind take, and without a shared-memory stage any 8 columns of any expert are a unit of
// work. A thread loads 16 bytes of a weight row (8 k), and the same k of a token: which k
// an MMA calls its first is the same for both operands.
//
// Every CTA sorts the T * topk entries by expert itself (in a stable order, so that sums
// do not depend on timing).
// - Up: a strip is 8 columns of one expert, gate and up rows as the two halves of A, so
//   that a thread ends with both of the same element. Strips are dealt evenly to the
//   CTAs; the warps of a CTA share its k. h = silu(g) * u is rounded to bf16 (as between
//   any two projections), one row per entry.
// - Down: a CTA owns 16 columns of Y for every expert, so nothing is summed between
//   CTAs: its warps share the named experts' k, in order, and keep weighted fp32 sums per
//   token in shared memory. Y is rounded once.
// Where there are fewer strips or columns than CTAs, a cluster shares the k further, and
// its first CTA adds the others' sums up.
//
// One token, 8 of 64 experts, N = 896, K = 7168: 308 MB of weights, 45 us at the copy
// bandwidth; 51 back to back (by themselves and cold, the kernels read 5.3 and 4.2 TB/s:
// a launch, the sort and the first data before each stream). 4 tokens (24 experts, 925 MB)
// 146 us and 8 (42, 1618 MB) 255, 0.93 and 0.94 of it.
//
// The second kernel starts while the first one ends (programmatic dependent launch),
// sorts its entries and prefetches its first weights into L2 before it waits for h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gsr_layer.h"
#include "gsr_routed.h"

namespace gsr {
namespace {

constexpr int kThreadsL = 256, kWarpsL = kThreadsL / 32;
constexpr int kResident = 3;      // CTAs per SM
constexpr int kMaxCluster = 8;
// Groups of 8 entries that share one read of the weights, at most. (8 of them leave no
// registers for their loads: one after the other, an expert of 51 entries took three times
// as long.)
constexpr int kGroupsAtOnce = 4;

// The entries by expert: expert[a] names entry[begin[a]] .. entry[begin[a + 1] - 1],
// ascending, of the a-th expert that has any.
struct Sorted {
  alignas(16) int id[kLayerEntries];      // of the sort, read four at a time; past every
  alignas(16) int first[kLayerEntries];   // expert: none
  int expert[kLayerEntries], begin[kLayerEntries + 1];
  int entry[kLayerEntries], token[kLayerEntries];
  float weight[kLayerEntries];
};

// Sorts the entries; their number of experts. By all threads, the first of which own an
// entry each and compare it with all.
__device__ int sort_entries(const LayerParams& p, Sorted& s) {
  static_assert(kLayerEntries <= kThreadsL && kLayerEntries % 4 == 0, "an entry per thread");
  constexpr int kNone = 1 << 30;
  const int i = static_cast<int>(threadIdx.x), n = p.T * p.topk;
  int mine = kNone;
  float weight = 0.f;
  if (i < n) {
    // Past L1: the second kernel reads them before it has waited for anything itself.
    const long long v = p.wide ? __ldcg(reinterpret_cast<const long long*>(p.ids) + i)
                               : __ldcg(reinterpret_cast<const int*>(p.ids) + i);
    weight = __ldcg(p.weights + i);
    if (v >= 0 && v < p.E) mine = static_cast<int>(v);
  }
  if (i < kLayerEntries) s.id[i] = mine;
  __syncthreads();
  const int quads = (n + 3) / 4;
  int place = 0;
  bool first = mine != kNone;
  if (first)
    for (int q = 0; q < quads; ++q) {
      const int4 o = reinterpret_cast<const int4*>(s.id)[q];
      const int id[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool before = id[j] == mine && 4 * q + j < i;
        place += id[j] < mine || before ? 1 : 0;
        first = first && !before;
      }
    }
  if (i < kLayerEntries) s.first[i] = first ? mine : kNone;
  const int kept = __syncthreads_count(mine != kNone);
  if (mine != kNone) {
    s.entry[place] = i;
    s.token[place] = i / p.topk;
    s.weight[place] = weight;
    if (first) {
      int a = 0;
      for (int q = 0; q < quads; ++q) {
        const int4 o = reinterpret_cast<const int4*>(s.first)[q];
        a += (o.x < mine) + (o.y < mine) + (o.z < mine) + (o.w < mine);
      }
      s.expert[a] = mine;
      s.begin[a] = place;
    }
  }
  const int active = __syncthreads_count(first);
  if (i == 0) s.begin[active] = kept;
  __syncthreads();
  return active;
}

__device__ __forceinline__ uint4 stream(const uint16_t* p, bool real) {
  return real ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint4 fetch(const uint16_t* p, bool real) {
  return real ? __ldcg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 k of 16 weight rows (lo: rows 0..7, hi: 8..15) times 8 entries.
__device__ __forceinline__ void multiply_32(float (&c)[4], const uint4& lo, const uint4& hi, const uint4& b) {
  mma(c, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
  mma(c, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
__device__ __forceinline__ float remote_float(const float* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// ------------------------------------------------------------ up

constexpr int kPartValues = 16;   // of a lane's fragments in a pass, at most
constexpr int kPartFloats = kWarpsL * kPartValues * 32;

// MT strips from column n0 on of expert e against NG groups of 8 entries: this CTA's
// share of k, the warps' sums added up, and h.
template <int MT, int NG>
__device__ void up_pass(const LayerParams& p, const Sorted& s, int e, int n0, int first, int count, float* part,
                        float* total, uint32_t rank, uint32_t ctas) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const size_t K = p.K;
  const uint16_t* gate = p.up + (static_cast<size_t>(e) * 2 * p.N + n0 + g) * K;
  const uint16_t* up = gate + static_cast<size_t>(p.N) * K;
  const uint16_t* x[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int at = 8 * i + g;
    x[i] = at < count ? p.x + static_cast<size_t>(s.token[first + at]) * K : nullptr;
  }
  float c[MT][NG][4] = {};
  for (int k0 = static_cast<int>(rank * kWarpsL + warp) * 64; k0 < p.K; k0 += static_cast<int>(ctas) * kWarpsL * 64) {
    const int k = k0 + 8 * t;
    uint4 lo[MT][2], hi[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        lo[m][j] = stream(gate + 8 * m * K + k + 32 * j, k + 32 * j < p.K);
        hi[m][j] = stream(up + 8 * m * K + k + 32 * j, k + 32 * j < p.K);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint4 b[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) b[i] = fetch(x[i] + k + 32 * j, x[i] && k + 32 * j < p.K);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NG; ++i) multiply_32(c[m][i], lo[m][j], hi[m][j], b[i]);
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[(warp * kPartValues + (m * NG + i) * 4 + v) * 32 + lane] = c[m][i][v];
  __syncthreads();
  if (ctas > 1) {
    for (int i = tid; i < MT * NG * 4 * 32; i += kThreadsL) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarpsL; ++w) sum += part[w * (kPartValues * 32) + i];
      total[i] = sum;
    }
    cluster_sync();
  }
  // Value v and v + 2 of a fragment are the gate and the up of one element.
  if (rank == 0)
    for (int i = tid; i < MT * NG * 2 * 32; i += kThreadsL) {
      const int l = i & 31, q = i >> 6, v = (i >> 5) & 1;
      const int at = (q * 4 + v) * 32 + l;
      float gv = 0.f, uv = 0.f;
      if (ctas == 1) {
#pragma unroll
        for (int w = 0; w < kWarpsL; ++w) {
          gv += part[w * (kPartValues * 32) + at];
          uv += part[w * (kPartValues * 32) + at + 64];
        }
      } else {
        for (uint32_t r = 0; r < ctas; ++r) {
          gv += remote_float(total + at, r);
          uv += remote_float(total + at + 64, r);
        }
      }
      const int entry = 8 * (q % NG) + 2 * (l & 3) + v, col = n0 + 8 * (q / NG) + (l >> 2);
      if (entry < count)
        p.h[static_cast<size_t>(s.entry[first + entry]) * p.N + col] =
            __bfloat16_as_ushort(__float2bfloat16(gv / (1.f + __expf(-gv)) * uv));
    }
  if (ctas > 1) cluster_sync();   // read by the first CTA before the next pass
  __syncthreads();
}

__global__ void __launch_bounds__(kThreadsL, kResident) gsr_layer_up_kernel(const __grid_constant__ LayerParams p) {
  __shared__ Sorted s;
  __shared__ float part[kPartFloats];
  __shared__ float total[kPartValues * 32];
  const uint32_t rank = cluster_rank(), ctas = cluster_ctas();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int active = sort_entries(p, s);
  const int strips = p.N / 8, G = static_cast<int>(gridDim.x / ctas), me = static_cast<int>(blockIdx.x / ctas);
  const long long all = static_cast<long long>(active) * strips;
  const int end = static_cast<int>(all * (me + 1) / G);
  for (int i = static_cast<int>(all * me / G); i < end;) {
    const int a = i / strips, strip = i - a * strips, e = s.expert[a];
    const int first = s.begin[a], count = s.begin[a + 1] - first;
    const bool two = count <= 16 && i + 1 < end && strip + 1 < strips;
    for (int from = 0; from < count; from += 8 * kGroupsAtOnce) {
      const int n = min(count - from, 8 * kGroupsAtOnce), at = first + from;
      if (two && n <= 8) up_pass<2, 1>(p, s, e, 8 * strip, at, n, part, total, rank, ctas);
      else if (two) up_pass<2, 2>(p, s, e, 8 * strip, at, n, part, total, rank, ctas);
      else if (n <= 8) up_pass<1, 1>(p, s, e, 8 * strip, at, n, part, total, rank, ctas);
      else if (n <= 16) up_pass<1, 2>(p, s, e, 8 * strip, at, n, part, total, rank, ctas);
      else up_pass<1, 4>(p, s, e, 8 * strip, at, n, part, total, rank, ctas);
    }
    i += two ? 2 : 1;
  }
}

// ------------------------------------------------------------ down

constexpr int kPieceK = 128;   // k of a warp's turn

// Pieces [from, to) of expert e's k, 16 columns of Y from o0 on, NG groups of 8 entries:
// weighted and added to this warp's sums (tokens x 16).
template <int NG>
__device__ void down_pass(const LayerParams& p, const Sorted& s, int e, int o0, int from, int to, int first, int count,
                          float* sums) {
  const int lane = static_cast<int>(threadIdx.x) & 31, g = lane >> 2, t = lane & 3;
  const size_t N = p.N;
  const bool in_lo = o0 + g < p.K, in_hi = o0 + 8 + g < p.K;
  const uint16_t* lo_row = p.down + (static_cast<size_t>(e) * p.K + o0 + g) * N;
  const uint16_t* hi_row = lo_row + 8 * N;
  const uint16_t* h[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int at = 8 * i + g;
    h[i] = at < count ? p.h + static_cast<size_t>(s.entry[first + at]) * N : nullptr;
  }
  float c[NG][4] = {};
  for (int piece = from; piece < to; ++piece) {
    constexpr int kAtOnce = NG <= 2 ? 4 : 2;   // steps of 32 k whose loads are in flight together
#pragma unroll 1
    for (int k = piece * kPieceK + 8 * t; k < (piece + 1) * kPieceK; k += 32 * kAtOnce) {
      uint4 lo[kAtOnce], hi[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const bool in = k + 32 * j < p.N;
        lo[j] = stream(lo_row + k + 32 * j, in && in_lo);
        hi[j] = stream(hi_row + k + 32 * j, in && in_hi);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const bool in = k + 32 * j < p.N;
        uint4 b[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) b[i] = fetch(h[i] + k + 32 * j, h[i] && in);
#pragma unroll
        for (int i = 0; i < NG; ++i) multiply_32(c[i], lo[j], hi[j], b[i]);
      }
    }
  }
  // Two entries of a group may be one token's: entry after entry.
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int turn = 0; turn < 4; ++turn) {
      if (t == turn) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int at = 8 * i + 2 * t + v;
          if (at < count) {
            const float w = s.weight[first + at];
            float* y = sums + s.token[first + at] * 16 + g;
            y[0] = fmaf(w, c[i][v], y[0]);
            y[8] = fmaf(w, c[i][v + 2], y[8]);
          }
        }
      }
      __syncwarp();
    }
}

__global__ void __launch_bounds__(kThreadsL, kResident) gsr_layer_down_kernel(const __grid_constant__ LayerParams p) {
  __shared__ Sorted s;
  __shared__ float sums[kWarpsL][kLayerTokens * 16];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_ctas();
  // The first kernel let this one start after it had waited for all before it, so the
  // call's inputs may be read; only h has to be waited for.
  const int active = sort_entries(p, s);
  const int pieces = (p.N + kPieceK - 1) / kPieceK, tiles = (p.K + 15) / 16;
  const int G = static_cast<int>(gridDim.x / ctas), workers = static_cast<int>(ctas) * kWarpsL;
  const int worker = static_cast<int>(rank) * kWarpsL + warp;
  const long long all = static_cast<long long>(active) * pieces;
  const int begin = static_cast<int>(all * worker / workers), end = static_cast<int>(all * (worker + 1) / workers);
  int tile = static_cast<int>(blockIdx.x / ctas);
  // The first weights of this warp: 16 rows x 256 bytes a piece, a line per lane.
  for (int i = begin; i < min(end, begin + 4); ++i) {
    const int a = i / pieces, row = tile * 16 + (lane >> 1), k = (i - a * pieces) * kPieceK + (lane & 1) * 64;
    if (row < p.K && k < p.N)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.down + (static_cast<size_t>(s.expert[a]) * p.K + row) * p.N + k));
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (; tile < tiles; tile += G) {
    __syncthreads();
    for (int i = lane; i < p.T * 16; i += 32) sums[warp][i] = 0.f;
    __syncwarp();
    const int o0 = tile * 16;
    for (int i = begin; i < end;) {
      const int a = i / pieces, from = i - a * pieces, to = min(pieces, from + end - i), e = s.expert[a];
      const int first = s.begin[a], count = s.begin[a + 1] - first;
      for (int f = 0; f < count; f += 8 * kGroupsAtOnce) {
        const int n = min(count - f, 8 * kGroupsAtOnce), at = first + f;
        if (n <= 8) down_pass<1>(p, s, e, o0, from, to, at, n, sums[warp]);
        else if (n <= 16) down_pass<2>(p, s, e, o0, from, to, at, n, sums[warp]);
        else down_pass<4>(p, s, e, o0, from, to, at, n, sums[warp]);
      }
      i += to - from;
    }
    __syncthreads();
    if (ctas > 1) {
      // Each element by the thread that read it: the CTA's sum in place of its first warp's.
      for (int i = tid; i < p.T * 16; i += kThreadsL) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kWarpsL; ++w) y += sums[w][i];
        sums[0][i] = y;
      }
      cluster_sync();
    }
    if (rank == 0)
      for (int i = tid; i < p.T * 16; i += kThreadsL) {
        const int col = o0 + (i & 15);
        if (col >= p.K) continue;
        const size_t at = static_cast<size_t>(i >> 4) * p.K + col;
        float y = p.base ? __uint_as_float(static_cast<uint32_t>(p.base[at]) << 16) : 0.f;
        if (ctas == 1) {
#pragma unroll
          for (int w = 0; w < kWarpsL; ++w) y += sums[w][i];
        } else {
          for (uint32_t r = 0; r < ctas; ++r) y += remote_float(&sums[0][i], r);
        }
        p.y[at] = __bfloat16_as_ushort(__float2bfloat16(y));
      }
    if (ctas > 1) cluster_sync();   // read by the first CTA before the next tile
  }
  // Not earlier: the next call's first kernel would be resident and wait beside this one,
  // which gains nothing (4 tokens of 8 entries 146 us, released early 147; 8 255 / 254).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A grid of clusters: as many CTAs per unit of work as fill the GPU, up to 8.
int cluster_of(int64_t units, int64_t slots) {
  int c = 1;
  while (c < kMaxCluster && units * c * 2 <= slots) c *= 2;
  return c;
}

cudaError_t launch_one(void (*kernel)(const LayerParams), const LayerParams& p, int64_t units, int sm_count,
                       cudaStream_t stream) {
  const int64_t slots = static_cast<int64_t>(sm_count) * kResident;
  const int c = cluster_of(units, slots);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(c * std::min<int64_t>(units, std::max<int64_t>(1, slots / c))), 1, 1);
  cfg.blockDim = dim3(kThreadsL, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_layer(const LayerParams& p, int sm_count, cudaStream_t stream) {
  const int64_t experts = std::min(p.E, p.T * p.topk);
  cudaError_t e = launch_one(gsr_layer_up_kernel, p, experts * (p.N / 8), sm_count, stream);
  if (e == cudaSuccess) e = launch_one(gsr_layer_down_kernel, p, (p.K + 15) / 16, sm_count, stream);
  return e;
}

}  // namespace gsr
