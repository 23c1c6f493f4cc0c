// gsr_lowrank.cu -- the low-rank rows of the adapters, for GB300 (sm_103a):
//
//   low[m, j] = scale[a] * sum_r X_r[m] . A_r[a][j],  a = adapter[m], j < rank
//
// in fp32, rounded once to bf16: they are an operand of the tensor cores'
// second product, which takes bf16 (the rounding adds about 2^-9 of the
// adapter's own part of Y, as rounding Y itself does).
//
// The rank is small (8 to 128), so the work is reading X and the adapters that
// some row has: a few hundred flops per row and byte at most, which warp-level
// mma.sync (m16n8k16) covers. One warp takes 16 rows and a share of k and reads
// both operands straight into the fragments, 16 bytes per lane: a lane's eight
// consecutive k are its two fragments' k (the sum does not mind the order, and X
// and A use the same), so no shared memory and no transpose is needed.
//
// 16 rows may have up to 16 adapters. Blocks take them in turn (blockIdx.y);
// each computes all 16 rows against its adapter and keeps those that have it.
// k is cut over the CTAs of a cluster (and, for few rows, over the warps of the
// CTA too); the fp32 shares meet in distributed shared memory and are added in
// a fixed order.
//
// Blocks past the rows write the adapter lists of the token tiles of the product
// that follows (ascending, without repeats).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gsr_routed.h"

namespace gsr {
namespace {

constexpr int kWarps = 8;
constexpr int kThreadsLow = 32 * kWarps;
constexpr int kMaxCluster = 8;       // CTAs that share the reduction, at most
constexpr int kUnit = 64;            // k per step of a warp (128 bytes of a row)

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16(const uint16_t* p, bool ok) {
  return ok ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ uint32_t cluster_shared_addr(const void* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(a), "r"(rank));
  return out;
}

__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();   // .aligned: whole warps arrive
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// Distinct adapters of a token tile's rows, ascending: a bit per adapter, then
// every thread lists the bits of its words behind those of the threads before.
__device__ void write_list(const LowRankParams& p, int tile, uint32_t* bits, int* sums) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int words = (p.L + 31) / 32, per = (words + kThreadsLow - 1) / kThreadsLow;
  const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
  const int row = tile * p.tile_tokens + tid;
  const int id = tid < p.tile_tokens && row < p.M ? p.adapter[row] : -1;
  for (int w = w0; w < w1; ++w) bits[w] = 0;
  __syncthreads();
  if (id >= 0 && id < p.L) atomicOr(&bits[id >> 5], 1u << (id & 31));
  __syncthreads();
  int mine = 0;
  for (int w = w0; w < w1; ++w) mine += __popc(bits[w]);
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int at = incl - mine, total = 0;
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) at += sums[i];
    total += sums[i];
  }
  int32_t* list = p.lists + static_cast<size_t>(tile) * kAdapterListStride;
  if (tid == 0) list[0] = total;
  for (int w = w0; w < w1; ++w)
    for (uint32_t b = bits[w]; b; b &= b - 1u) list[1 + at++] = 32 * w + __ffs(b) - 1;
}

// NT: 8-column tiles of a pass over the padded rank (128 columns take two passes of
// 64). SPLIT: the warps of a CTA share k (16 rows per CTA) or take 16 rows each
// (128 rows per CTA).
//
// The shares go through shared memory 32 columns at a time.
constexpr int kShareCols = 32;
constexpr int kSmemBytes = kWarps * 16 * kShareCols * 4;
static_assert(kSmemBytes >= kMaxAdapters / 8, "a bit per adapter");

template <int NT, bool SPLIT>
__global__ void __launch_bounds__(kThreadsLow, NT <= 4 ? 3 : 2) gsr_lowrank_kernel(const __grid_constant__ LowRankParams p) {
  extern __shared__ float share[];                 // [kWarps][16][columns of a turn]
  __shared__ int ids[kWarps], keeps[16 * kWarps];
  constexpr int kCols = 8 * NT < kShareCols ? 8 * NT : kShareCols, kTurnTiles = kCols / 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int z = static_cast<int>(blockIdx.z), ctas = static_cast<int>(gridDim.z);
  const int blocks = (p.M + (SPLIT ? 16 : 16 * kWarps) - 1) / (SPLIT ? 16 : 16 * kWarps);
  if (static_cast<int>(blockIdx.x) >= blocks) {   // whole clusters
    if (blockIdx.y == 0)
      for (int tile = (static_cast<int>(blockIdx.x) - blocks) * ctas + z; tile < p.m_tiles;
           tile += (static_cast<int>(gridDim.x) - blocks) * ctas) {
        write_list(p, tile, reinterpret_cast<uint32_t*>(share), ids);
        __syncthreads();
      }
    return;
  }

  const int row0 = static_cast<int>(blockIdx.x) * (SPLIT ? 16 : 16 * kWarps) + (SPLIT ? 0 : 16 * warp);
  const int group = lane >> 2, quad = lane & 3;
  // The distinct adapters of this warp's 16 rows: lane i (< 16) holds row i's;
  // `leaders` marks the first row of each.
  int id = lane < 16 && row0 + lane < p.M ? p.adapter[row0 + lane] : -1;
  if (id < 0 || id >= p.L) id = -1;
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  const uint32_t leaders =
      __ballot_sync(0xffffffffu, id >= 0 && (same & ((1u << lane) - 1u)) == 0);
  int most = __popc(leaders);
  if constexpr (!SPLIT) {
    // The CTA's warps go through their adapters together.
    if (lane == 0) ids[warp] = most;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) most = max(most, ids[i]);
  }
  const int units = p.unit_begin[p.R];
  const int parts = SPLIT ? ctas * kWarps : ctas;
  const int part = SPLIT ? z * kWarps + warp : z;
  const int u0 = static_cast<int>(static_cast<long long>(part) * units / parts);
  const int u1 = static_cast<int>(static_cast<long long>(part + 1) * units / parts);
  const bool row_a = row0 + group < p.M, row_b = row0 + group + 8 < p.M;

  for (int turn = static_cast<int>(blockIdx.y); turn < most; turn += static_cast<int>(gridDim.y)) {
    // The turn-th distinct adapter of this warp's rows (none: nothing to add).
    uint32_t left = leaders;
    for (int i = 0; i < turn; ++i) left &= left - 1u;
    const int a = left ? __shfl_sync(0xffffffffu, id, __ffs(left) - 1) : -1;
    if constexpr (!SPLIT) {
      if (lane < 16) keeps[warp * 16 + lane] = a >= 0 && id == a ? a : -1;   // rows to keep
    } else {
      if (warp == 0 && lane < 16) keeps[lane] = id == a ? a : -1;
    }
    for (int pass = 0; pass < p.rank_pad; pass += 8 * NT) {
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
      if (a >= 0) {
        for (int r = 0; r < p.R; ++r) {
          const int lo = max(u0, p.unit_begin[r]), hi = min(u1, p.unit_begin[r + 1]);
          if (lo >= hi) continue;
          const int64_t K = p.k[r];
          int k = (lo - p.unit_begin[r]) * kUnit + quad * 8;
          const int k_end = min(static_cast<int>(K), (hi - p.unit_begin[r]) * kUnit);
          const uint16_t* xa = p.x[r] + static_cast<int64_t>(row0 + group) * K;
          const uint16_t* xb = xa + 8 * K;
          const uint16_t* aa = p.a[r] + (static_cast<int64_t>(a) * p.rank + pass + group) * K;
#pragma unroll 2
          for (; k - quad * 8 < k_end; k += 32) {
            const bool in = k < k_end;
            const uint4 f = load16(xa + k, in && row_a);
            const uint4 s = load16(xb + k, in && row_b);
            uint4 b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
              b[n] = load16(aa + static_cast<int64_t>(8 * n) * K + k, in && pass + 8 * n + group < p.rank);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_16816(acc[n], f.x, s.x, f.y, s.y, b[n].x, b[n].y);
              mma_16816(acc[n], f.z, s.z, f.w, s.w, b[n].z, b[n].w);
            }
          }
        }
      }
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += kTurnTiles) {
        float* mine = share + warp * (16 * kCols);
#pragma unroll
        for (int n = 0; n < kTurnTiles; ++n) {
          const float* c = acc[n0 + n];
          *reinterpret_cast<float2*>(mine + group * kCols + 8 * n + 2 * quad) = make_float2(c[0], c[1]);
          *reinterpret_cast<float2*>(mine + (group + 8) * kCols + 8 * n + 2 * quad) = make_float2(c[2], c[3]);
        }
        cluster_sync_all();
        // Each CTA of the cluster adds up a share of the elements, in k order.
        constexpr int kElems = (SPLIT ? 16 : 16 * kWarps) * kCols;
        for (int e = z * kThreadsLow + tid; e < kElems; e += ctas * kThreadsLow) {
          const int row = e / kCols, col = pass + 8 * n0 + e - row * kCols;
          const int keep = keeps[row];
          if (keep < 0) continue;
          float sum = 0.f;
          for (int c = 0; c < ctas; ++c) {
            const uint32_t at = cluster_shared_addr(share, static_cast<uint32_t>(c));
#pragma unroll
            for (int w = 0; w < (SPLIT ? kWarps : 1); ++w) {
              float v;
              asm volatile("ld.shared::cluster.f32 %0, [%1];"
                           : "=f"(v)
                           : "r"(at + 4u * static_cast<uint32_t>(SPLIT ? w * kElems + e : e)));
              sum += v;
            }
          }
          const float s = p.scale ? __ldg(p.scale + keep) : 1.f;
          const int m = static_cast<int>(blockIdx.x) * (SPLIT ? 16 : 16 * kWarps) + row;
          p.low[static_cast<size_t>(m) * p.rank_pad + col] =
              __bfloat16_as_ushort(__float2bfloat16(sum * s));
        }
        cluster_sync_all();   // read by all before the next share is written
      }
    }
  }
}

template <int NT, bool SPLIT>
cudaError_t launch_nt(const LowRankParams& p, cudaStream_t stream) {
  const int rows = SPLIT ? 16 : 16 * kWarps, blocks = (p.M + rows - 1) / rows;
  // 16 rows have at most 16 adapters, each a turn of its own. k is cut among the
  // CTAs of a cluster until they are about four times the SMs (the reduction over a
  // cluster costs more).
  const int turns = SPLIT ? std::min(16, std::min(p.L, p.M)) : 1;
  int cluster = kMaxCluster;
  if (SPLIT)
    while (cluster > 1 && blocks * turns * cluster > 608) cluster /= 2;
  const int list_blocks = (std::min(p.m_tiles, 16) + cluster - 1) / cluster;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = cluster;
  cfg.gridDim = dim3(blocks + list_blocks, turns, cluster);
  cfg.blockDim = dim3(kThreadsLow, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gsr_lowrank_kernel<NT, SPLIT>, p);
}

}  // namespace

cudaError_t launch_low_rank(const LowRankParams& p, cudaStream_t stream) {
  const bool split = p.rows_per_cta == 16;
  switch (p.rank_pad) {
    case 16: return split ? launch_nt<2, true>(p, stream) : launch_nt<2, false>(p, stream);
    case 32: return split ? launch_nt<4, true>(p, stream) : launch_nt<4, false>(p, stream);
    default: return split ? launch_nt<8, true>(p, stream) : launch_nt<8, false>(p, stream);
  }
}

}  // namespace gsr
