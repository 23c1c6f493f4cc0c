// gsr_lowrank.cu -- the low-rank rows of the adapters, for GB300 (sm_103a):
//
//   low[m, j] = scale[a] * sum_r X_r[m] . A_r[a][j],  a = adapter[m], j < rank
//
// in fp32, rounded once to bf16: they are an operand of the tensor cores'
// second product, which takes bf16 (the rounding adds about 2^-9 of the
// adapter's own part of Y, as rounding Y itself does).
//
// The rank is small (8 to 128), so the work is reading X and the adapters that
// some row has: a few hundred flops per byte at most, which warp-level mma.sync
// (m16n8k16) covers. Both operands stream through a ring in shared memory, 16
// bytes per asynchronous copy, eight copies to a 128-byte line, swizzled for
// ldmatrix. (Loads straight into the fragments ask for 64 bytes of a line at a
// time: at 64 adapters and 128 rows the requests in flight held the kernel to
// 2.6 TB/s from memory.)
//
// With few rows a block takes an adapter and gathers the rows that have it, 16 at a
// time, and its warps share k; with many, a block takes 128 consecutive rows, 16
// per warp, and goes through their adapters. k is also cut over the CTAs of a
// cluster; the fp32 shares meet in distributed shared memory and are added in a
// fixed order. The adapter lists of the token tiles of the product that follows
// (ascending, without repeats) are written on the side.
// Measured: 128 rows over 64 adapters of rank 32, K = 7168, 10 us before the product (29
// MB of A: 4.3 at the copy bandwidth; the rest is the launch, first data and the
// cluster's sum); 4096 rows over 8 of rank 64, 20 us. With many rows a block's time is its
// distinct adapters' times a pass over k: runs of rows are what that kernel is for. 64
// adapters of rank 32 mixed row by row, the whole call: 132 us for 1024 rows (the kernel
// for few), 910 for 1025, 969 for 2048 and 1660 for 4096; in runs of 200, 8 adapters, 113
// for 1024 rows, 90 for 1025, 146 and 263.
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

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void load_matrices(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 16 bytes to shared memory, or 16 zeros; asynchronous.
__device__ __forceinline__ void copy_16(uint32_t dst, const uint16_t* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ uint32_t cluster_shared_addr(const void* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(a), "r"(rank));
  return out;
}

// For reads of the cluster's shared memory that are done (their values used): no
// release, which would wait for global stores.
__device__ __forceinline__ void cluster_sync_reads() {
  __syncwarp();
  asm volatile(
      "barrier.cluster.arrive.relaxed.aligned;\n\t"
      "barrier.cluster.wait.aligned;" ::
          : "memory");
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

// The shards' table in shared memory, filled before the kernel waits for its
// predecessor: the first reads of the parameters come from memory, and one by one,
// where they are used, took longer than the products.
struct Shards {
  const uint16_t *x[kMaxShards], *a[kMaxShards];
  int k[kMaxShards];
  __device__ __forceinline__ void fill(const LowRankParams& p) {
    const int r = static_cast<int>(threadIdx.x);
    if (r < kMaxShards) {
      x[r] = p.x[r];
      a[r] = p.a[r];
      k[r] = r < p.R ? static_cast<int>(p.k[r]) : 0;
    }
  }
};

// A block's stream: ROWS rows (their indices in `rows`, < 0: zeros) against columns
// pass .. pass + 8 NT of adapter a, over this CTA's share of k, in stages of KSTEP.
// 128 rows: warp w has rows 16 w ..; 16 rows: the warps share a stage's k.
template <int ROWS, int NT>
struct Stream {
  static constexpr int KSTEP = ROWS == 16 ? 128 : 64, kPitch = 2 * KSTEP, kChunks = KSTEP / 8;
  static constexpr int kLines = ROWS + 8 * NT, kStage = kLines * kPitch;
  static constexpr int S = ROWS == 16 ? (NT == 8 ? 5 : 6) : 3;
  static constexpr int kBytes = S * kStage;

  static __device__ __forceinline__ void run(const LowRankParams& p, const Shards& sh, uint32_t ring,
                                             const int* rows, int a, int pass, int z, int ctas,
                                             float (&acc)[NT][4]) {
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    int total = 0;
    for (int r = 0; r < p.R; ++r) total += (sh.k[r] + KSTEP - 1) / KSTEP;
    const int first = static_cast<int>(static_cast<long long>(z) * total / ctas);
    const int count = static_cast<int>(static_cast<long long>(z + 1) * total / ctas) - first;
    int shard = 0, k0 = 0;   // of the next stage to copy
    for (int left = first; left > 0;) {
      const int here = (sh.k[shard] - k0 + KSTEP - 1) / KSTEP, n = min(left, here);
      left -= n;
      k0 += n * KSTEP;
      if (n == here) {
        ++shard;
        k0 = 0;
      }
    }
    const int chunk = tid % kChunks;
    auto copy = [&](int slot) {
      const int K = sh.k[shard], k = k0 + 8 * chunk;
      const uint16_t* x = sh.x[shard];
      const uint16_t* aa = sh.a[shard] + (static_cast<int64_t>(a) * p.rank + pass) * K;
      const bool in = k < K;
      const uint32_t base = ring + slot * kStage;
#pragma unroll
      for (int line = tid / kChunks; line < kLines; line += kThreadsLow / kChunks) {
        const int j = line - ROWS, row = line < ROWS ? rows[line] : j;
        const bool real = in && (line < ROWS ? row >= 0 : pass + j < p.rank);
        const uint16_t* src = (line < ROWS ? x : aa) + (real ? static_cast<int64_t>(row) * K + k : 0);
        copy_16(base + line * kPitch + ((chunk ^ (line & 7)) << 4), src, real);
      }
      k0 += KSTEP;
      if (k0 >= K) {
        ++shard;
        k0 = 0;
      }
    };
    __syncthreads();   // rows[] written, the ring no longer read
    int copied = 0;
#pragma unroll
    for (; copied < S - 1; ++copied) {
      if (copied < count) copy(copied);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    const int x_row = (ROWS == 16 ? 0 : 16 * warp) + (lane & 15), x_chunk = lane >> 4;
    const int a_line = ROWS + (lane & 7) + ((lane >> 4) << 3), a_chunk = (lane >> 3) & 1;
    int slot = 0, next = S - 1;
    for (int i = 0; i < count; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
      __syncthreads();   // stage i has landed, stage i - 1 is read
      if (copied < count) copy(next);
      ++copied;
      asm volatile("cp.async.commit_group;" ::: "memory");
      const uint32_t base = ring + slot * kStage;
#pragma unroll
      for (int q = 0; q < (ROWS == 16 ? 1 : KSTEP / 16); ++q) {
        const int ks = ROWS == 16 ? warp : q;
        uint32_t x[4];
        load_matrices(base + x_row * kPitch + (((2 * ks + x_chunk) ^ (x_row & 7)) << 4), x);
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t w[4];
          const int line = a_line + 8 * n;
          load_matrices(base + line * kPitch + (((2 * ks + a_chunk) ^ (line & 7)) << 4), w);
          mma_16816(acc[n], x[0], x[1], x[2], x[3], w[0], w[1]);
          mma_16816(acc[n + 1], x[0], x[1], x[2], x[3], w[2], w[3]);
        }
      }
      slot = slot + 1 == S ? 0 : slot + 1;
      next = next + 1 == S ? 0 : next + 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();   // the ring may hold the shares now
  }
};

// The shares use the ring's memory, 32 columns at a time; the adapter lists too, a
// bit per adapter.
constexpr int kShareCols = 32;
static_assert(Stream<16, 2>::kBytes >= kWarps * 16 * kShareCols * 4, "shares");
static_assert(Stream<16, 2>::kBytes >= kMaxAdapters / 8, "a bit per adapter");

// Adds up the shares share[warp][16][columns] in k order, over the warps of the CTA
// (KW of them share a row group) and then over the cluster, and writes them,
// scaled, to columns `first` .. of the rows at[] (< 0: none) that have the adapters
// keeps[].
template <int COLS, int KW>
__device__ __forceinline__ void write_rows(const LowRankParams& p, float* share, const int* at,
                                           const int* keeps, int first, int z, int ctas) {
  constexpr int kElems = 16 * (kWarps / KW) * COLS;
  const int tid = static_cast<int>(threadIdx.x);
  if constexpr (KW > 1) {
    __syncthreads();
    for (int e = tid; e < kElems; e += kThreadsLow) {
      float sum = share[e];
#pragma unroll
      for (int w = 1; w < KW; ++w) sum += share[w * kElems + e];
      share[e] = sum;   // read by this thread alone
    }
  }
  cluster_sync_all();
  for (int e = z * kThreadsLow + tid; e < kElems; e += ctas * kThreadsLow) {
    const int row = e / COLS;
    if (at[row] < 0) continue;
    float v[kMaxCluster];
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      v[c] = 0.f;
      if (c < ctas)
        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                     : "=f"(v[c])
                     : "r"(cluster_shared_addr(share + e, static_cast<uint32_t>(c))));
    }
    float sum = v[0];
#pragma unroll
    for (int c = 1; c < kMaxCluster; ++c) sum += v[c];
    const float s = p.scale ? p.scale[keeps[row]] : 1.f;
    p.low[static_cast<size_t>(at[row]) * p.rank_pad + first + e - row * COLS] =
        __bfloat16_as_ushort(__float2bfloat16(sum * s));
  }
  cluster_sync_reads();   // read by all before the next share is written
}

// The product that follows may start its blocks where these leave room, and its
// base product with them: everything before this kernel has completed by now.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int NT>
__device__ __forceinline__ void put_share(float* share, const float (*acc)[4], int cols) {
  const int lane = static_cast<int>(threadIdx.x) & 31, group = lane >> 2, quad = lane & 3;
  float* mine = share + (static_cast<int>(threadIdx.x) >> 5) * (16 * cols);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    *reinterpret_cast<float2*>(mine + group * cols + 8 * n + 2 * quad) = make_float2(acc[n][0], acc[n][1]);
    *reinterpret_cast<float2*>(mine + (group + 8) * cols + 8 * n + 2 * quad) = make_float2(acc[n][2], acc[n][3]);
  }
}

// Few rows (at most kFewRows): block (x, y) takes the y-th adapter that a row has
// and, of its rows, every gridDim.x-th group of 16, so that an adapter is read
// about once however its rows are spread. k is cut over the cluster and the warps.
// NT: 8-column tiles of a pass over the padded rank.
constexpr int kFewRows = 1024;

template <int NT>
__global__ void __launch_bounds__(kThreadsLow, 2) gsr_lowrank_few_kernel(const __grid_constant__ LowRankParams p) {
  extern __shared__ float share[];                 // the ring; [kWarps][16][columns of a turn]
  __shared__ int sums[kWarps], members[kFewRows], group_rows[16], group_ids[16], found;
  __shared__ Shards shards;
  constexpr int kCols = 8 * NT < kShareCols ? 8 * NT : kShareCols, kTurnTiles = kCols / 8;
  shards.fill(p);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  let_next_start();
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int z = static_cast<int>(blockIdx.z), ctas = static_cast<int>(gridDim.z);
  const int nth = static_cast<int>(blockIdx.y);

  // The list of token tile `tile`, by one block of each column of the grid; the
  // whole call's distinct adapters likewise (a bit per adapter).
  uint32_t* bits = reinterpret_cast<uint32_t*>(share);
  if (nth == 0 && z == 0)
    for (int tile = static_cast<int>(blockIdx.x); tile < p.m_tiles; tile += static_cast<int>(gridDim.x)) {
      write_list(p, tile, bits, sums);
      __syncthreads();
    }
  constexpr int kPer = kFewRows / kThreadsLow;
  int id[kPer];
  const int words = (p.L + 31) / 32, per = (words + kThreadsLow - 1) / kThreadsLow;
  const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
  for (int w = w0; w < w1; ++w) bits[w] = 0;
  if (tid == 0) found = -1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    // Rows in order over warps, then lanes.
    const int m = (warp * kPer + i) * 32 + lane;
    id[i] = m < p.M ? p.adapter[m] : -1;
    if (id[i] < 0 || id[i] >= p.L) id[i] = -1;
    if (id[i] >= 0) atomicOr(&bits[id[i] >> 5], 1u << (id[i] & 31));
  }
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
  int before = incl - mine;
  for (int i = 0; i < warp; ++i) before += sums[i];
  if (nth >= before && nth < before + mine) {
    int left = nth - before, w = w0;
    while (__popc(bits[w]) <= left) left -= __popc(bits[w++]);
    uint32_t b = bits[w];
    for (; left > 0; --left) b &= b - 1u;
    found = 32 * w + __ffs(b) - 1;
  }
  __syncthreads();
  const int a = found;
  if (a < 0) return;   // fewer adapters (the whole cluster)
  // Its rows, in order.
  uint32_t has[kPer];
  int count = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    has[i] = __ballot_sync(0xffffffffu, id[i] == a);
    count += __popc(has[i]);
  }
  __syncthreads();
  if (lane == 0) sums[warp] = count;
  __syncthreads();
  int at = 0, total = 0;
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) at += sums[i];
    total += sums[i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (id[i] == a) members[at + __popc(has[i] & ((1u << lane) - 1u))] = (warp * kPer + i) * 32 + lane;
    at += __popc(has[i]);
  }
  __syncthreads();

  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(share));
  for (int g = 16 * static_cast<int>(blockIdx.x); g < total; g += 16 * static_cast<int>(gridDim.x)) {
    if (tid < 16) {
      group_rows[tid] = g + tid < total ? members[g + tid] : -1;
      group_ids[tid] = a;
    }
    for (int pass = 0; pass < p.rank_pad; pass += 8 * NT) {
      float acc[NT][4] = {};
      Stream<16, NT>::run(p, shards, ring, group_rows, a, pass, z, ctas, acc);
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += kTurnTiles) {
        put_share<kTurnTiles>(share, acc + n0, kCols);
        write_rows<kCols, kWarps>(p, share, group_rows, group_ids, pass + 8 * n0, z, ctas);
      }
    }
  }
}

// Many rows: block x takes 128 rows, 16 per warp, and their adapters one after the
// other, ascending. A row has one adapter, so the turns' sums share one buffer, and
// the cluster adds up once (4096 rows, 8 adapters, alone: 43 us adding up every turn,
// 37 so).
template <int NT>
constexpr int many_bytes() { return Stream<128, NT>::kBytes + kWarps * 16 * 8 * NT * 4; }

template <int NT>
__global__ void __launch_bounds__(kThreadsLow, 2) gsr_lowrank_kernel(const __grid_constant__ LowRankParams p) {
  extern __shared__ float ring_mem[];              // the ring, then sums [128][8 NT]
  __shared__ int sums[kWarps], keeps[16 * kWarps], rows[16 * kWarps], at[16 * kWarps];
  __shared__ Shards shards;
  constexpr int kCols = 8 * NT;
  shards.fill(p);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  let_next_start();
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int z = static_cast<int>(blockIdx.z), ctas = static_cast<int>(gridDim.z);
  const int blocks = (p.M + 16 * kWarps - 1) / (16 * kWarps);
  if (static_cast<int>(blockIdx.x) >= blocks) {   // whole clusters: the token tiles' lists
    for (int tile = (static_cast<int>(blockIdx.x) - blocks) * ctas + z; tile < p.m_tiles;
         tile += (static_cast<int>(gridDim.x) - blocks) * ctas) {
      write_list(p, tile, reinterpret_cast<uint32_t*>(ring_mem), sums);
      __syncthreads();
    }
    return;
  }
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_mem));
  float* share = ring_mem + Stream<128, NT>::kBytes / 4;
  const int m = static_cast<int>(blockIdx.x) * 16 * kWarps + tid;   // thread i < 128 has row i
  int id = tid < 16 * kWarps && m < p.M ? p.adapter[m] : -1;
  if (id < 0 || id >= p.L) id = -1;
  if (tid < 16 * kWarps) {
    at[tid] = id >= 0 ? m : -1;
    keeps[tid] = id;
  }
  for (int pass = 0; pass < p.rank_pad; pass += kCols) {
    for (int last = -1;;) {
      // The smallest adapter above the last one.
      const int mine = id > last ? id : INT32_MAX;
      const int least = __reduce_min_sync(0xffffffffu, mine);
      __syncthreads();   // the last turn's reads
      if (lane == 0) sums[warp] = least;
      __syncthreads();
      int a = INT32_MAX;
      for (int i = 0; i < kWarps; ++i) a = min(a, sums[i]);
      if (a == INT32_MAX) break;
      last = a;
      if (tid < 16 * kWarps) rows[tid] = id == a ? m : -1;   // the others are not read (zeros)
      float acc[NT][4] = {};
      Stream<128, NT>::run(p, shards, ring, rows, a, pass, z, ctas, acc);
      // Only the adapter's own rows: zeros times an infinite weight are NaN.
      const int group = lane >> 2, quad = lane & 3, r0 = 16 * warp + group;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (rows[r0 + 8 * h] >= 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            *reinterpret_cast<float2*>(share + (r0 + 8 * h) * kCols + 8 * n + 2 * quad) =
                make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
        }
    }
    write_rows<kCols, 1>(p, share, at, keeps, pass, z, ctas);
  }
}

template <class K>
cudaError_t launch_clusters(K kernel, const LowRankParams& p, dim3 grid, int smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = grid.z;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreadsLow, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int NT>
cudaError_t launch_nt(const LowRankParams& p, cudaStream_t stream) {
  if (p.M <= kFewRows) {
    // About two CTAs per SM: k cut over up to eight of a cluster, then, where there
    // are few adapters, their rows over blocks. (Blocks that find no adapter or rows
    // leave at once, but the others are not spread over the SMs anew.)
    const int adapters = std::min(p.L, p.M);
    int cluster = kMaxCluster;
    while (cluster > 1 && adapters * cluster > 304) cluster /= 2;
    const int groups = std::min((p.M + 15) / 16, std::max(1, 304 / (adapters * cluster)));
    return launch_clusters(gsr_lowrank_few_kernel<NT>, p, dim3(groups, adapters, cluster),
                           Stream<16, NT>::kBytes, stream);
  }
  const int blocks = (p.M + 16 * kWarps - 1) / (16 * kWarps);
  const int list_blocks = (std::min(p.m_tiles, 16) + kMaxCluster - 1) / kMaxCluster;
  return launch_clusters(gsr_lowrank_kernel<NT>, p, dim3(blocks + list_blocks, 1, kMaxCluster),
                         many_bytes<NT>(), stream);
}

}  // namespace

template <int NT>
cudaError_t set_limits() {
  cudaError_t e = cudaFuncSetAttribute(gsr_lowrank_few_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       Stream<16, NT>::kBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(gsr_lowrank_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              many_bytes<NT>());
}

cudaError_t prepare_lowrank_kernels() {
  cudaError_t e = set_limits<2>();
  if (e == cudaSuccess) e = set_limits<4>();
  if (e == cudaSuccess) e = set_limits<8>();
  return e;
}

cudaError_t launch_low_rank(const LowRankParams& p, cudaStream_t stream) {
  switch (p.rank_pad) {
    case 16: return launch_nt<2>(p, stream);
    case 32: return launch_nt<4>(p, stream);
    default: return launch_nt<8>(p, stream);
  }
}

}  // namespace gsr
