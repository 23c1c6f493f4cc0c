// gsr_fp8.cu -- products of 8-bit operands with scales per block of 128, for GB300
// (sm_103a): the K-sharded sum (AR) and the product of gathered row shards (AG).
//
//   Y[m, n] = sum_b sx[b, m] * sw[n / 128, b] * sum_{k in b} x[m, k] * w[n, k]
//
// over the blocks b of 128 columns of every K-shard, x and w in e4m3. The inner sums
// run on the tensor cores (tcgen05.mma kind::f8f6f4, fp32), a block in a fresh
// accumulator; the epilogue warps multiply each block's sums by its scales and add
// them up in fp32 registers: the scales are fp32 numbers, so they cannot go into
// the tensor cores' own block scales (powers of two).
//
// So that a scale is one number per thread, the tokens are the MMA's M: a TMEM lane is
// a token row, and a warp's columns lie in two blocks of weight rows at most. A CTA
// pair owns a tile of tokens x tile_n weight rows over the whole of K:
// - kFp8Wide: 256 tokens (128 per CTA) x up to 256. A CTA's 128 x 256 sums are 128
//   registers of each of its 256 epilogue threads. A ring stage is a k-block for tiles of
//   192 and 256 weight rows, two for those of up to 128, and the TMEM holds two stages'
//   accumulators: while the tensor cores fill one stage's, the other's are read.
// - kFp8Narrow: up to 128 tokens x up to 128, a stream of weights. The pair MMA of 128
//   rows keeps a CTA's 64 rows twice over in TMEM: lanes 64..127 hold the second half
//   of the columns. A stage is four k-blocks, each with an accumulator of its own, so
//   that the hand-over between the roles comes once per stage.
//
// A CTA's tokens are `boxes` boxes of box_rows rows, each from one row shard, so that
// short row shards share a tile.
//
// What bounds it. Wide: a k-block's MMAs take 512 cycles (256 x 256), but the epilogue's chain
// of a k-block, two waits, four reads of TMEM at about 100 cycles each and the sums, some
// 800; without it the copies would take 700 (L2). M = 4096, N = K = 7168 150 us, 2.8 PFLOP/s
// (61 % of the time the tensor cores are busy, as ncu counts them at M = 2048); M = 16384 586
// us. (Of the instances this one alone spills: 12 bytes stored and 48 loaded a thread.)
// Narrow: W from memory, 51 MB at N = K = 7168 in 7.6 us, and the launch, the first data and
// the way out, about 5.5: M = 1 13.3 us, M = 128 14.5.
// Measured and dropped: the next k-block's wait and first read before the last sums of this
// one (no gain with 192 columns, spills with 256); the MMAs issued by one thread for the
// whole loop (M = 1 13 -> 19 us); a ring of four stages of 256 x 256 (M = 4096 258 us,
// against 165 with five); weight tiles of 96 for one tile of up to 256 tokens (M = 256 20.2
// us, with 128 19.4); the producer's start before the TMEM allocation and the cluster's
// barrier (M = 512 27 -> 31 us); sixteen epilogue warps of 64 columns (M = 4096 154 us, against
// 151); K shared by the two pairs of a cluster (2.4 us more per call: M = 64, N = 1024, K = 2048
// 5.6 -> 7.6 us, K = 7168, N = 512 10.4 -> 9.4).
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer (the pair's leader), warp 2 copies the
// scales ahead into a ring of their own and warp 3 multiplies them (loaded by the epilogue
// itself, even four k-blocks ahead, they cost it 0.4 us a k-block), warps 4 and up
// epilogue. Every wait is bounded like the other kernels'.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gsr_device.cuh"
#include "gsr_fp8.h"

namespace gsr {
namespace {

template <int FORM_, int TILE_N_>
struct Cfg {
  static constexpr int FORM = FORM_, TILE_N = TILE_N_, KZ = fp8_kblocks(FORM, TILE_N);
  static constexpr bool WIDE = FORM == kFp8Wide;
  static constexpr int kRows = fp8_cta_rows(FORM);          // token rows of a CTA
  static constexpr int kEpi = WIDE ? 256 : 128;
  static constexpr int kThreads = 128 + kEpi;
  // Registers: three warpgroups of kFp8Wide leave 168 a thread, too few for an epilogue
  // thread's 128 sums, so the first one gives some of its own up (504 = 72 + 2 x 216).
  static constexpr int kLaunchRegs = 168, kRoleRegs = 72, kEpiRegs = 216;
  static_assert(kRoleRegs + 2 * kEpiRegs <= 3 * kLaunchRegs, "more registers than the launch's");
  static constexpr int kCols = TILE_N / 2;                  // columns of an epilogue warp
  // Blocks of weight rows that a tile meets (its first row is a multiple of TILE_N) and
  // that a warp's columns do.
  static constexpr int kBlocks = kScaleBlock % TILE_N == 0 ? 1 : 2;
  static constexpr bool kOneBlock = kBlocks == 1 || kCols == kScaleBlock;
  // A k-block's sums are read from TMEM in units, the next one while one is added up: as
  // wide ones as there are registers for (a read takes about 100 cycles whatever it reads).
  static constexpr int kUnit = kCols <= 64 ? kCols : kCols == 96 ? 48 : 32, kPerBlock = kCols / kUnit, kUnits = KZ * kPerBlock;
  // TMEM columns of a k-block's sums, and accumulators (of KZ k-blocks).
  static constexpr uint32_t kAccCols = 256 / KZ;
  static constexpr uint32_t kAccs = 2;
  static constexpr uint32_t kTmemCols = kAccs * KZ * kAccCols;
  static_assert(kTmemCols == 512, "all of the TMEM");
  // full[16], empty[16], tmem_full[2], tmem_empty[2], drain; the products of the scales: full,
  // empty; the scales: full, empty
  static constexpr uint32_t kScaleBarsOff = (2 * kFp8MaxRing + 2 * kAccs + 1) * 8;
  static constexpr uint32_t kRawBarsOff = kScaleBarsOff + 2 * kFp8ScaleRing * 8;
  static constexpr uint32_t kBars = kRawBarsOff + 2 * kFp8RawRing * 8;
  static constexpr uint32_t kStagingOff = fp8_ring_bytes(FORM, TILE_N);
  static constexpr uint32_t kBarsOff = kStagingOff + fp8_staging_bytes(FORM, TILE_N);
  static constexpr uint32_t kMiscOff = kBarsOff + kBars;
  static constexpr uint32_t kTableOff = (kMiscOff + 16 + 15) / 16 * 16;
};

// The products of the scales of four k-blocks, for each of the CTA's token rows and each
// block of weight rows of the tile.
template <class C>
struct GroupScales {
  float4 s[C::kBlocks][C::kRows];
};

template <class C>
struct RawScales {
  float x[4][C::kRows], w[4][2];
};

// The shards as the roles read them (a cold parameter is a memory access).
struct Table {
  const float *sx[kMaxShards], *sw[kMaxShards];
  int64_t row_begin[kMaxShards];
  int kb[kMaxShards], rows[kMaxShards], box_begin[kMaxShards + 1];
};

template <class C>
struct Shared {
  Table table;
  GroupScales<C> scales[kFp8ScaleRing];
  RawScales<C> raw[kFp8RawRing];
};
template <class C>
constexpr uint32_t smem_bytes() { return 1024 + C::kTableOff + sizeof(Shared<C>); }
static_assert(smem_bytes<Cfg<kFp8Wide, 256>>() <= kSmallSmemLimit, "shared memory");
static_assert(smem_bytes<Cfg<kFp8Narrow, 128>>() <= kSmallSmemLimit, "shared memory");

// The four MMAs of one k-block of 128 e4m3 columns (32 columns, 32 bytes, each), into a
// fresh accumulator.
__device__ __forceinline__ void mma4_e4m3_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t"
      "setp.ne.b32 p, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %5, %9, p;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %2, %6, %9, t;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %3, %7, %9, t;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %4, %8, %9, t;\n\t}" ::"r"(d),
      "l"(a), "l"(a + 2), "l"(a + 4), "l"(a + 6), "l"(b), "l"(b + 2), "l"(b + 4), "l"(b + 6), "r"(idesc)
      : "memory");
}

// Instruction descriptor for kind::f8f6f4: D fp32 (bits 4-5 = 1), A and B e4m3 (7-9 and
// 10-12 = 0), both K-major, N >> 3 in 17-22, M >> 4 in 24-28.
__device__ __forceinline__ uint32_t make_idesc_e4m3(uint32_t mma_m, uint32_t mma_n) {
  return (1u << 4) | ((mma_n >> 3) << 17) | ((mma_m >> 4) << 24);
}

// The commits of mma_commit_pair by the one thread that issues.
__device__ __forceinline__ void commit_pair_here(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}

// Token tile and first weight row of tile `id`: group_m token tiles run before the
// next weight tile, so that concurrent pairs share both operands in L2.
__device__ __forceinline__ void place(const Fp8Params& p, int id, int& m, int& n0) {
  const int span = p.group_m * p.n_tiles;
  const int sup = id / span, in = id - sup * span;
  const int gm = min(p.m_tiles - sup * p.group_m, p.group_m);
  const int col = in / gm;
  m = sup * p.group_m + in - col * gm;
  n0 = col * p.tile_n;
}

// Row shard and first row in it of box `b` of the call (past the last one: a row that
// no shard has).
__device__ __forceinline__ void find_box(const Fp8Params& p, const int* box_begin, int b, int& shard, int& row) {
  shard = p.pad_shard;
  row = 1 << 30;
  for (int r = 0; r < p.m_shards; ++r)
    if (b >= box_begin[r] && b < box_begin[r + 1]) {
      shard = r;
      row = (b - box_begin[r]) * p.box_rows;
    }
}

template <class C>
__device__ void produce(const Fp8Params& p, const Table& table, uint32_t base, uint32_t rank, const Ctl& ctl) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t full0 = base + C::kBarsOff, empty0 = full0 + 8 * kFp8MaxRing;
  const uint32_t lead0 = map_shared_to_rank(full0, 0);
  const uint64_t pol_w = make_l2_policy(p.policy_w), pol_x = make_l2_policy(p.policy_x);
  constexpr uint32_t w_bytes = C::TILE_N / 2 * kScaleBlock;
  const uint32_t box_bytes = p.box_rows * kScaleBlock, x_bytes = p.boxes * box_bytes;
  const uint32_t stage_bytes = C::KZ * (w_bytes + x_bytes), ring = p.ring;
  const uint32_t lead = rank == 0 ? 1u : 0u;
  const int begins = p.shard_st_begin[lane <= kMaxShards ? lane : kMaxShards];
  const int G = static_cast<int>(gridDim.x) >> 1;
  // The usual case in a loop of its own: this loop alone feeds the tensor cores, and every
  // instruction in it costs.
  const bool simple = p.boxes == 1 && (C::KZ == 1 || p.whole_boxes);
  uint32_t slot = 0, phase = 1, issued = 0;
  bool ok = true;
  for (int id = static_cast<int>(blockIdx.x) >> 1; ok && id < p.tiles; id += G) {
    int m, n0;
    place(p, id, m, n0);
    const int w_row = n0 + static_cast<int>(rank) * (C::TILE_N / 2);
    // Lane i holds box i of this CTA.
    int shard_x, row_x;
    find_box(p, table.box_begin, (2 * m + static_cast<int>(rank)) * p.boxes + lane, shard_x, row_x);
    const int shard_0 = __shfl_sync(0xffffffffu, shard_x, 0), row_0 = __shfl_sync(0xffffffffu, row_x, 0);
    int begin = 0;
    for (int shard = 0; ok && shard < p.k_shards; ++shard) {
      const int end = __shfl_sync(0xffffffffu, begins, shard + 1);
      const CUtensorMap* map_w = &p.tmap_w[shard];
      const CUtensorMap* map_x = &p.tmap_x[p.ag ? shard_0 : shard];
      for (int st = begin; st < end; ++st) {
        ok = wait_bounded(empty0 + 8 * slot, phase, ctl, (kRoleProducer << 8) | 1);
        __syncwarp();
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int kb = (st - begin) * C::KZ;
        const uint32_t full = full0 + 8 * slot, pair = lead0 + 8 * slot;
        const uint32_t sw = base + slot * stage_bytes, sx = sw + C::KZ * w_bytes;
        if (simple) {
          if constexpr (C::KZ == 1)
            stage_copies_pair(lead, full, 2 * stage_bytes, pair, sx, map_x, row_0, sw, map_w, w_row, kb * kScaleBlock,
                              pol_x, pol_w);
          else
            stage_copies_pair_3d(lead, full, 2 * stage_bytes, pair, sx, map_x, row_0, sw, map_w, w_row, kb, pol_x, pol_w);
        } else {
          if (lane == 0) {
            if (rank == 0) arm(full, 2 * stage_bytes);
            if (p.whole_boxes) {
              copy_3d(sw, map_w, pair, 0, w_row, kb, pol_w);
            } else {
#pragma unroll
              for (int j = 0; j < C::KZ; ++j)
                copy_2d(sw + j * w_bytes, map_w, pair, (kb + j) * kScaleBlock, w_row, pol_w);
            }
          }
          __syncwarp();
          if (lane < p.boxes) {
            const CUtensorMap* map = &p.tmap_x[p.ag ? shard_x : shard];
            const uint32_t dst = sx + lane * box_bytes;
#pragma unroll
            for (int j = 0; j < C::KZ; ++j)
              if (p.whole_boxes)
                copy_3d(dst + j * x_bytes, map, pair, 0, row_x, kb + j, pol_x);
              else
                copy_2d(dst + j * x_bytes, map, pair, (kb + j) * kScaleBlock, row_x, pol_x);
          }
          __syncwarp();
        }
        ++issued;
        if (++slot == ring) {
          slot = 0;
          phase ^= 1u;
        }
      }
      begin = end;
    }
  }
  // Let the copies issued land, and the commits that free their slots, before the shared
  // memory goes away. (If a role gave up, no commit may come for the last ones: then the
  // copies complete on the leader's barriers, and the peer waits its limit.)
  const uint32_t first = issued > ring ? issued - ring : 0;
  for (uint32_t i = first; i < issued; ++i) {
    const uint32_t s = i % ring, parity = (i / ring) & 1u;
    if (rank == 0) wait_drain(full0 + 8 * s, parity, 100000000ull);
    if (ok)
      ok = __all_sync(0xffffffffu, wait_bounded(empty0 + 8 * s, parity, ctl, (kRoleProducer << 8) | 2));
    else if (rank != 0)
      wait_drain(empty0 + 8 * s, parity, 100000000ull);
  }
}

// The pair's MMAs (rank 0). What it waits for last, the accumulator, is on the way from the
// epilogue's last read to the next MMA.
template <class C>
__device__ void multiply(const Fp8Params& p, uint32_t base, uint32_t tmem, const Ctl& ctl) {
  const uint32_t full0 = base + C::kBarsOff, empty0 = full0 + 8 * kFp8MaxRing;
  const uint32_t tfull0 = empty0 + 8 * kFp8MaxRing, tempty0 = tfull0 + 8 * C::kAccs, drain = tempty0 + 8 * C::kAccs;
  const uint32_t w_bytes = C::TILE_N / 2 * kScaleBlock, x_bytes = p.boxes * p.box_rows * kScaleBlock;
  const uint32_t stage_bytes = C::KZ * (w_bytes + x_bytes), ring = p.ring;
  const uint32_t idesc = make_idesc_e4m3(2 * C::kRows, C::TILE_N);
  const int G = static_cast<int>(gridDim.x) >> 1;
  uint32_t slot = 0, phase = 0, acc = 0, acc_phase = 1;
  bool ok = true, issued = false;
  for (int id = static_cast<int>(blockIdx.x) >> 1; ok && id < p.tiles; id += G) {
    for (int st = 0; st < p.stages_per_tile; ++st) {
      ok = wait_bounded(full0 + 8 * slot, phase, ctl, (kRoleMma << 8) | 2) &&
           wait_bounded(tempty0 + 8 * acc, acc_phase, ctl, (kRoleMma << 8) | 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t sw = base + slot * stage_bytes, sx = sw + C::KZ * w_bytes;
      if (elected()) {
#pragma unroll
        for (int j = 0; j < C::KZ; ++j)
          mma4_e4m3_pair(tmem + (acc * C::KZ + j) * C::kAccCols, smem_desc_sw128(sx + j * x_bytes),
                         smem_desc_sw128(sw + j * w_bytes), idesc);
        commit_pair_here(tfull0 + 8 * acc, 0x3);
        commit_pair_here(empty0 + 8 * slot, 0x3);
      }
      __syncwarp();
      issued = true;
      if (++slot == ring) {
        slot = 0;
        phase ^= 1u;
      }
      if (++acc == C::kAccs) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }
  // No MMA may be in flight when the accumulators go away, whichever role gave up.
  if (issued) {
    mma_commit_pair(drain, 0x1);
    wait_drain(drain, 0, 100000000ull);
  }
}

// An epilogue thread's N sums. PAIRS: two by two in 64-bit registers, whose operands the
// compiler has to place in pairs; with 128 sums it has no room to (tiles of 256 at M = 4096,
// N = K = 7168: 165 us in pairs, 150 alone; of 192 169 and 175).
template <bool PAIRS, int N>
struct Sums {
  float v[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
  }
  // 16 columns from c on += s * x.
  __device__ __forceinline__ void add(int c, const uint32_t* x, float s) {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[c + e] = fmaf(__uint_as_float(x[e]), s, v[c + e]);
  }
  __device__ __forceinline__ uint32_t two(int c) const { return pack_bf16x2(__float_as_uint(v[c]), __float_as_uint(v[c + 1])); }
};
template <int N>
struct Sums<true, N> {
  unsigned long long v[N / 2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v[i] = 0;
  }
  __device__ __forceinline__ void add(int c, const uint32_t* x, float s) {
    unsigned long long ss, xx;
    asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      asm("mov.b64 %0, {%1, %2};" : "=l"(xx) : "r"(x[e]), "r"(x[e + 1]));
      asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(v[(c + e) / 2]) : "l"(xx), "l"(ss));
    }
  }
  __device__ __forceinline__ uint32_t two(int c) const {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v[c / 2]));
    return pack_bf16x2(a, b);
  }
};
// 8 sums from c on in bf16.
template <class S>
__device__ __forceinline__ uint4 pack_8(const S& sums, int c) {
  return make_uint4(sums.two(c), sums.two(c + 2), sums.two(c + 4), sums.two(c + 6));
}

// 4 bytes to shared memory, or zeros; asynchronous.
__device__ __forceinline__ void copy_4(uint32_t dst, const float* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}

// The scales as they are, by one warp, four k-blocks of the tile's walk over K at a time.
// Rows that no shard has and positions past the walk's end or that pad a K-shard to whole
// stages have scale 0 (the sums of the latter are 0).
template <class C>
__device__ void copy_scales(const Fp8Params& p, Shared<C>& sh, uint32_t base, uint32_t rank, const Ctl& ctl) {
  constexpr int kPer = C::kRows / 32;   // rows of a lane
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t rfull0 = base + C::kBarsOff + C::kRawBarsOff, rempty0 = rfull0 + 8 * kFp8RawRing;
  const int G = static_cast<int>(gridDim.x) >> 1;
  const int last_block = (p.N - 1) / kScaleBlock;
  uint32_t slot = 0, phase = 1;
  bool ok = true;
  for (int id = static_cast<int>(blockIdx.x) >> 1; ok && id < p.tiles; id += G) {
    int m, n0;
    place(p, id, m, n0);
    int shard_x[kPer], row[kPer];
    bool live[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = lane + 32 * i, box = r / p.box_rows;
      find_box(p, sh.table.box_begin, (2 * m + static_cast<int>(rank)) * p.boxes + box, shard_x[i], row[i]);
      row[i] += r - box * p.box_rows;
      live[i] = box < p.boxes && row[i] < sh.table.rows[shard_x[i]];
    }
    const int block = min(n0 / kScaleBlock + lane, last_block);   // (of the first lanes)
    int shard = 0, n = sh.table.kb[0], kb = 0;
    const float *x[kPer], *w = nullptr;
    int64_t step[kPer];
    auto enter = [&]() {   // K-shard `shard`
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] = sh.table.sx[p.ag ? shard_x[i] : shard] + (live[i] ? row[i] : 0);
      w = sh.table.sw[shard] + static_cast<int64_t>(block) * n;
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) step[i] = live[i] ? sh.table.rows[shard_x[i]] : 0;
    enter();
    while (shard < p.k_shards) {
      ok = wait_bounded(rempty0 + 8 * slot, phase, ctl, (kRoleProducer << 8) | 3);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const RawScales<C>& to = sh.raw[slot];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool real = shard < p.k_shards && kb < n;
#pragma unroll
        for (int i = 0; i < kPer; ++i) copy_4(smem_u32(&to.x[j][lane + 32 * i]), x[i], real && live[i]);
        if (lane < C::kBlocks) copy_4(smem_u32(&to.w[j][lane]), w, real);
        if (real && kb + 1 < n) {   // (never past the last one's address)
#pragma unroll
          for (int i = 0; i < kPer; ++i) x[i] += step[i];
          ++w;
        }
        if (++kb >= (n + C::KZ - 1) / C::KZ * C::KZ && shard < p.k_shards) {
          kb = 0;
          if (++shard < p.k_shards) {
            n = sh.table.kb[shard];
            enter();
          }
        }
      }
      sign_copies(rfull0 + 8 * slot);
      if (++slot == kFp8RawRing) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Their products, by another warp.
template <class C>
__device__ void multiply_scales(const Fp8Params& p, Shared<C>& sh, uint32_t base, const Ctl& ctl) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t sfull0 = base + C::kBarsOff + C::kScaleBarsOff, sempty0 = sfull0 + 8 * kFp8ScaleRing;
  const uint32_t rfull0 = base + C::kBarsOff + C::kRawBarsOff, rempty0 = rfull0 + 8 * kFp8RawRing;
  const int G = static_cast<int>(gridDim.x) >> 1;
  const int groups = (p.stages_per_tile * C::KZ + 3) / 4;
  uint32_t group = 0;
  for (int id = static_cast<int>(blockIdx.x) >> 1; id < p.tiles; id += G)
    for (int i = 0; i < groups; ++i, ++group) {
      const uint32_t in = group % kFp8RawRing, out = group % kFp8ScaleRing;
      const bool ok = wait_bounded(rfull0 + 8 * in, (group / kFp8RawRing) & 1u, ctl, (kRoleMma << 8) | 3) &&
                      wait_bounded(sempty0 + 8 * out, ((group / kFp8ScaleRing) & 1u) ^ 1u, ctl, (kRoleMma << 8) | 4);
      if (!__all_sync(0xffffffffu, ok)) return;
      const RawScales<C>& from = sh.raw[in];
#pragma unroll
      for (int r = lane; r < C::kRows; r += 32) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = from.x[j][r];
#pragma unroll
        for (int b = 0; b < C::kBlocks; ++b)
          sh.scales[out].s[b][r] =
              make_float4(x[0] * from.w[0][b], x[1] * from.w[1][b], x[2] * from.w[2][b], x[3] * from.w[3][b]);
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(sfull0 + 8 * out);
        mbar_arrive(rempty0 + 8 * in);
      }
    }
}

// wait_bounded without its call, across which the epilogue's registers would be saved.
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, const Ctl& c, uint32_t site) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns(), limit = c.timeout_ns * (site >> 8);
  while (!mbar_try_wait(bar, parity)) {
    if (*c.abort) return false;
    if (global_timer_ns() - t0 > limit) {
      *c.abort = 1;
      atomicCAS(c.status, 0u, kStatusTimeout | site);
      return false;
    }
  }
  return true;
}

// N columns of the sums at `at`, a multiple of 16 up to 64: issued, and waited for.
template <int N>
__device__ __forceinline__ void read_sums(uint32_t at, uint32_t (&v)[N]) {
  if constexpr (N == 64) {
    tmem_ld_64cols(at, v);
  } else if constexpr (N == 16) {
    tmem_ld_16cols(at, v);
  } else {
    tmem_ld_32cols(at, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
    if constexpr (N == 48) tmem_ld_16cols(at + 32, &v[32]);
  }
}
template <int N>
__device__ __forceinline__ void wait_sums(uint32_t (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  // No use of the registers before the wait.
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]),
                      "+r"(v[i + 6]), "+r"(v[i + 7]));
}

__device__ __forceinline__ void load_scales(uint32_t at, float (&s)[4]) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(s[0]), "=f"(s[1]), "=f"(s[2]), "=f"(s[3])
               : "r"(at)
               : "memory");
}

// A warp's 32 rows x COLS columns through its staging, 64 or 32 columns at a time in the
// swizzled layout of the copy (128 or 64 bytes a row: 8 lanes' 16-byte stores meet in no
// bank), then a copy each, which leave out what lies past the shard's rows and N. They
// read the staging while the next tile is under way. (Stored straight from the registers,
// a row per lane, a tile took 2.6 us; with staging for 32 columns alone, 2.)
template <int COLS, class S>
__device__ __forceinline__ void store_tile(const CUtensorMap* map, uint32_t staging, int row, int col, int N, bool rows,
                                           const S& sums) {
  constexpr int kWidth = fp8_store_cols(2 * COLS);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t at = staging + lane * (2 * kWidth);
  const int turn = kWidth == 64 ? lane & 7 : lane >> 1 & 3;
  constexpr int kStaged = fp8_staged_cols(2 * COLS);
#pragma unroll
  for (int c0 = 0; c0 < COLS; c0 += kStaged) {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // (lane 0's: the others have none)
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kStaged; c += 8) {
      const uint4 w = pack_8(sums, c0 + c);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::
                   "r"(at + c / kWidth * (64 * kWidth) + (((c % kWidth >> 3) ^ turn) << 4)), "r"(w.x), "r"(w.y), "r"(w.z),
                   "r"(w.w)
                   : "memory");
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0 && rows) {
#pragma unroll
      for (int c = 0; c < kStaged; c += kWidth)
        if (col + c0 + c < N)
          asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::
                       "l"(reinterpret_cast<uint64_t>(map)), "r"(col + c0 + c), "r"(row),
                       "r"(staging + c / kWidth * (64 * kWidth))
                       : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
}

template <class C>
__device__ void finish(const Fp8Params& p, const Shared<C>& sh, uint32_t base, uint32_t tmem, uint32_t rank,
                       const Ctl& ctl) {
  const Table& table = sh.table;
  const uint32_t tfull0 = base + C::kBarsOff + 16 * kFp8MaxRing, tempty0 = tfull0 + 8 * C::kAccs;
  const uint32_t sfull0 = base + C::kBarsOff + C::kScaleBarsOff, sempty0 = sfull0 + 8 * kFp8ScaleRing;
  const uint32_t lead_tempty = map_shared_to_rank(tempty0, 0);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int warp = static_cast<int>(threadIdx.x) >> 5;
  const int quad = warp & 3;                        // TMEM lanes this warp may read
  const int half = C::WIDE ? (warp - 4) >> 2 : quad >> 1;   // of the tile's columns
  const int row0 = C::WIDE ? quad * 32 : (quad & 1) * 32;   // first token row of the CTA
  const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + (C::WIDE ? half * C::kCols : 0);
  const uint32_t scales0 = smem_u32(&sh.scales[0].s[0][row0 + lane]);
  const int G = static_cast<int>(gridDim.x) >> 1;
  uint32_t acc = 0, acc_phase = 0, slot = 0, phase = 0;
  bool ok = true;
  for (int id = static_cast<int>(blockIdx.x) >> 1; ok && id < p.tiles; id += G) {
    int m, n0;
    place(p, id, m, n0);
    const int col0 = n0 + half * C::kCols;
    // The warp's block of weight rows among the tile's, if it has one, or its columns before
    // the tile's second block.
    const int b0 = col0 / kScaleBlock - n0 / kScaleBlock;
    const int split = (n0 / kScaleBlock + 1) * kScaleBlock - col0;
    Sums<C::TILE_N != 256, C::kCols> sums;
    sums.clear();
    float s0[4], s1[4];
    auto next_scales = [&]() {   // four k-blocks'
      ok = wait_here(sfull0 + 8 * slot, phase, ctl, (kRoleEpilogue << 8) | 2) && ok;
      const uint32_t at = scales0 + slot * static_cast<uint32_t>(sizeof(GroupScales<C>));
      load_scales(at + (C::kOneBlock ? b0 : 0) * (16 * C::kRows), s0);
      if constexpr (!C::kOneBlock) load_scales(at + 16 * C::kRows, s1);
      __syncwarp();   // read by every lane
      if (lane == 0) mbar_arrive(sempty0 + 8 * slot);
      if (++slot == kFp8ScaleRing) {
        slot = 0;
        phase ^= 1u;
      }
    };
    for (int st = 0; ok && st < p.stages_per_tile;) {
      next_scales();
#pragma unroll
      for (int i = 0; i < 4 / C::KZ; ++i) {
        if (st >= p.stages_per_tile) break;
        ++st;
        ok = ok && wait_here(tfull0 + 8 * acc, acc_phase, ctl, (kRoleEpilogue << 8) | 1);
        // Every lane together, also after a wait that ran out (the vote is below).
        __syncwarp();
        tc_fence_after_sync();
        const uint32_t at = taddr + acc * C::KZ * C::kAccCols;
        uint32_t v[2][C::kUnit];
        read_sums<C::kUnit>(at, v[0]);
#pragma unroll
        for (int u = 0; u < C::kUnits; ++u) {
          wait_sums<C::kUnit>(v[u & 1]);
          if (u + 1 < C::kUnits) {
            read_sums<C::kUnit>(at + (u + 1) / C::kPerBlock * C::kAccCols + (u + 1) % C::kPerBlock * C::kUnit,
                                v[(u + 1) & 1]);
          } else {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) sign_pair(lead_tempty + 8 * acc);
          }
          const int j = i * C::KZ + u / C::kPerBlock, c0 = u % C::kPerBlock * C::kUnit;
#pragma unroll
          for (int c = 0; c < C::kUnit; c += 16)
            sums.add(c0 + c, v[u & 1] + c, C::kOneBlock || c0 + c < split ? s0[j] : s1[j]);
        }
        if (++acc == C::kAccs) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
    if (!ok) break;
    // The warp's rows: their box, the box's shard and row.
    if constexpr (C::WIDE) {
      if (p.tma_store) {
        const int box = row0 / p.box_rows;
        int shard, row;
        find_box(p, table.box_begin, (2 * m + static_cast<int>(rank)) * p.boxes + box, shard, row);
        row += row0 - box * p.box_rows;
        const uint32_t staging = base + C::kStagingOff + (warp - 4) * (64 * fp8_staged_cols(C::TILE_N));
        store_tile<C::kCols>(&p.tmap_y[shard], staging, row, col0, p.N, box < p.boxes && row < table.rows[shard], sums);
        continue;
      }
    }
    const int box = (row0 + lane) / p.box_rows;
    int shard, row;
    find_box(p, table.box_begin, (2 * m + static_cast<int>(rank)) * p.boxes + box, shard, row);
    row += row0 + lane - box * p.box_rows;
    if (box < p.boxes && row < table.rows[shard]) {
      uint16_t* y = p.y + static_cast<size_t>(table.row_begin[shard] + row) * p.N + col0;
#pragma unroll
      for (int c = 0; c < C::kCols; c += 8)
        if (col0 + c < p.N) *reinterpret_cast<uint4*>(y + c) = pack_8(sums, c);
    }
  }
  // The last copies have read the staging before the shared memory goes away.
  if (C::WIDE) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) gsr_fp8_kernel(const __grid_constant__ Fp8Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + C::kMiscOff + 4);
  Shared<C>& sh = *reinterpret_cast<Shared<C>*>(base_ptr + C::kTableOff);
  Table& table = sh.table;
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t bars = base + C::kBarsOff;
  if (warp == 0) {
    if (lane < p.k_shards) fetch_descriptor(&p.tmap_w[lane]);
    if (lane < (p.ag ? p.m_shards : p.k_shards)) fetch_descriptor(&p.tmap_x[lane]);
    if (C::WIDE && p.tma_store && lane < p.m_shards) fetch_descriptor(&p.tmap_y[lane]);
  } else if (warp == 1) {
    if (lane == 0) {
      for (uint32_t i = 0; i < kFp8MaxRing; ++i) {
        mbar_init(bars + 8 * i, 1);                    // full: the leader's expect_tx + the pair's bytes
        mbar_init(bars + 8 * (kFp8MaxRing + i), 1);    // empty: the MMAs' commit
      }
      for (uint32_t i = 0; i < C::kAccs; ++i) {
        mbar_init(bars + 16 * kFp8MaxRing + 8 * i, 1);                             // sums ready
        mbar_init(bars + 16 * kFp8MaxRing + 8 * (C::kAccs + i), 2 * C::kEpi / 32);   // read by the pair's warps
      }
      mbar_init(bars + 16 * kFp8MaxRing + 16 * C::kAccs, 1);
      for (uint32_t i = 0; i < kFp8ScaleRing; ++i) {
        mbar_init(bars + C::kScaleBarsOff + 8 * i, 1);
        mbar_init(bars + C::kScaleBarsOff + 8 * (kFp8ScaleRing + i), C::kEpi / 32);   // read by the warps
      }
      for (uint32_t i = 0; i < kFp8RawRing; ++i) {
        mbar_init(bars + C::kRawBarsOff + 8 * i, 32);   // each lane's copies
        mbar_init(bars + C::kRawBarsOff + 8 * (kFp8RawRing + i), 1);
      }
      *abort_flag = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
    tmem_alloc_pair(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish_pair();
  } else if (warp == 2) {
    if (lane < kMaxShards) {
      table.sx[lane] = p.sx[lane];
      table.sw[lane] = p.sw[lane];
      table.row_begin[lane] = p.shard_row_begin[lane];
      table.kb[lane] = p.shard_kb[lane];
      table.rows[lane] = p.shard_rows[lane];
    }
    if (lane <= kMaxShards) table.box_begin[lane] = p.box_begin[lane];
  }
  tc_fence_before_sync();
  cluster_barrier();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  grid_dependency_wait();

  Ctl ctl{abort_flag, p.status, p.timeout_ns};
  if (warp < 4) {
    if constexpr (C::WIDE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRoleRegs));
    if (warp == 0)
      produce<C>(p, table, base, rank, ctl);
    else if (warp == 1 && rank == 0)
      multiply<C>(p, base, tmem, ctl);
    else if (warp == 2)
      copy_scales<C>(p, sh, base, rank, ctl);
    else if (warp == 3)
      multiply_scales<C>(p, sh, base, ctl);
  } else {
    if constexpr (C::WIDE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kEpiRegs));
    finish<C>(p, sh, base, tmem, rank, ctl);
  }
  __syncwarp();
  tc_fence_before_sync();
  cluster_barrier();   // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, C::kTmemCols);
  }
  // After a timed-out wait, the peer may have sent what this CTA stopped waiting for:
  // the CTA stays until that has surely landed.
  if (threadIdx.x == 0 && *abort_flag) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 20000ull) __nanosleep(1000);
  }
}

template <class C>
cudaError_t set_limit() {
  if (C::WIDE) {   // the split of the registers counts on the launch's
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, gsr_fp8_kernel<C>);
    if (e != cudaSuccess) return e;
    if (a.numRegs < C::kLaunchRegs) return cudaErrorInvalidKernelImage;
  }
  return cudaFuncSetAttribute(gsr_fp8_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(smem_bytes<C>()));
}

template <class C>
cudaError_t launch_one(const Fp8Params& p, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes<C>();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gsr_fp8_kernel<C>, p);
}

template <int FORM>
cudaError_t set_limits() {
  constexpr int n = fp8_max_tile_n(FORM) / 4;
  cudaError_t e = set_limit<Cfg<FORM, n>>();
  if (e == cudaSuccess) e = set_limit<Cfg<FORM, 2 * n>>();
  if (e == cudaSuccess) e = set_limit<Cfg<FORM, 3 * n>>();
  if (e == cudaSuccess) e = set_limit<Cfg<FORM, 4 * n>>();
  return e;
}

template <int FORM>
cudaError_t launch_form(const Fp8Params& p, int ctas, cudaStream_t stream) {
  constexpr int n = fp8_max_tile_n(FORM) / 4;
  switch (p.tile_n) {
    case n: return launch_one<Cfg<FORM, n>>(p, ctas, stream);
    case 2 * n: return launch_one<Cfg<FORM, 2 * n>>(p, ctas, stream);
    case 3 * n: return launch_one<Cfg<FORM, 3 * n>>(p, ctas, stream);
    default: return launch_one<Cfg<FORM, 4 * n>>(p, ctas, stream);
  }
}

}  // namespace

cudaError_t prepare_fp8_kernels() {
  const cudaError_t e = set_limits<kFp8Wide>();
  return e == cudaSuccess ? set_limits<kFp8Narrow>() : e;
}

cudaError_t launch_fp8(const Fp8Params& p, int form, int ctas, cudaStream_t stream) {
  return form == kFp8Wide ? launch_form<kFp8Wide>(p, ctas, stream) : launch_form<kFp8Narrow>(p, ctas, stream);
}

}  // namespace gsr
