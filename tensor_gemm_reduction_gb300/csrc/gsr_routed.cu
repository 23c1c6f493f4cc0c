// gsr_routed.cu -- products whose weights the row picks, for GB300 (sm_103a).
//
//   kGrouped  Y[i] = X[i] . W[e]^T          for the rows i of group e
//   kGated    Y[i] = silu(g) * u, g = X[i] . Wg[e]^T, u = X[i] . Wu[e]^T
//   kLora     Y[i] = sum_r X_r[i] . W_r^T + low[i] . B[a]^T, a = adapter[i]
//
// The groups' sizes are known on the device only, from none to every row. So
// the weights' rows, not the tokens, are the MMA's M: a CTA pair owns a tile of
// 256 weight rows (tcgen05.mma.cta_group::2, 128 rows per CTA) against n
// tokens of one group, n any multiple of 16 up to the instance's capacity, as
// the MMA's N. A group of one row costs 16 columns of an MMA and not 128, and
// with few rows the kernel is a stream of weights; with many it is a 256 x 256
// tile. A group's tokens are cut into tiles of equal width.
//
// Every CTA counts the tiles itself from the offsets (a scan over the groups in
// shared memory). Whole waves of tiles are dealt round-robin. The remaining ones are
// walked first; where their number leaves pairs idle and k is long, each is cut
// along k into equal pieces, one per pair, whose fp32 partials the last piece to
// arrive sums in k order. The cuts depend on the group sizes alone, so results are
// reproducible. (Cutting the remaining k evenly over all pairs, most of which then
// hold pieces of two tiles, was slower in every case measured: 36 tiles of 256 rows
// x 256 tokens, K = 7168, 49 us whole tiles 44; 24 tiles 41, in threes 38.)
//
// Roles: warp 0 TMA producer, warp 1 MMA issuer (the pair's leader), warps 2..5
// epilogue. With gathered rows, warps 6..9 copy them and warp 10 signs them.
// kLora has warps 6..9 besides, which place the low-rank rows: the
// adapters of a token tile are more steps over k, in which the weights are
// B[a] and a token's row is low[i] if its adapter is a and zero if not, so the
// sum stays in the same fp32 accumulator. Those masked rows exist in shared
// memory alone.
//
// Epilogue: a warp takes 32 output columns of 32 tokens at a time from TMEM in
// the fragment layout of 8 x 8 matrices, writes them transposed to 2 KB of shared
// memory of its own (stmatrix) and stores them as 16-byte vectors, 64 bytes per
// row. (Stores of two columns straight from registers took 6.3 us for 256 tokens
// x 128 columns, more than the MMAs of a tile at K = 896.)
//
// Measured. Streams of weights: 64 groups of a row or two, N = 7168, K = 896, 104 us
// (0.97 of the copy bandwidth); AR with adapters, M = 1, N = K = 7168, 25 us (a single
// launch's fixed cost beside 15). Tiles, in short bursts, below the power limit: one
// group of 4096 rows, N = K = 7168, 1.95 PFLOP/s; 64 uneven groups of about 512, bound by
// reading tiles from L2 (14 TB/s) and by their starts, 1.36 at K = 896 and 1.47 gathered,
// gated, at K = 7168; M = 4096 with 8 adapters of rank 64, 1.58 with the low-rank kernel's
// 20 of 270 us. In long runs at the limit the last three take 350, 655 and 304 us: 1.20,
// 1.28 and 1.40 PFLOP/s.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gsr_device.cuh"
#include "gsr_routed.h"

namespace gsr {
namespace {

constexpr int kEpi = 128;              // epilogue threads
constexpr int kPlacers = 4;            // warps that place (or gather) the rows of a stage
constexpr uint32_t kRolePlacer = 4;
// kLora: more than the tiles in flight between the placing warps and the epilogue (a
// ring of single-stage tiles and two accumulators).
constexpr int kMarks = 32;

// 16 bytes to shared memory, or 16 zeros; asynchronous.
__device__ __forceinline__ void copy_16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0)
               : "memory");
}
// 32 TMEM columns of 16 lanes: v[4 g + e] is column 8 g + 2 (lane % 4) + e % 2 of
// lane (lane / 4) + 8 (e / 2).
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
// Four 8 x 8 matrices of 16-bit elements, transposed: lane l gives the address of
// row l % 8 of matrix l / 8.
__device__ __forceinline__ void store_transposed(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                 uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void sign_many(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// ------------------------------------------------------------ geometry

// The shards of X and A, read from the parameters at the kernel's start (cold
// parameters cost a memory access each where they are used).
struct SelfTable {
  const uint16_t *x[kMaxShards], *a[kMaxShards];
  int k[kMaxShards];
};

template <int KIND_, bool GATHER_, bool HALF_, int TOK_, int KZ_, int STAGES_>
struct Cfg {
  static constexpr int KIND = KIND_, TOK = TOK_, S = STAGES_, KZ = KZ_;
  static constexpr bool GATHER = GATHER_, HALF = HALF_;
  static constexpr int kTeams = HALF ? 2 : 1;           // kLora: of four warps that place rows
  static constexpr bool SELF = HALF && TOK == kRoutedSmall;   // may compute the low-rank rows itself
  static constexpr int kRows = HALF ? 64 : 128;         // weight rows of a CTA, at most
  static constexpr int kThreads = 64 + kEpi + (KIND == kLora ? 32 * kPlacers : GATHER ? 32 * (kPlacers + 1) : 0);
  // Arrivals that complete a full barrier: the leader's expect_tx and, from both
  // CTAs, the placing warps or the warp that signs for the gathered rows.
  static constexpr uint32_t kSigns = 1 + (KIND == kLora ? 2 * kPlacers : GATHER ? 2 : 0);
  static constexpr uint32_t kW = kRows * 128;           // a k-block of this CTA's weight rows
  static constexpr uint32_t kX = TOK / 2 * 128;         // a k-block of this CTA's tokens
  static constexpr uint32_t kStage = KZ * (kW + kX);
  static constexpr uint32_t kRing = S * kStage;
  // Half tiles lay the ring out by the call's own rows and tokens, so that few of
  // them leave more stages in flight: kSlots is the most.
  static constexpr uint32_t kSlots = HALF ? kHalfSlots : S;
  static_assert(!HALF || kRing >= kHalfRing, "the host counts the stages");
  // full[kSlots], empty[kSlots], tmem_full[2], tmem_empty[2], drain; landed[kSlots]: this CTA's
  // adapter weights (kLora) or gathered rows; granted[kSlots] (kLora): the slot is free
  // for an adapter stage; looked (kLora): the tile's adapters are looked over
  static constexpr uint32_t kBars = (2 * kSlots + 5 + (KIND == kLora ? 2 * kSlots + 1 : GATHER ? kSlots : 0)) * 8;
  static constexpr uint32_t kLandedOff = (2 * kSlots + 5) * 8, kGrantedOff = kLandedOff + kSlots * 8;
  static constexpr uint32_t kLookedOff = kGrantedOff + kSlots * 8;
  static constexpr uint32_t kGroups = KIND == kLora ? 0 : 4 * (3 * kMaxGroups + 1 + 32);
  static constexpr uint32_t kStaging = 4 * 2048;        // 2 KB per epilogue warp
  static constexpr uint32_t kBarsOff = kRing;
  static constexpr uint32_t kMiscOff = kBarsOff + kBars;
  static constexpr uint32_t kStagingOff = (kMiscOff + 16 + 4 * (kMarks + 3) + 127) / 128 * 128;
  static constexpr uint32_t kGroupsOff = kStagingOff + kStaging;
  static constexpr uint32_t kSelf = SELF ? sizeof(SelfTable) + 8 * 4 * kSelfElements : 0;
  static constexpr uint32_t kSmem = 1024 + kGroupsOff + kGroups + kSelf;
  static_assert(kSmem <= kSmallSmemLimit, "shared memory");
  static_assert(kX % 1024 == 0, "swizzle atoms");
  static_assert(!GATHER || TOK <= 256, "gathered rows: one MMA's tokens");
  // Accumulators: two, so that a tile's epilogue runs beside the next tile's
  // MMAs, or one of 512 tokens.
  static constexpr uint32_t kAccs = TOK == 512 ? 1 : 2;
  static constexpr uint32_t kTmemCols = kAccs * TOK;
};

// The ring's geometry: bytes of a k-block of weights and of tokens, of a stage, of a
// unit of an adapter stage, and the stages in use.
template <class C>
struct Geometry {
  uint32_t w, x, stage, slots, unit_w, unit_x;
  __device__ __forceinline__ explicit Geometry(const RoutedParams& p) {
    w = C::HALF ? 128u * p.w_rows : C::kW;
    x = C::HALF ? 64u * p.tile_tokens : C::kX;
    stage = C::KZ * (w + x);
    slots = C::HALF ? static_cast<uint32_t>(p.stages) : C::S;
    unit_w = C::KIND == kLora ? w / 64u * p.unit_cols : 0u;
    unit_x = C::KIND == kLora ? x / 64u * p.unit_cols : 0u;
  }
};

// The groups as every CTA counts them (shared memory).
struct Groups {
  int *row, *count, *tile;    // first row, rows, first token tile (E + 1)
};

struct Tile {
  int row0, rows, n;          // first row of Y, rows, MMA columns (a multiple of 16; above
                              // 256 in two MMAs, see halves)
  int col0;                   // first output column of the pair
  int group, m;               // group; lora: token tile
  int piece, npieces, slot, cut;    // cut: index among the cut tiles
  int st, st_end;             // stages
};

// a / b for small operands by a float reciprocal: (a + 1/2) / b is at least 1 / 2b
// from an integer and the quotient's error below a / b * 2^-21, so it is exact
// while a < 2^19. An integer division takes some hundred cycles, and a tile's
// place takes four.
__device__ __forceinline__ int quotient(int a, int b) {
  if (a >= (1 << 19)) return a / b;
  return static_cast<int>(__fdividef(static_cast<float>(a) + 0.5f, static_cast<float>(b)));
}

template <class C>
__device__ __forceinline__ void place(const RoutedParams& p, const Groups& g, int id, Tile& t) {
  int local, mt, width, count;
  if constexpr (C::KIND == kLora) {
    local = id;
    mt = p.m_tiles;
    width = p.tile_tokens;
    count = p.M;
    t.row0 = 0;
    t.group = 0;
  } else {
    // The last group whose first token tile is at or below this one (empty
    // groups share their successor's).
    const int key = quotient(id, p.n_tiles);
    int lo = 0, hi = p.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g.tile[mid] <= key) lo = mid; else hi = mid;
    }
    t.group = lo;
    mt = g.tile[lo + 1] - g.tile[lo];
    local = id - g.tile[lo] * p.n_tiles;
    count = g.count[lo];
    t.row0 = g.row[lo];
    width = (quotient(count + mt - 1, mt) + 15) & ~15;
  }
  // Raster: 16 token tiles at a time, tokens fastest, so that concurrent pairs
  // share weight rows.
  const int span = 16 * p.n_tiles;
  const int sup = quotient(local, span);
  const int gm = min(mt - sup * 16, 16);
  const int in = local - sup * span, col = quotient(in, gm);
  t.m = sup * 16 + in - col * gm;
  t.col0 = col * (2 * p.cta_cols);
  t.row0 += t.m * width;
  t.rows = min(width, count - t.m * width);
  t.n = C::KIND == kLora ? width : (t.rows + 15) & ~15;
}

// A CTA's rows of the tokens [0, n) of a tile: with n <= 256, h[0] = n / 2 rows from
// rank * h[0] on; with more, two MMAs' worth, the second from 2 h[0] + rank * h[1] on.
struct Halves {
  int h[2];
  __device__ __forceinline__ explicit Halves(int n) {
    h[0] = n <= 256 ? n / 2 : ((n / 2 + 15) / 16) * 8;
    h[1] = n / 2 - h[0];
  }
};

constexpr int kMinPiece = 2;   // stages of a piece, at least

// Every role walks the same tiles: this worker's piece of a cut tile, or a whole
// one, of the remainder, then its other tiles.
struct Walk {
  int G, next, whole, S;
  int cut, piece, pieces;   // of the remainder: tile (-1: none, or done), piece of it

  __device__ __forceinline__ void begin(const RoutedParams& p, int tiles) {
    const int w = static_cast<int>(blockIdx.x) >> 1;
    G = static_cast<int>(gridDim.x) >> 1;
    S = p.stages_per_tile;
    const int rem = tiles % G;
    whole = tiles - rem;
    next = w;
    pieces = 1;
    if (rem > 0) {
      const int n = min(min(G / rem, p.max_pieces), S / kMinPiece);
      if (n > 1 && S - S / n > (whole ? p.cut_ahead : p.cut_alone)) pieces = n;
    }
    cut = w < rem * pieces ? w / pieces : -1;
    piece = w % pieces;
  }
  // First stage of a piece.
  __device__ __forceinline__ int bound(int i) const {
    return static_cast<int>(static_cast<long long>(i) * S / pieces);
  }

  template <class C>
  __device__ __forceinline__ bool step(const RoutedParams& p, const Groups& g, Tile& t) {
    int id;
    if (cut >= 0) {
      id = whole + cut;
      t.cut = cut;
      t.st = bound(piece);
      t.st_end = bound(piece + 1);
      t.piece = piece;
      t.npieces = pieces;
      t.slot = cut * pieces;
      cut = -1;
    } else {
      if (next >= whole) return false;
      id = next;
      next += G;
      t.cut = 0;
      t.st = 0;
      t.st_end = S;
      t.piece = 0;
      t.npieces = 1;
      t.slot = 0;
    }
    place<C>(p, g, id, t);
    return true;
  }
};

// The groups' rows clamped to the matrix, and the prefix of their token tiles:
// each thread scans a run of groups, warps and then the block add up. Called by
// all threads of the block.
template <class C>
__device__ int count_groups(const RoutedParams& p, const Groups& g, int* sums) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = C::kThreads / 32;
  const int per = (p.E + C::kThreads - 1) / C::kThreads;
  const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
  int mine = 0;
  for (int e = e0; e < e1; ++e) {
    const int lo = min(max(p.offsets[e], 0), p.M), hi = min(max(p.offsets[e + 1], 0), p.M);
    const int count = max(hi - lo, 0);
    g.row[e] = lo;
    g.count[e] = count;
    mine += (count + C::TOK - 1) / C::TOK;
  }
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int at = incl - mine, total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) at += sums[i];
    total += sums[i];
  }
  for (int e = e0; e < e1; ++e) {
    g.tile[e] = at;
    at += (g.count[e] + C::TOK - 1) / C::TOK;
  }
  if (tid == 0) g.tile[p.E] = total;
  __syncthreads();
  return total;
}

// ------------------------------------------------------------ adapters of a tile

// The steps over the adapters of token tile m that belong to this piece: a piece
// of a cut tile takes the share that it has of the base product. Read by whole warps, after the
// low-rank kernel has completed; the lanes hold 32 of the tile's adapters.
struct AdapterSteps {
  const int32_t* list;
  int units, st, st_end, per_stage;
  int held, first;   // this lane's adapter, and lane 0's place in the list
  template <class C>
  __device__ __forceinline__ void begin(const RoutedParams& p, const Tile& t) {
    list = p.lists + static_cast<size_t>(t.m) * kAdapterListStride;
    const bool self = C::SELF && p.self_rows;
    int count = 0, own = -1;
    uint32_t leaders = 0;
    if (self) {
      // No list for so few rows: their adapters in the order of their first rows.
      const int lane = static_cast<int>(threadIdx.x) & 31;
      own = lane < p.M ? p.adapter[lane] : -1;
      if (own >= p.L) own = -1;
      const uint32_t same = __match_any_sync(0xffffffffu, own);
      leaders = __ballot_sync(0xffffffffu, own >= 0 && (same & ((1u << lane) - 1u)) == 0);
      count = __popc(leaders);
    } else {
      count = __ldcg(list);
    }
    units = count * p.units_per_adapter;
    per_stage = C::KZ * 64 / p.unit_cols;
    const int stages = (units + per_stage - 1) / per_stage;
    st = t.st * stages / p.stages_per_tile;
    st_end = t.st_end * stages / p.stages_per_tile;
    if (self) {
      first = 0;
      const int lane = static_cast<int>(threadIdx.x) & 31;
      held = __shfl_sync(0xffffffffu, own, lane < count ? __fns(leaders, 0, lane + 1) : 0);
    } else {
      hold(st * per_stage / p.units_per_adapter);
    }
  }
  // (Past the list's end: whatever the workspace holds, never used.)
  __device__ __forceinline__ void hold(int at) {
    first = at;
    const int i = at + (static_cast<int>(threadIdx.x) & 31);
    held = i < kRoutedMaxTokens ? __ldcg(list + 1 + i) : 0;
  }
  // The adapter of unit u (warp-uniform, ascending over the calls).
  __device__ __forceinline__ int adapter(const RoutedParams& p, int u) {
    const int at = p.units_per_adapter == 2 ? u >> 1 : u;
    if (at >= first + 32) hold(at);
    return __shfl_sync(0xffffffffu, held, at - first);
  }
  __device__ __forceinline__ int units_in(int s) const { return min(per_stage, units - s * per_stage); }
};

// Matrix descriptor of rows of `cols` bf16 (16, 32 or 64), swizzled over 32, 64
// or 128 bytes: 8-row groups 16 * cols bytes apart.
__device__ __forceinline__ uint64_t unit_desc(uint32_t saddr, int cols) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(cols) << 32;               // 16 * cols >> 4
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(cols == 64 ? 2 : cols == 32 ? 4 : 6) << 61;
  return d;
}

// The MMAs of one adapter stage, by one thread: an election and fresh descriptors
// per MMA took 75 ns of its issue, three times the tensor cores' own time.
template <int COLS, class C>
__device__ __forceinline__ void multiply_units(const Geometry<C>& geo, uint32_t d, uint32_t sw, uint32_t sx,
                                               uint32_t idesc, int units) {
  uint64_t w = unit_desc(sw, COLS), x = unit_desc(sx, COLS);
  for (int u = 0; u < units; ++u) {
#pragma unroll
    for (int k = 0; k < COLS / 16; ++k)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "setp.eq.b32 p, 0, 0;\n\t"
          "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
          "l"(w + 2 * k), "l"(x + 2 * k), "r"(idesc)
          : "memory");
    w += geo.unit_w / 16;   // addresses are in units of 16 bytes
    x += geo.unit_x / 16;
  }
}

// ------------------------------------------------------------ roles

struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t slots) {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

template <class C>
__device__ void produce(const RoutedParams& p, const Groups& g, int tiles, uint32_t base,
                        uint32_t rank, const Ctl& ctl) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const Geometry<C> geo(p);
  const uint32_t full0 = base + C::kBarsOff, empty0 = full0 + 8 * C::kSlots;
  const uint32_t lead0 = map_shared_to_rank(full0, 0);
  const uint64_t pol_w = make_l2_policy(p.policy_w), pol_x = make_l2_policy(p.policy_x);
  int begins = 0;
  if constexpr (C::KIND == kLora) begins = p.shard_st_begin[lane <= kMaxShards ? lane : kMaxShards];
  Ring ring;
  uint32_t issued = 0;
  uint32_t weighed = 0, weighings = 0;   // slots that had adapter stages; the parity of their number
  bool ok = true, waited = C::KIND != kLora;
  Walk walk;
  walk.begin(p, tiles);
  Tile t, tn;
  bool have = walk.step<C>(p, g, t);
  while (ok && have) {
    bool looked = false, have_next = false;
    const int half = t.n / 2;
    const int w_row = t.col0 + static_cast<int>(rank) * p.cta_cols;
    const int x_row = t.row0 + static_cast<int>(rank) * half;
    const uint32_t bytes = 2 * C::KZ * (128u * p.w_rows + (C::GATHER ? 0u : static_cast<uint32_t>(half) * 128));
    int shard = 0, shard_begin = 0, shard_end = 0;
    AdapterSteps a{};
    if constexpr (C::KIND == kLora) {
      if (waited) a.template begin<C>(p, t);   // its reads come back during the base product
      shard_end = __shfl_sync(0xffffffffu, begins, 1);
      while (shard_end <= t.st) shard_end = __shfl_sync(0xffffffffu, begins, ++shard + 1);
      shard_begin = __shfl_sync(0xffffffffu, begins, shard);
    }
    for (int st = t.st; st < t.st_end; ++st) {
      ok = wait_bounded(empty0 + 8 * ring.slot, ring.phase ^ 1u, ctl, (kRoleProducer << 8) | 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t lead = lead0 + 8 * ring.slot;
      const uint32_t sw = base + ring.slot * geo.stage, sx = sw + C::KZ * geo.w;
      if constexpr (C::KIND == kLora) {
        while (shard_end <= st) {
          shard_begin = shard_end;
          shard_end = __shfl_sync(0xffffffffu, begins, ++shard + 1);
        }
      }
      const int kx = (st - shard_begin) * (C::KZ * BK);
      if (lane == 0) {
        if (rank == 0) {
          arm(full0 + 8 * ring.slot, bytes);
          if constexpr (C::KIND == kLora) sign_many(full0 + 8 * ring.slot, 2 * kPlacers);   // nothing to place
        }
        // A box of all the stage's k-blocks, where no shard ends inside one.
        const bool whole = C::HALF && p.whole_boxes;
        if (whole) {
          copy_3d(sw, &p.tmap_w[shard], lead, 0, w_row, kx / BK, pol_w);
          copy_3d(sx, &p.tmap_x[shard], lead, 0, x_row, kx / BK, pol_x);
        }
#pragma unroll
        for (int j = 0; j < C::KZ; ++j) {
          if (whole) break;
          const uint32_t dw = sw + j * geo.w;
          if constexpr (C::KIND == kLora) {
            copy_2d(dw, &p.tmap_w[shard], lead, kx + j * BK, w_row, pol_w);
            copy_2d(sx + j * geo.x, &p.tmap_x[shard], lead, kx + j * BK, x_row, pol_x);
          } else {
            copy_3d(dw, &p.tmap_w[0], lead, kx + j * BK, w_row, t.group, pol_w);
            if constexpr (C::KIND == kGated)
              copy_3d(dw + geo.w / 2, &p.tmap_w[0], lead, kx + j * BK, p.N + w_row, t.group, pol_w);
            // The map whose boxes are exactly this tile's rows.
            if constexpr (!C::GATHER && C::TOK <= 256)
              copy_2d(sx + j * geo.x, &p.tmap_x[half / 8 - 1], lead, kx + j * BK, x_row, pol_x);
            if constexpr (!C::GATHER && C::TOK > 256) {
              const Halves q(t.n);
              copy_2d(sx + j * geo.x, &p.tmap_x[q.h[0] / 8 - 1], lead, kx + j * BK,
                      t.row0 + static_cast<int>(rank) * q.h[0], pol_x);
              if (q.h[1])
                copy_2d(sx + j * geo.x + q.h[0] * 128, &p.tmap_x[q.h[1] / 8 - 1], lead, kx + j * BK,
                        t.row0 + 2 * q.h[0] + static_cast<int>(rank) * q.h[1], pol_x);
            }
          }
        }
      }
      __syncwarp();
      if (!looked && st - t.st == static_cast<int>(geo.slots) - 1) {   // place the next tile while the ring is full
        have_next = walk.step<C>(p, g, tn);
        looked = true;
      }
      ++issued;
      ring.next(geo.slots);
    }
    if constexpr (C::KIND == kLora) {
      if (!ok) break;
      if (!waited) {
        grid_dependency_wait();
        waited = true;
        a.template begin<C>(p, t);
      }
      const uint32_t unit_bytes = 2u * p.w_rows * p.unit_cols;
      for (int st = a.st; st < a.st_end; ++st) {
        ok = wait_bounded(empty0 + 8 * ring.slot, ring.phase ^ 1u, ctl, (kRoleProducer << 8) | 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int units = a.units_in(st), u0 = st * a.per_stage;
        const uint32_t landed = full0 + C::kLandedOff + 8 * ring.slot;
        if (lane == 0) {
          arm(landed, unit_bytes * units);
          mbar_arrive(full0 + C::kGrantedOff + 8 * ring.slot);
          if (rank == 0) mbar_arrive(full0 + 8 * ring.slot);
        }
        __syncwarp();
        // Each unit's columns of its adapter's B. They complete on this CTA's own
        // barrier, which the placing warps follow.
        for (int u = 0; u < units; ++u) {
          const int id = a.adapter(p, u0 + u);
          if (lane == 0)
            copy_3d(base + ring.slot * geo.stage + u * geo.unit_w, &p.tmap_b, landed,
                    p.units_per_adapter == 2 ? ((u0 + u) & 1) * p.unit_cols : 0, w_row, id, pol_w);
        }
        __syncwarp();
        weighed |= 1u << ring.slot;
        weighings ^= 1u << ring.slot;
        ++issued;
        ring.next(geo.slots);
      }
    }
    if (!looked) have_next = walk.step<C>(p, g, tn);
    t = tn;
    have = have_next;
  }
  // Let the copies issued land before the shared memory goes away, whether this role
  // gave up or another one did: they complete on the leader's barriers, whose MMAs free
  // the slots, and adapter weights on a barrier of their own. (Otherwise they have
  // landed before the epilogue is done.)
  const uint32_t first = issued > geo.slots ? issued - geo.slots : 0;
  for (uint32_t i = first; i < issued; ++i) {
    if (rank == 0)
      wait_drain(full0 + 8 * (i % geo.slots), (i / geo.slots) & 1u, 100000000ull);
    else
      wait_drain(empty0 + 8 * (i % geo.slots), (i / geo.slots) & 1u, 100000000ull);
  }
  if constexpr (C::KIND == kLora)
    for (uint32_t i = 0; i < geo.slots; ++i)
      if ((weighed >> i) & 1u)
        wait_drain(full0 + C::kLandedOff + 8 * i, ((weighings >> i) & 1u) ^ 1u, 100000000ull);
}

// The pair's MMAs (rank 0).
template <class C>
__device__ void multiply(const RoutedParams& p, const Groups& g, int tiles, uint32_t base,
                         uint32_t tmem, const Ctl& ctl) {
  const Geometry<C> geo(p);
  const uint32_t full0 = base + C::kBarsOff, empty0 = full0 + 8 * C::kSlots;
  const uint32_t tfull0 = empty0 + 8 * C::kSlots, tempty0 = tfull0 + 16, drain = tempty0 + 16;
  Ring ring;
  uint32_t local = 0;
  bool ok = true, issued = false, waited = C::KIND != kLora;
  Walk walk;
  walk.begin(p, tiles);
  Tile t, tn;
  bool have = walk.step<C>(p, g, t);
  for (; ok && have; ++local) {
    const uint32_t acc = local % C::kAccs;
    ok = wait_bounded(tempty0 + 8 * acc, ((local / C::kAccs) & 1u) ^ 1u, ctl, (kRoleMma << 8) | 1);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    tc_fence_after_sync();
    const uint32_t d = tmem + acc * C::TOK;
    const Halves q(t.n);
    const uint32_t idesc = make_idesc(2 * C::kRows, static_cast<uint32_t>(C::TOK > 256 ? 2 * q.h[0] : t.n));
    const uint32_t idesc2 = make_idesc(2 * C::kRows, static_cast<uint32_t>(2 * q.h[1]));
    bool looked = false, have_next = false;
    AdapterSteps a{};
    if constexpr (C::KIND == kLora)
      if (waited) a.template begin<C>(p, t);
    for (int st = t.st; st < t.st_end; ++st) {
      ok = wait_bounded(full0 + 8 * ring.slot, ring.phase, ctl, (kRoleMma << 8) | 2);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after_sync();
      const uint32_t sw = base + ring.slot * geo.stage, sx = sw + C::KZ * geo.w;
#pragma unroll
      for (int j = 0; j < C::KZ; ++j) {
        mma4_bf16_pair(d, smem_desc_sw128(sw + j * geo.w), smem_desc_sw128(sx + j * geo.x), idesc,
                       (st > t.st || j > 0) ? 1u : 0u);
        if constexpr (C::TOK > 256)
          if (q.h[1])
            mma4_bf16_pair(d + 2 * q.h[0], smem_desc_sw128(sw + j * geo.w),
                           smem_desc_sw128(sx + j * geo.x + q.h[0] * 128), idesc2,
                           (st > t.st || j > 0) ? 1u : 0u);
      }
      issued = true;
      mma_commit_pair(empty0 + 8 * ring.slot, 0x3);
      ring.next(geo.slots);
      if (!looked) {   // place the next tile while this one's first stage runs
        have_next = walk.step<C>(p, g, tn);
        looked = true;
      }
    }
    if constexpr (C::KIND == kLora) {
      if (!ok) break;
      if (!waited) {
        grid_dependency_wait();
        waited = true;
        a.template begin<C>(p, t);
      }
      for (int st = a.st; st < a.st_end; ++st) {
        ok = wait_bounded(full0 + 8 * ring.slot, ring.phase, ctl, (kRoleMma << 8) | 2);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t sw = base + ring.slot * geo.stage, sx = sw + C::KZ * geo.w;
        const int units = a.units_in(st);
        // The commit below is by the same thread.
        if (elected()) {
          if (p.unit_cols == 16)
            multiply_units<16, C>(geo, d, sw, sx, idesc, units);
          else if (p.unit_cols == 32)
            multiply_units<32, C>(geo, d, sw, sx, idesc, units);
          else
            multiply_units<64, C>(geo, d, sw, sx, idesc, units);
        }
        __syncwarp();
        issued = true;
        mma_commit_pair(empty0 + 8 * ring.slot, 0x3);
        ring.next(geo.slots);
      }
    }
    if (!ok) break;
    mma_commit_pair(tfull0 + 8 * acc, 0x3);
    if (!looked) have_next = walk.step<C>(p, g, tn);
    t = tn;
    have = have_next;
  }
  // No MMA may be in flight when the accumulators go away, whichever role gave up.
  if (issued) {
    mma_commit_pair(drain, 0x1);
    wait_drain(drain, 0, 100000000ull);
  }
}

// Gathered rows. TMA's four-row gathers cost about 30 ns each, whatever their
// size, 32 of them per k-block at 256 tokens: four times the MMAs' time. So four
// warps copy the rows, 16 bytes per thread and copy, eight threads to a row's 128
// bytes of a k-block, into the 128-byte swizzle that TMA would write.
template <class C>
__device__ void gather_rows(const RoutedParams& p, const Groups& g, int tiles, uint32_t base,
                            uint32_t rank, const Ctl& ctl) {
  constexpr int kPasses = (C::TOK / 2 + 15) / 16;   // 16 rows a pass
  const int tid = static_cast<int>(threadIdx.x) - 64 - kEpi;
  const int chunk = tid & 7, row0 = tid >> 3;
  const Geometry<C> geo(p);
  const uint32_t full0 = base + C::kBarsOff, empty0 = full0 + 8 * C::kSlots;
  const uint32_t dst0 = static_cast<uint32_t>(row0 * 128 + ((chunk ^ (row0 & 7)) << 4));
  const int K = p.K;
  Ring ring;
  bool ok = true;
  Walk walk;
  walk.begin(p, tiles);
  Tile t, tn;
  // This CTA's rows of a tile; the MMA's rows past them hold whatever is there
  // (columns that are never stored).
  auto rows_of = [&](const Tile& q) {
    return min(q.n / 2, q.rows - static_cast<int>(rank) * (q.n / 2));
  };
  // Rows of X that this thread copies.
  int at[kPasses], next[kPasses];
  auto look = [&](const Tile& q, int (&r)[kPasses]) {
    const int first = q.row0 + static_cast<int>(rank) * (q.n / 2), rows = rows_of(q);
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      r[i] = row0 + 16 * i < rows ? p.rows[first + row0 + 16 * i] : -1;
  };
  bool have = walk.step<C>(p, g, t);
  if (have) look(t, at);
  while (ok && have) {
    const int rows = rows_of(t);
    const uint16_t* src[kPasses];
    uint32_t real = 0;   // an index outside X: zeros
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const bool in = at[i] >= 0 && at[i] < p.T;
      real |= in ? 1u << i : 0u;
      src[i] = p.x + static_cast<size_t>(in ? at[i] : 0) * K + 8 * chunk;
    }
    bool looked = false, have_next = false;
    for (int st = t.st; st < t.st_end; ++st) {
      ok = wait_bounded(empty0 + 8 * ring.slot, ring.phase ^ 1u, ctl, (kRolePlacer << 8) | 3);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t sx = base + ring.slot * geo.stage + C::KZ * geo.w + dst0;
#pragma unroll
      for (int j = 0; j < C::KZ; ++j) {
        const int k0 = (st * C::KZ + j) * BK;
        const bool in_k = k0 + 8 * chunk < K;
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
          if (row0 + 16 * i < rows)
            copy_16(sx + j * geo.x + i * 2048, src[i] + (in_k ? k0 : 0), in_k && ((real >> i) & 1u));
      }
      sign_copies(full0 + C::kLandedOff + 8 * ring.slot);
      ring.next(geo.slots);
      if (!looked) {
        have_next = walk.step<C>(p, g, tn);
        if (have_next) look(tn, next);
        looked = true;
      }
    }
    if (!ok) break;
    t = tn;
    have = have_next;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) at[i] = next[i];
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Signs the gathered rows on the leader's full barrier: when the copies of a
// stage have landed, they are made visible to the tensor cores' reads.
template <class C>
__device__ void sign_rows(const RoutedParams& p, int tiles, uint32_t base, const Ctl& ctl) {
  const Geometry<C> geo(p);
  const uint32_t full0 = base + C::kBarsOff, landed0 = full0 + C::kLandedOff;
  const uint32_t lead0 = map_shared_to_rank(full0, 0);
  Ring ring;
  Walk walk;
  walk.begin(p, tiles);
  uint32_t stages = walk.cut >= 0 ? walk.bound(walk.piece + 1) - walk.bound(walk.piece) : 0;
  for (int id = walk.next; id < walk.whole; id += walk.G) stages += walk.S;
  for (; stages > 0; --stages) {
    bool ok = wait_bounded(landed0 + 8 * ring.slot, ring.phase, ctl, (kRolePlacer << 8) | 4);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    if ((threadIdx.x & 31) == 0) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      sign_pair(lead0 + 8 * ring.slot);
    }
    __syncwarp();
    ring.next(geo.slots);
  }
}

// One adapter stage's rows: this lane's row `v` (COLS columns, the adapter `id`)
// in the units of that adapter, zeros in the others.
template <int COLS, class C>
__device__ __forceinline__ void place_stage(const RoutedParams& p, AdapterSteps& a, uint32_t unit_x, uint32_t sx, int st,
                                            int id, int who, int row, int ways, int half,
                                            const uint4 (&v)[kMaxRank / 8]) {
  constexpr uint32_t kMask = COLS == 64 ? 7 : COLS == 32 ? 3 : 1;
  const int units = a.units_in(st), u0 = st * a.per_stage;
  const uint32_t at_row = static_cast<uint32_t>(row) * COLS * 2;
#pragma unroll 2
  for (int u = who * ways / (32 * kPlacers); u < units; u += ways) {
    const bool hit = a.adapter(p, u0 + u) == id;
    const bool upper = COLS == 64 && p.units_per_adapter == 2 && ((u0 + u) & 1);   // columns 64..127
    if (row < half) {
      const uint32_t dst = sx + u * unit_x;
#pragma unroll
      for (int c = 0; c < COLS / 8; ++c) {
        const uint4 w = COLS == 64 && upper ? v[8 + c] : v[c];
        uint32_t off = at_row + 16u * c;
        off ^= ((off >> 7) & kMask) << 4;   // the copies' swizzle over 2 * COLS bytes
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + off), "r"(hit ? w.x : 0u),
                     "r"(hit ? w.y : 0u), "r"(hit ? w.z : 0u), "r"(hit ? w.w : 0u)
                     : "memory");
      }
    }
  }
}

// bf16 pairs: x * 0 + sum stays 0 for finite x and turns NaN for the others.
__device__ __forceinline__ void add_zeros(uint32_t& sum, const uint4& w) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w.x), "r"(0u));
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w.y), "r"(0u));
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w.z), "r"(0u));
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(w.w), "r"(0u));
}

// A masked row times an infinite or NaN weight would be NaN, so the tile's
// adapters (this CTA's weight rows of them) are looked over while the base
// product streams. That also brings them into L2 for the copies to come. Thread
// `who` of `threads`; true if a weight that it read is not finite.
template <class C>
__device__ __forceinline__ bool look_over(const RoutedParams& p, const Tile& t, const AdapterSteps& steps,
                                          uint32_t rank, int who, int threads) {
  const int count = steps.units / p.units_per_adapter, lane = who & 31;
  const bool self = C::SELF && p.self_rows;
  const int col = t.col0 + static_cast<int>(rank) * p.cta_cols;
  const int vecs = max(min(p.cta_cols, p.N - col), 0) * p.rank / 8;   // 16-byte vectors, contiguous
  uint32_t sum[4] = {0, 0, 0, 0};
  for (int i = who >> 5; i < count; i += threads >> 5) {
    const int id = self ? __shfl_sync(0xffffffffu, steps.held, i) : __ldcg(steps.list + 1 + i);
    const uint4* w = reinterpret_cast<const uint4*>(p.b + (static_cast<size_t>(id) * p.N + col) * p.rank);
    for (int at = lane; at < vecs; at += 4 * 32) {
      uint4 x[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] = at + 32 * q < vecs ? __ldcg(w + at + 32 * q) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) add_zeros(sum[q], x[q]);
    }
  }
  return ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) != 0;
}

// The weights of a marked tile's stage that are not finite become 1 or -1, by their
// sign (the epilogue adds their products to the rows that have the adapter). A masked
// row's product with those is 0, a finite row's is lost in the infinity or NaN that is
// added, and an infinite row's is the infinity that it is due; with 0 it would be NaN.
template <class C>
__device__ __noinline__ void take_out(const RoutedParams& p, uint32_t sw, int units, int who) {
  const uint32_t unit = Geometry<C>(p).unit_w, bytes = 2u * p.w_rows * p.unit_cols;
  for (int u = 0; u < units; ++u)
    for (uint32_t at = 16u * who; at < bytes; at += 16 * 32 * kPlacers) {
      uint32_t w[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(sw + u * unit + at)
                   : "memory");
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // Bits 15 and 31: an exponent of all ones in the half below.
        const uint32_t odd = ((w[j] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        const uint32_t taken = (odd >> 15) * 0xffffu;
        w[j] = (w[j] & ~taken) | (((w[j] & 0x80008000u) | 0x3f803f80u) & taken);
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sw + u * unit + at), "r"(w[0]),
                   "r"(w[1]), "r"(w[2]), "r"(w[3])
                   : "memory");
    }
}

// One row or two: the two teams compute the low-rank rows themselves, in
// every CTA that holds them, from L2 and while the weights stream, and no kernel
// runs before the product. The 8 warps take every 8th chunk of 256 k of all columns
// (16 rows of A in flight per warp); part[w][m][j] is warp w's sum.
__device__ __forceinline__ void self_rows(const RoutedParams& p, const SelfTable& s, float* part, int who) {
  const int lane = who & 31, warp = who >> 5;
  for (int m = 0; m < p.M; ++m) {
    const int id = p.adapter[m];
    if (id < 0 || id >= p.L) continue;
    for (int j0 = 0; j0 < p.rank_pad; j0 += 16) {
      float sum[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) sum[j] = 0.f;
      int at = 8 * lane + 256 * warp;   // this lane's k in shard r
      for (int r = 0; r < p.R;) {
        const int K = s.k[r], chunks = (K + 255) >> 8;
        if (at >= chunks * 256) {
          at -= chunks * 256;
          ++r;
          continue;
        }
        if (at < K) {
          const uint4 u = __ldcg(reinterpret_cast<const uint4*>(s.x[r] + static_cast<size_t>(m) * K + at));
          const uint16_t* a = s.a[r] + (static_cast<size_t>(id) * p.rank + j0) * K + at;
          uint4 v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[j] = j0 + j < p.rank ? __ldcg(reinterpret_cast<const uint4*>(a + static_cast<size_t>(j) * K))
                                   : make_uint4(0, 0, 0, 0);
          const uint32_t xw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t aw[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              sum[j] = fmaf(__uint_as_float(xw[i] << 16), __uint_as_float(aw[i] << 16), sum[j]);
              sum[j] = fmaf(__uint_as_float(xw[i] & 0xffff0000u), __uint_as_float(aw[i] & 0xffff0000u), sum[j]);
            }
          }
        }
        __syncwarp();
        at += 8 * 256;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
        if (lane == j) part[warp * kSelfElements + m * p.rank_pad + j0 + j] = sum[j];
      }
    }
  }
}

// Element (m, j) of the rows that self_rows summed, as bf16 bits.
__device__ __forceinline__ uint32_t self_low(const RoutedParams& p, const float* part, int m, int j, float scale) {
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) sum += part[w * kSelfElements + m * p.rank_pad + j];
  return __bfloat16_as_ushort(__float2bfloat16(sum * scale));
}

// The adapter stages of one tile, for one team of four warps (thread `i` of
// them). The threads are the rows of this CTA's tokens, or, with at most 64 or 32
// rows, two or four times the rows, on alternate adapters. The rows are placed
// once the producer grants the slot, while its adapter weights are on their way;
// every warp signs the stage on the leader's full barrier when they have landed.
// The base product's stages pass by, and with two teams every other stage: a wait
// by parity is safe all the same. A slot is not granted again before its stage is
// signed, so the wait is never late; the producer grants in order, at least the
// stage S before this one before the team's last one (S >= 3), so it is never a
// phase early; and a granted slot's earlier weights have landed.
struct Placing {
  Ring ring;
  uint32_t phases = 0;   // bit s: phase of slot s's granted and landed barriers
  uint32_t count = 0;    // adapter stages so far: the teams take turns
  const SelfTable* table;   // shared memory, for self_rows
  float* part;              // its sums
};
template <int TEAM, class C>
__device__ bool place_tile(const RoutedParams& p, const Tile& t, uint32_t local, Placing& q, int i,
                           uint32_t base, uint32_t rank, volatile int* marks, const Ctl& ctl) {
  const int lane = i & 31;
  const Geometry<C> geo(p);
  const uint32_t full0 = base + C::kBarsOff;
  const uint32_t lead0 = map_shared_to_rank(full0, 0);
  q.ring.slot = (q.ring.slot + static_cast<uint32_t>(t.st_end - t.st)) % geo.slots;
  AdapterSteps a{};
  a.template begin<C>(p, t);
  const int half = t.n / 2, ways = half <= 32 ? 4 : half <= 64 ? 2 : 1;
  const int row = i & (32 * kPlacers / ways - 1), m = t.row0 + static_cast<int>(rank) * half + row;
  int id = -1;
  uint4 v[kMaxRank / 8];
  if (row < half && m < p.M) id = p.adapter[m];
  if (id >= p.L) id = -1;   // no adapter of the list is negative
  const bool self = C::SELF && p.self_rows;
  // Columns from the rank to its padding are zeros here, whatever the low-rank rows
  // hold there: an infinite activation times the padding of A is NaN.
  if (self) {
    // Rank 0 places every row (half a tile's tokens are 8 at least), but either CTA's
    // epilogue may need them (add_unbounded).
    if (local == 0) self_rows(p, *q.table, q.part, i + TEAM * 32 * kPlacers);
  } else {
#pragma unroll
    for (int c = 0; c < kMaxRank / 8; ++c)
      v[c] = id >= 0 && 8 * c < p.rank
                 ? __ldcg(reinterpret_cast<const uint4*>(p.low + static_cast<size_t>(m) * p.rank_pad) + c)
                 : make_uint4(0, 0, 0, 0);
  }
  // What the teams' warps saw, of this tile and the next two.
  volatile int* seen = marks + kMarks;
  const bool odd = look_over<C>(p, t, a, rank, i + TEAM * 32 * kPlacers, 32 * kPlacers * C::kTeams);
  if (odd) seen[local % 3] = 1;
  if (TEAM == 0 && i == 0) seen[(local + 1) % 3] = 0;   // read by all two tiles ago
  __syncwarp();
  if (lane == 0) mbar_arrive(full0 + C::kLookedOff);
  bool all = wait_bounded(full0 + C::kLookedOff, local & 1u, ctl, (kRolePlacer << 8) | 5);
  if (!__all_sync(0xffffffffu, all)) return false;
  const bool marked = seen[local % 3] != 0;
  if (self) {
    const float scale = id >= 0 && p.scale ? p.scale[id] : 1.f;
#pragma unroll
    for (int c = 0; c < kMaxRank / 8; ++c) {
      uint32_t w[4] = {0, 0, 0, 0};
      if (8 * c < kSelfElements && id >= 0 && 8 * c < p.rank) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = self_low(p, q.part, m, 8 * c + 2 * i, scale) |
                 self_low(p, q.part, m, 8 * c + 2 * i + 1, scale) << 16;
      }
      v[c] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  for (int st = a.st; st < a.st_end; ++st, ++q.count) {
    if (q.count % C::kTeams == TEAM) {
      const uint32_t phase = (q.phases >> q.ring.slot) & 1u;
      bool ok = wait_bounded(full0 + C::kGrantedOff + 8 * q.ring.slot, phase, ctl, (kRolePlacer << 8) | 1);
      if (!__all_sync(0xffffffffu, ok)) return false;
      // (The producer is few tiles past the epilogue here: kMarks are enough.)
      if (marked && i == 0) marks[local % kMarks] = 1;
      const uint32_t sw = base + q.ring.slot * geo.stage, sx = sw + C::KZ * geo.w;
      if (p.unit_cols == 16)
        place_stage<16, C>(p, a, geo.unit_x, sx, st, id, i, row, ways, half, v);
      else if (p.unit_cols == 32)
        place_stage<32, C>(p, a, geo.unit_x, sx, st, id, i, row, ways, half, v);
      else
        place_stage<64, C>(p, a, geo.unit_x, sx, st, id, i, row, ways, half, v);
      ok = wait_bounded(full0 + C::kLandedOff + 8 * q.ring.slot, phase, ctl, (kRolePlacer << 8) | 2);
      if (!__all_sync(0xffffffffu, ok)) return false;
      if (marked) take_out<C>(p, sw, a.units_in(st), i);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) sign_pair(lead0 + 8 * q.ring.slot);
    }
    q.phases ^= 1u << q.ring.slot;
    q.ring.next(geo.slots);
  }
  return true;
}

// The placing warps: team 0 of every tile. With half tiles, the epilogue's warps,
// which then wait for the accumulator, are team 1.
template <class C>
__device__ void place_rows(const RoutedParams& p, const Groups& g, int tiles, uint32_t base,
                           uint32_t rank, Placing q, volatile int* marks, const Ctl& ctl) {
  const int i = static_cast<int>(threadIdx.x) - 64 - kEpi;
  Walk walk;
  walk.begin(p, tiles);
  Tile t;
  grid_dependency_wait();
  for (uint32_t local = 0; walk.step<C>(p, g, t); ++local)
    if (!place_tile<0, C>(p, t, local, q, i, base, rank, marks, ctl)) break;
}

// The products of adapter weights that are not finite, which the placing warps
// took out of the tile, added to a warp's fragments v of 32 tokens x 32 columns
// (`valid` rows from `row` on, columns from `col` to `end`), for the adapters of
// this piece.
template <class C>
__device__ __noinline__ void add_unbounded(const RoutedParams& p, const float* part, const Tile& t, int row,
                                           int valid, int col, int end, float (&v)[32]) {
  AdapterSteps a{};
  a.template begin<C>(p, t);
  const int u0 = a.st * a.per_stage, u1 = min(a.st_end * a.per_stage, a.units);
  const int lane = static_cast<int>(threadIdx.x) & 31;
#pragma unroll 1
  for (int i = 0; i < 32; ++i) {
    const int token = 8 * ((i >> 2) & 3) + 2 * (lane & 3) + (i & 1);
    const int n = col + 16 * (i >> 4) + 8 * ((i >> 1) & 1) + (lane >> 2);
    const int m = row + token;
    const int id = token < valid && n < end ? p.adapter[m] : -1;
    if (id < 0 || id >= p.L) continue;
    // Its place in the tile's list, which has every row's adapter (computed rows:
    // the adapters that appear first in earlier rows).
    int at = 0;
    if (C::SELF && p.self_rows) {
      for (int i0 = 0; p.adapter[i0] != id; ++i0) {
        const int other = p.adapter[i0];
        bool first = other >= 0 && other < p.L;
        for (int i1 = 0; i1 < i0; ++i1) first = first && p.adapter[i1] != other;
        at += first;
      }
    } else {
      while (__ldcg(a.list + 1 + at) != id) ++at;
    }
    float sum = 0.f;
    bool any = false;
    for (int k = 0; k < p.rank; ++k) {
      const int u = at * p.units_per_adapter + k / p.unit_cols;
      if (u < u0 || u >= u1) continue;
      const uint32_t w = p.b[(static_cast<size_t>(id) * p.N + n) * p.rank + k];
      if ((w & 0x7f80u) != 0x7f80u) continue;
      const uint32_t x = C::SELF && p.self_rows
                             ? self_low(p, part, m, k, p.scale ? p.scale[id] : 1.f)
                             : __ldcg(p.low + static_cast<size_t>(m) * p.rank_pad + k);
      sum += __uint_as_float(w << 16) * __uint_as_float(x << 16);
      any = true;
    }
    if (any) v[i] += sum;
  }
}

// Stores GROUPS x 8 tokens x 32 columns, packed as 8 x 8 matrices (w[g][b]: tokens
// 8 g .., columns 8 b ..), through the warp's 2 KB of staging: a token's 64 bytes
// are four 16-byte chunks, turned by the token so that neither the transposed
// stores nor the reads meet in a bank.
template <int GROUPS>
__device__ __forceinline__ void store_tokens(uint16_t* y, int N, int row, int valid, int col, int end,
                                             uint32_t staging, const uint32_t (&w)[GROUPS][4]) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const uint32_t in = staging + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) store_transposed(in + g * 512, w[g][0], w[g][1], w[g][2], w[g][3]);
  __syncwarp();
  const int r = lane >> 2, c = lane & 3;
  const uint32_t out = staging + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  uint16_t* at = y + static_cast<size_t>(row + r) * N + col + 8 * c;
  const bool in_cols = col + 8 * c < end;
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(out + g * 512)
                 : "memory");
    if (in_cols && r + 8 * g < valid) *reinterpret_cast<uint4*>(at + static_cast<size_t>(8 * g) * N) = v;
  }
  __syncwarp();   // read before the next chunk is written
}

template <class C>
__device__ void finish(const RoutedParams& p, const Groups& g, int tiles, uint32_t base,
                       uint8_t* base_ptr, uint32_t tmem, uint32_t rank, volatile int* last_flag,
                       Placing placing, volatile int* marks, const Ctl& ctl) {
  const uint32_t tfull0 = base + C::kBarsOff + 16 * C::kSlots, tempty0 = tfull0 + 16;
  const int et = static_cast<int>(threadIdx.x) - 64;
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int quad = (static_cast<int>(threadIdx.x) >> 5) & 3;   // TMEM lanes this warp may read
  // This warp's first weight row. The accumulator of a pair MMA with 128 rows holds
  // a CTA's 64 rows twice over: lanes 64..127 hold the second half of the tokens.
  const int wrow = (C::HALF ? quad & 1 : quad) * 32;
  const uint32_t lead_tempty = map_shared_to_rank(tempty0, 0);
  float* swap = reinterpret_cast<float*>(base_ptr + C::kStagingOff);
  const uint32_t staging = base + C::kStagingOff + quad * 2048;
  uint32_t local = 0;
  Walk walk;
  walk.begin(p, tiles);
  Tile t, tn;
  bool have = walk.step<C>(p, g, tn);
  for (; have; ++local) {
    t = tn;
    have = walk.step<C>(p, g, tn);   // while this tile's accumulator fills
    const uint32_t acc = local % C::kAccs;
    bool placed = true;
    if constexpr (C::KIND == kLora && C::HALF) {
      if (local == 0) grid_dependency_wait();
      placed = place_tile<1, C>(p, t, local, placing, et, base, rank, marks, ctl);
    }
    const bool ok = placed && wait_bounded(tfull0 + 8 * acc, (local / C::kAccs) & 1u, ctl, (kRoleEpilogue << 8) | 1);
    if (!epilogue_bar_and(ok)) break;
    tc_fence_after_sync();
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * C::TOK;
    const int tok0 = C::HALF ? (quad >> 1) * (t.n / 2) : 0;   // this thread's first token
    const int mine = C::HALF ? max(min(t.rows - tok0, t.n / 2), 0) : t.rows;
    const int chunks = (mine + 31) >> 5;
    const int col0 = t.col0 + static_cast<int>(rank) * p.cta_cols;
    const int col_end = min(p.N, col0 + p.cta_cols);
    bool marked = false;
    if constexpr (C::KIND == kLora) {
      marked = marks[local % kMarks] != 0;
      epilogue_bar_sync();
      if (marked && et == 0) marks[local % kMarks] = 0;
    }

    // This warp's fragments of 32 tokens from token 32 * c on: v[16 h + 4 g + e] is
    // token 8 g + 2 (lane % 4) + e % 2, column 16 h + 8 (e / 2) + lane / 4.
    auto load = [&](int c, float (&v)[32]) {
      uint32_t r[32];
      tmem_ld_16x32(taddr + 32 * c, r);
      tmem_ld_16x32(taddr + (16u << 16) + 32 * c, r + 16);
      tmem_ld_wait(r);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
      if constexpr (C::KIND == kLora) {
        if (marked)
          add_unbounded<C>(p, placing.part, t, t.row0 + tok0 + 32 * c, mine - 32 * c, col0 + wrow, col_end, v);
      }
    };
    auto release = [&]() {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) sign_pair(lead_tempty + 8 * acc);
    };
    auto emit = [&](int c, const float (&v)[32]) {
      const int row = t.row0 + tok0 + 32 * c, valid = mine - 32 * c;
      if constexpr (C::KIND != kGated) {
        uint32_t w[4][4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int j = 16 * (b >> 1) + 4 * g + 2 * (b & 1);
            w[g][b] = pack_bf16x2(__float_as_uint(v[j]), __float_as_uint(v[j + 1]));
          }
        store_tokens<4>(p.y, p.N, row, valid, col0 + wrow, col_end, staging, w);
      } else {
        // Quads 0 and 1 hold the gates, 2 and 3 the ups, of the same columns, in
        // the same layout. Each pair of warps swaps halves through their staging:
        // the gate's warp finishes tokens 0..15, the up's warp 16..31.
        const int pair = quad & 1, up = quad >> 1;
        float* own = swap + quad * 512;
        const float* theirs = swap + (quad ^ 2) * 512;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int i = 16 * (j >> 3) + (j & 7);   // of the first two token groups
          own[j * 32 + lane] = up ? v[i] : v[i + 8];
        }
        named_sync(2 + pair, 64);
        uint32_t w[2][4];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            float out[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int j = 8 * (b >> 1) + 4 * g + 2 * (b & 1) + e, i = 16 * (j >> 3) + (j & 7);
              const float other = theirs[j * 32 + lane];
              const float gate = up ? other : v[i], mul = up ? v[i + 8] : other;
              out[e] = gate / (1.f + __expf(-gate)) * mul;
            }
            w[g][b] = pack_bf16x2(__float_as_uint(out[0]), __float_as_uint(out[1]));
          }
        named_sync(2 + pair, 64);   // read by the other warp: the staging is free
        store_tokens<2>(p.y, p.N, row + 16 * up, valid - 16 * up, col0 + pair * 32, col_end, staging, w);
      }
    };

    if (t.npieces == 1) {
      for (int c = 0; c < chunks; ++c) {
        float v[32];
        load(c, v);
        emit(c, v);
      }
      release();
      continue;
    }

    // A piece of a cut tile: publish the fp32 partial (each thread its fragments) and
    // count it; the piece that finds all others counted sums them in k order.
    constexpr size_t kSlot = static_cast<size_t>(C::TOK) * C::kRows;
    float4* slot = reinterpret_cast<float4*>(p.partials + (static_cast<size_t>(t.slot + t.piece) * 2 + rank) * kSlot);
    for (int c = 0; c < chunks; ++c) {
      float v[32];
      load(c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        __stcg(slot + (8 * c + j) * kEpi + et,
               make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
    }
    release();
    __threadfence();
    epilogue_bar_sync();
    uint32_t* counter = p.counters + 2 * t.cut + rank;
    if (et == 0) *last_flag = atomicAdd(counter, 1u) == static_cast<uint32_t>(t.npieces - 1);
    epilogue_bar_sync();
    const bool last = *last_flag != 0;
    epilogue_bar_sync();   // read by all before the next tile writes it
    if (!last) continue;
    __threadfence();
    const float4* first = reinterpret_cast<const float4*>(p.partials + (static_cast<size_t>(t.slot) * 2 + rank) * kSlot);
    for (int c = 0; c < chunks; ++c) {
      float v[32] = {};
      auto add = [&](const float4 (&f)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[4 * j] += f[j].x;
          v[4 * j + 1] += f[j].y;
          v[4 * j + 2] += f[j].z;
          v[4 * j + 3] += f[j].w;
        }
      };
      auto read = [&](int s, float4 (&f)[8]) {
        const float4* src = first + static_cast<size_t>(s) * (2 * kSlot / 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __ldcg(src + (8 * c + j) * kEpi + et);
      };
      // In k order (0 + x is x, but for the sign of a zero); two pieces' reads in
      // flight where there are registers for them.
      int s = 0;
      if constexpr (C::KIND != kLora) {
        for (; s + 1 < t.npieces; s += 2) {
          float4 f[8], h[8];
          read(s, f);
          read(s + 1, h);
          add(f);
          add(h);
        }
      }
      for (; s < t.npieces; ++s) {
        float4 f[8];
        read(s, f);
        add(f);
      }
      emit(c, v);
    }
    if (et == 0) atomicExch(counter, 0u);   // ready for the next call
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) gsr_routed_kernel(const __grid_constant__ RoutedParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base_ptr + C::kMiscOff + 4);
  volatile int* last_flag = reinterpret_cast<volatile int*>(base_ptr + C::kMiscOff + 8);
  volatile int* marks = reinterpret_cast<volatile int*>(base_ptr + C::kMiscOff + 16);
  const int warp = static_cast<int>(threadIdx.x) >> 5;
  const uint32_t rank = cluster_rank();
  const uint32_t bars = base + C::kBarsOff;
  Placing placing{};
  if constexpr (C::SELF) {
    SelfTable* table = reinterpret_cast<SelfTable*>(base_ptr + C::kGroupsOff);
    placing.table = table;
    placing.part = reinterpret_cast<float*>(table + 1);
    if (p.self_rows && threadIdx.x >= 64 && threadIdx.x < 64 + kMaxShards) {
      const int r = static_cast<int>(threadIdx.x) - 64;
      table->x[r] = p.x_r[r];
      table->a[r] = p.a_r[r];
      table->k[r] = p.k_r[r];
    }
  }
  if (warp == 1) {
    // Every descriptor that the copies may use, one per lane: each is a memory access
    // otherwise, where a shard begins or a tile has another width.
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int maps = C::KIND == kLora ? p.R : min(C::TOK, 256) / 16;
    if (lane < (C::KIND == kLora ? maps : 1)) fetch_descriptor(&p.tmap_w[lane]);
    if (!C::GATHER && lane < maps) fetch_descriptor(&p.tmap_x[lane]);
    if (C::KIND == kLora && lane == 0) fetch_descriptor(&p.tmap_b);
    __syncwarp();
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < static_cast<int>(C::kSlots); ++i) {
      mbar_init(bars + 8 * i, C::kSigns);
      mbar_init(bars + 8 * (C::kSlots + i), 1);                   // empty: the MMAs' commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 16 * C::kSlots + 8 * i, 1);                // accumulator full
      mbar_init(bars + 16 * C::kSlots + 16 + 8 * i, 8);           // empty: the pair's epilogue warps
    }
    mbar_init(bars + 16 * C::kSlots + 32, 1);
    if constexpr (C::KIND == kLora || C::GATHER)
      for (int i = 0; i < static_cast<int>(C::kSlots); ++i)
        mbar_init(bars + C::kLandedOff + 8 * i, C::GATHER ? 32 * kPlacers : 1);
    if constexpr (C::KIND == kLora)
      for (int i = 0; i < static_cast<int>(C::kSlots); ++i) mbar_init(bars + C::kGrantedOff + 8 * i, 1);
    if constexpr (C::KIND == kLora) {
      mbar_init(bars + C::kLookedOff, kPlacers * C::kTeams);
      for (int i = 0; i < kMarks + 3; ++i) marks[i] = 0;
    }
    *abort_flag = 0;
    *last_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_barrier();
  tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

  // Programmatic dependent launch. The grouped kinds wait here for the previous
  // kernel, and kLora where it computes the low-rank rows itself. Else kLora follows
  // the low-rank kernel, which lets it start only once everything before that kernel
  // has completed: X and W may be read at once, and the roles wait before they read
  // what the low-rank kernel writes.
  Groups g{};
  int tiles;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (C::KIND == kLora) {
    if (C::SELF && p.self_rows) grid_dependency_wait();
    tiles = p.m_tiles * p.n_tiles;
  } else {
    grid_dependency_wait();
    int* mem = reinterpret_cast<int*>(base_ptr + C::kGroupsOff);
    g.row = mem;
    g.count = mem + kMaxGroups;
    g.tile = mem + 2 * kMaxGroups;
    tiles = count_groups<C>(p, g, mem + 3 * kMaxGroups + 1) * p.n_tiles;
  }

  Ctl ctl{abort_flag, p.status, p.timeout_ns};
  if (warp == 0) {
    produce<C>(p, g, tiles, base, rank, ctl);
  } else if (warp == 1) {
    if (rank == 0) multiply<C>(p, g, tiles, base, tmem, ctl);
  } else if (warp < 6) {
    finish<C>(p, g, tiles, base, base_ptr, tmem, rank, last_flag, placing, marks, ctl);
  } else if constexpr (C::KIND == kLora) {
    place_rows<C>(p, g, tiles, base, rank, placing, marks, ctl);
  } else if constexpr (C::GATHER) {
    if (warp < 6 + kPlacers)
      gather_rows<C>(p, g, tiles, base, rank, ctl);
    else
      sign_rows<C>(p, tiles, base, ctl);
  }
  __syncwarp();
  if constexpr (C::KIND == kLora) {
    // Every thread, also one without a tile: this grid must not complete before
    // the low-rank kernel has.
    grid_dependency_wait();
  }
  tc_fence_before_sync();
  cluster_barrier();   // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, C::kTmemCols);
  }
}

// Ring depths that fill shared memory.
template <int KIND, bool GATHER, int TOK>
using Instance = Cfg<KIND, GATHER, false, TOK, routed_kblocks(false, TOK),
                     TOK == kRoutedSmall ? 5 : TOK == kRoutedWide ? 3 : 4>;
// Few tokens: tiles of at most 128 weight rows.
template <int TOK>
using HalfInstance = Cfg<kLora, false, true, TOK, routed_kblocks(true, TOK),
                         TOK == kRoutedMid ? 3 : 4>;

template <class C>
cudaError_t set_limit() {
  return cudaFuncSetAttribute(gsr_routed_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(C::kSmem));
}

template <class C>
cudaError_t launch_one(const RoutedParams& p, int ctas, cudaStream_t stream) {
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
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gsr_routed_kernel<C>, p);
}

template <int KIND, bool GATHER>
cudaError_t set_limits() {
  cudaError_t e = set_limit<Instance<KIND, GATHER, kRoutedSmall>>();
  if (e == cudaSuccess) e = set_limit<Instance<KIND, GATHER, kRoutedMid>>();
  if (e == cudaSuccess) e = set_limit<Instance<KIND, GATHER, kRoutedWide>>();
  if constexpr (!GATHER)
    if (e == cudaSuccess) e = set_limit<Instance<KIND, GATHER, kRoutedDouble>>();
  return e;
}

template <int KIND, bool GATHER>
cudaError_t launch_kind(const RoutedParams& p, int tokens, int ctas, cudaStream_t stream) {
  if (tokens == kRoutedSmall) return launch_one<Instance<KIND, GATHER, kRoutedSmall>>(p, ctas, stream);
  if (tokens == kRoutedMid) return launch_one<Instance<KIND, GATHER, kRoutedMid>>(p, ctas, stream);
  if constexpr (!GATHER)
    if (tokens == kRoutedDouble) return launch_one<Instance<KIND, GATHER, kRoutedDouble>>(p, ctas, stream);
  return launch_one<Instance<KIND, GATHER, kRoutedWide>>(p, ctas, stream);
}

}  // namespace

cudaError_t prepare_routed_kernels() {
  cudaError_t e = set_limits<kGrouped, false>();
  if (e == cudaSuccess) e = set_limits<kGrouped, true>();
  if (e == cudaSuccess) e = set_limits<kGated, false>();
  if (e == cudaSuccess) e = set_limits<kGated, true>();
  if (e == cudaSuccess) e = set_limit<Instance<kLora, false, kRoutedWide>>();
  if (e == cudaSuccess) e = set_limit<HalfInstance<kRoutedSmall>>();
  if (e == cudaSuccess) e = set_limit<HalfInstance<kRoutedMid>>();
  if (e == cudaSuccess) e = set_limit<HalfInstance<kRoutedWide>>();
  return e;
}

cudaError_t launch_routed(const RoutedParams& p, int kind, bool gather, bool half, int tokens, int ctas,
                          cudaStream_t stream) {
  if (kind == kLora && !half) return launch_one<Instance<kLora, false, kRoutedWide>>(p, ctas, stream);
  if (kind == kLora)
    return tokens == kRoutedSmall ? launch_one<HalfInstance<kRoutedSmall>>(p, ctas, stream)
           : tokens == kRoutedMid ? launch_one<HalfInstance<kRoutedMid>>(p, ctas, stream)
                                  : launch_one<HalfInstance<kRoutedWide>>(p, ctas, stream);
  if (kind == kGated)
    return gather ? launch_kind<kGated, true>(p, tokens, ctas, stream)
                  : launch_kind<kGated, false>(p, tokens, ctas, stream);
  return gather ? launch_kind<kGrouped, true>(p, tokens, ctas, stream)
                : launch_kind<kGrouped, false>(p, tokens, ctas, stream);
}

}  // namespace gsr
