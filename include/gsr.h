/*
 * gsr.h -- C ABI of the GB300 (sm_103a) shard-reduction GEMM.
 *
 * A BF16 linear projection whose cross-shard reduction is fused into the GEMM,
 * stated for one GPU: the R "ranks" of a tensor-parallel group are R shard
 * buffers in this GPU's memory, and one kernel launch reads them all in place.
 *
 *   gemm_ar  Y   = sum_r X_r . W_r^T                (all-reduce over K-shards)
 *   gemm_rs  Y_s = rows [s*rps, min(M,(s+1)*rps)) of sum_r X_r . W_r^T
 *                  with rps = ceil(M / R)           (reduce-scatter by rows)
 *   gemm_ag  Y   = concat_r(A_r) . W^T              (all-gather of M-shards)
 *   gemm_ar_replicated  the AR sum written into each of R output buffers
 *
 * Sources of the definitions: vLLM PR #53053 summary ("Extend GEMM-RS to
 * GEMM-AR"), implementation breakdown step 1 (one kernel serves RS and AR;
 * AR accepts any M with no padding or input copy; flags handled inside the
 * kernel) and the test's `_reference` (torch.mm(x, weight.T) per rank, then
 * dist.all_reduce, or dist.reduce_scatter_single over rows padded to
 * ceil(M/R)*R); vLLM PR #54151 "[Kimi-K3] AG-GEMM for Sequence Parallelism",
 * Purpose (GEMM over the gathered activation shards).
 *
 * Conventions shared by every call
 *   - Element type: bf16 in and out; products accumulate in fp32; the output
 *     is rounded once, to nearest even.
 *   - Layout: dense row-major, leading dimension = last dimension. Every GEMM
 *     operand is K-major like an nn.Linear weight: X_r is M x K_r, W_r is
 *     N x K_r, A_r is M_r x K, W is N x K. Outputs are rows x N.
 *   - Alignment: every pointer 16-byte aligned; N and every K_r (AR/RS) or K
 *     (AG) a multiple of 8, so that each row starts on a 16-byte boundary.
 *   - Ownership: the caller owns every device buffer (shards, outputs,
 *     workspace) and the stream. The library owns only the plan, a host
 *     object; it allocates no device memory. Host pointer arrays are read
 *     during the call only.
 *   - Streams: calls are stream-ordered and asynchronous. Nothing synchronises
 *     except gemm_shard_check_status. One workspace must not be used by two
 *     calls that may run at the same time.
 *   - Graphs: gemm_ar, gemm_rs and gemm_ag may be recorded in a CUDA graph
 *     (stream capture). A call's tensor maps and kernel parameters are built
 *     on the host when the call is made, so the graph holds that call's
 *     pointers and shapes, and a replay reads the buffers' current contents.
 *     The workspace's split-K counters are back at zero after every launch,
 *     so replays need no re-initialisation. gemm_shard_check_status
 *     synchronises and cannot be captured.
 *   - Errors: argument errors are detected before any launch and return
 *     GSR_ERR_INVALID_VALUE / GSR_ERR_WORKSPACE without touching the GPU. A
 *     failed launch returns GSR_ERR_CUDA. Every wait inside the kernel is
 *     bounded; a wait that runs out records GSR_ERR_TIMEOUT in the workspace
 *     status word, the kernel returns cleanly, and gemm_shard_check_status
 *     reports it. The library never aborts the process and never traps.
 *     gsr_last_error_string() describes the last failure on this thread.
 *   - Logging: with the environment variable GSR_LOG_CONFIG set (to anything
 *     but "0") when the library is first used, every GEMM call that passes
 *     validation and has rows to compute writes one line to stderr before its
 *     launch: the mode, the shape and the kernel configuration it chose (the
 *     fields of gsr_config). Nothing is logged otherwise.
 */
#ifndef GSR_H
#define GSR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream; NULL is the legacy default stream. */
typedef struct CUstream_st *gsr_stream_t;

typedef struct gemm_shard_plan gemm_shard_plan;

typedef enum {
    GSR_OK = 0,
    GSR_ERR_INVALID_VALUE = 1, /* bad pointer, shape, alignment or option      */
    GSR_ERR_UNSUPPORTED = 2,   /* device is not a GB300-class sm_103 part      */
    GSR_ERR_WORKSPACE = 3,     /* workspace missing, misaligned or too small   */
    GSR_ERR_CUDA = 4,          /* a CUDA runtime or driver call failed         */
    GSR_ERR_TIMEOUT = 5        /* a bounded in-kernel wait ran out             */
} gsr_status;

/* Largest number of shards (ranks) one call accepts; the pages' gating allows
 * tensor-parallel sizes 2..16 (PR #53053 summary, model.py gating chain). */
#define GSR_MAX_SHARDS 16

/* Plan options (gemm_shard_plan_set_option). 0 restores the default. */
typedef enum {
    GSR_OPT_SPLIT_K = 1,    /* pieces per output tile: 0 = heuristic, 1..16 forced */
    GSR_OPT_BLOCK_N = 2,    /* output tile width: 0 = heuristic, 128, 192 (CTA
                               pairs only; 256 otherwise) or 256              */
    GSR_OPT_TIMEOUT_NS = 3, /* limit of every in-kernel wait, ns (default 2e9)      */
    GSR_OPT_MAX_CTAS = 4,   /* cap on persistent CTAs: 0 = one per SM               */
    GSR_OPT_RASTER_M = 5,   /* m-tiles per raster group (m runs fastest inside a
                               group): 0 = heuristic, 1..64                         */
    GSR_OPT_L2_HINTS = 6,   /* TMA L2 eviction hints: 0 = heuristic (main kernel:
                               2 where both operands together fit in the L2,
                               else none; small-M kernel: 2), 1 = none,
                               2 = A evict-last / B evict-first,
                               3 = A evict-first / B evict-last                     */
    GSR_OPT_CTA_GROUP = 7,  /* CTAs per MMA tile: 0 = heuristic, 1 = one CTA per
                               128-row tile, 2 = a CTA pair per 256-row tile,
                               4 = two CTA pairs per cluster on two 256-row
                               tiles of the same columns                      */
    GSR_OPT_SCHEDULE = 8,   /* work schedule: 0 = heuristic (uniform while there
                               are fewer single-CTA tiles than SMs; else whole
                               tiles for the full waves and, for a partial last
                               wave, a split tail (5) when it is at most half a
                               wave and its pieces keep at least 60 % of the
                               workers busy, whole tiles when at least 70 % of
                               the workers have one, stream-K (3) otherwise),
                               1 = uniform (every tile cut
                               into the same number of pieces), 2 = stream-K
                               over the last one or two waves, 3 = stream-K
                               over the partial last wave, each worker's
                               stream-K range before its whole tiles, 4 = as 3
                               with the whole tiles first, 5 = split tail: each
                               tile of the partial last wave cut into the same
                               k-pieces (2 or 3, one per worker, at most as many
                               pieces as workers), walked before the whole
                               tiles                                             */
    GSR_OPT_SMALL_M = 9,    /* the small-M kernel (AR/RS, M <= 256): 0 = heuristic
                               (used when M <= 256 and no other option above
                               forces a configuration), 1 = never, 2 = whenever
                               M <= 256. It streams W in tiles of rows
                               (GSR_OPT_SMALL_TILE_ROWS, at most 256), one CTA
                               pair per tile over the whole K range, against
                               all M rows at once (the activation rows are the
                               pair MMA's M, the tile's rows its N); it needs
                               no workspace beyond the status word               */
    GSR_OPT_SMALL_TILE_ROWS = 10, /* W rows per tile of the small-M kernel: 0 =
                               heuristic (the fewest rows, in multiples of 16 up
                               to 256, that spread N over every SM pair in the
                               fewest waves), else a multiple of 16 in 16..256   */
    GSR_OPT_RASTER_N = 11,  /* main kernel: n-tiles per raster group, n running
                               fastest inside a group (0 = off: GSR_OPT_RASTER_M
                               applies), 1..64                                   */
    GSR_OPT_SMALL_KBLOCKS = 12 /* small-M kernel: k-blocks of 64 per copy: 0 =
                               heuristic (the largest of 4, 3, 2 that leaves a
                               ring of four stages, where every K_r is a
                               multiple of 64; else 1), else 1..4: at most that
                               many, by the same rule                            */
} gsr_option;

/*
 * Create a plan for device `device` (a CUDA ordinal). The plan records the
 * device's SM count and shared-memory limit and the largest shapes it will
 * accept: max_M rows (AR/RS: M; AG: sum of M_r), max_N output columns, max_K
 * reduction length (AR/RS: sum of K_r; AG: K) and max_R shards. It mirrors the
 * pages' init_gemm_rs_ar(max_M, N, all_reduce) singleton (PR #53053 summary,
 * model.py), minus the mode, which here is chosen per call.
 * Returns GSR_ERR_UNSUPPORTED (and no plan) on anything but a compute
 * capability 10.3 device or when no CUDA driver is present;
 * GSR_ERR_INVALID_VALUE when out is NULL, a maximum is < 1, max_N or max_K is
 * not a multiple of 8, max_R is outside 1..GSR_MAX_SHARDS, or the maxima give
 * 2^27 or more output tiles of 128 x 128 (an output of about 2.2e12 elements,
 * far past any device's memory; the kernels count tiles and their pieces in
 * 32-bit integers).
 */
gsr_status gemm_shard_plan_create(gemm_shard_plan **out, int device, int64_t max_M,
                                  int64_t max_N, int64_t max_K, int max_R);

/*
 * Create a plan bound to no device, for a machine without a GPU: it describes
 * a device with `sm_count` SMs. Calls made with it check their arguments and
 * workspace exactly as on a device, then return GSR_ERR_UNSUPPORTED instead of
 * launching (no device pointer is touched). It takes a GB300's L2 size (126
 * MiB) where the configuration depends on it. gemm_shard_describe and
 * gemm_shard_workspace_size work as for a device plan. Errors as
 * gemm_shard_plan_create, plus GSR_ERR_INVALID_VALUE for sm_count < 1.
 */
gsr_status gemm_shard_plan_create_host(gemm_shard_plan **out, int sm_count, int64_t max_M,
                                       int64_t max_N, int64_t max_K, int max_R);

/* Destroy a plan (NULL is accepted). Outstanding calls are unaffected. */
gsr_status gemm_shard_plan_destroy(gemm_shard_plan *plan);

/* Set an option (see gsr_option). Options change the kernel configuration of
 * later calls only; they never change which elements are computed. */
gsr_status gemm_shard_plan_set_option(gemm_shard_plan *plan, gsr_option option,
                                      int64_t value);

/*
 * Bytes of workspace that every call under this plan (at any shape within its
 * maxima, with its current options) needs. Always > 0: the workspace holds a
 * status word, per-tile split-K arrival counters and fp32 split-K partials.
 * Returns 0 for a NULL plan.
 */
size_t gemm_shard_workspace_size(const gemm_shard_plan *plan);

/*
 * Zero the workspace's status word and counters (stream-ordered memset). Do
 * this once after allocating it, and again after a GSR_ERR_TIMEOUT. Kernels
 * leave the counters at zero when they finish, so no reset is needed between
 * calls. ws must be 256-byte aligned and at least gemm_shard_workspace_size
 * bytes.
 */
gsr_status gemm_shard_workspace_init(const gemm_shard_plan *plan, void *ws,
                                     size_t ws_bytes, gsr_stream_t stream);

/*
 * AR: Y = sum_{r<R} X_r . W_r^T.
 *   M      rows of every X_r and of Y; 0 returns GSR_OK with no launch
 *   N      rows of every W_r and columns of Y (multiple of 8)
 *   R      number of shards, 1..plan max_R
 *   K_r    host array of R shard widths, each >= 8 and a multiple of 8
 *   X_r    host array of R device pointers, X_r[r] is M x K_r[r] bf16 (may be
 *          NULL when M == 0; so may Y)
 *   W_r    host array of R device pointers, W_r[r] is N x K_r[r] bf16
 *   Y      device pointer, M x N bf16; rows [0, M) are written, nothing else
 *   ws     workspace of ws_bytes bytes (gemm_shard_workspace_size)
 * Shards are read in place from their own allocations; no input is copied or
 * padded. The sum over shards is accumulated in fp32 in a fixed order (shards
 * ascending, k ascending within a shard, split-K pieces ascending), so results
 * are deterministic and identical to the rows gemm_rs writes.
 */
gsr_status gemm_ar(const gemm_shard_plan *plan, int64_t M, int64_t N, int R,
                   const int64_t *K_r, const void *const *X_r, const void *const *W_r,
                   void *Y, void *ws, size_t ws_bytes, gsr_stream_t stream);

/*
 * RS: the AR sum, scattered by rows. With rps = ceil(M / R), shard s receives
 * global rows [s*rps, min(M, (s+1)*rps)) as rows [0, count_s) of Y_r[s];
 * Y_r[s] must hold rps rows of N bf16. Rows of Y_r[s] at or past count_s
 * (the reference's zero-padding rows) are not written. Arguments otherwise as
 * gemm_ar. Every written element is bit-identical to the same element of
 * gemm_ar on the same inputs.
 */
gsr_status gemm_rs(const gemm_shard_plan *plan, int64_t M, int64_t N, int R,
                   const int64_t *K_r, const void *const *X_r, const void *const *W_r,
                   void *const *Y_r, void *ws, size_t ws_bytes, gsr_stream_t stream);

/*
 * AR with replicated outputs: the AR sum written whole into each of R output
 * buffers, Y_r[r] = sum_q X_q . W_q^T for every r. This is the one-GPU
 * statement of an all-reduce whose result every rank holds: the GEMM-AR page
 * reduces each row once and multicasts it to all ranks (PR #53053 summary,
 * implementation breakdown step 1, and key source snippets: AR mode takes
 * local_M = partial_uc.shape[0] // num_ranks and stores through
 * multimem_st_16B). Here the reduced tile is rounded once and stored R times
 * from the same epilogue. Y_r[r] must each hold M x N bf16. Every written
 * element is bit-identical to gemm_ar's on the same inputs. Arguments otherwise
 * as gemm_ar.
 */
gsr_status gemm_ar_replicated(const gemm_shard_plan *plan, int64_t M, int64_t N, int R,
                              const int64_t *K_r, const void *const *X_r,
                              const void *const *W_r, void *const *Y_r, void *ws,
                              size_t ws_bytes, gsr_stream_t stream);

/*
 * AG: Y = concat_r(A_r) . W^T.
 *   N      rows of W and columns of Y (multiple of 8)
 *   K      columns of every A_r and of W (multiple of 8)
 *   R      number of shards, 1..plan max_R
 *   M_r    host array of R row counts (>= 0; a shard of 0 rows is skipped)
 *   A_r    host array of R device pointers, A_r[r] is M_r[r] x K bf16 (ignored
 *          when M_r[r] == 0)
 *   W      device pointer, N x K bf16
 *   Y      device pointer, (sum M_r) x N bf16; shard r's rows start at
 *          sum_{q<r} M_q. A sum of 0 returns GSR_OK with no launch (Y may then
 *          be NULL).
 */
gsr_status gemm_ag(const gemm_shard_plan *plan, int64_t N, int64_t K, int R,
                   const int64_t *M_r, const void *const *A_r, const void *W, void *Y,
                   void *ws, size_t ws_bytes, gsr_stream_t stream);

/*
 * AG whose shards may still be arriving when the call starts: the single-kernel
 * AG-GEMM with in-kernel waiting that the AG-GEMM page names as future work
 * ("[Kimi-K3] AG-GEMM for Sequence Parallelism", Component breakdown, closing
 * remark). Before the kernel reads any row of A_r it waits until the device
 * word ready[r] reaches `epoch` (compared with wrap-around: (int32)(ready[r] -
 * epoch) >= 0), so the copies that bring the shards in (a copy stream, in shard
 * order) overlap the GEMM on the shards already present. Pass a new epoch per
 * call instead of resetting the flags.
 *   ready  device array of R uint32 words, 4-byte aligned; written by another
 *          agent, typically gemm_shard_signal on the copy stream
 * The wait is bounded by the plan's timeout (GSR_OPT_TIMEOUT_NS): if a flag
 * never arrives the kernel records GSR_ERR_TIMEOUT in the workspace status
 * word, lets its in-flight copies land, frees its resources and returns;
 * gemm_shard_check_status reports it and the workspace must be re-initialised.
 * Y is then incomplete. Arguments otherwise as gemm_ag.
 */
gsr_status gemm_ag_flagged(const gemm_shard_plan *plan, int64_t N, int64_t K, int R,
                           const int64_t *M_r, const void *const *A_r, const void *W, void *Y,
                           const uint32_t *ready, uint32_t epoch, void *ws, size_t ws_bytes,
                           gsr_stream_t stream);

/*
 * Enqueue on `stream` a write of `value` to the device word `flag`, after all
 * earlier work on the stream and behind a system-wide memory fence. It is a
 * stream memory operation (cuStreamWriteValue32): it runs no kernel, so it can
 * signal a kernel that occupies every SM, such as gemm_ag_flagged.
 * GSR_ERR_INVALID_VALUE for a NULL or misaligned flag; GSR_ERR_UNSUPPORTED on
 * a host plan or a driver without stream memory operations.
 */
gsr_status gemm_shard_signal(const gemm_shard_plan *plan, uint32_t *flag, uint32_t value,
                             gsr_stream_t stream);

/*
 * AR exactly as gemm_ar, for callers that cannot allocate device memory: there
 * is no workspace argument. (The pages have no counterpart; this entry point
 * exists for callers such as an inference engine that claims all free HBM for
 * its KV cache at start-up, or code on a latency-critical path where
 * cudaMalloc's implicit synchronisation is not acceptable.)
 *
 * Its scratch (status word, split-K counters and partials) is one fixed array
 * of 24 MiB in device global memory, part of the library image: every GPU that
 * loads the library holds it until the process exits. Nothing is allocated or
 * freed by the call.
 *   - When the plan's configuration for a shape needs more than 24 MiB of
 *     scratch, the call runs the uniform schedule instead (the same results
 *     within rounding; split pieces then need at most one 128 KiB slot per
 *     SM), unless the plan forces a split (GSR_OPT_SPLIT_K) or a schedule
 *     (GSR_OPT_SCHEDULE): a forced configuration is never replaced, and one
 *     that does not fit is rejected with GSR_ERR_WORKSPACE before anything is
 *     launched; use gemm_ar with a workspace for it. The uniform schedule
 *     always fits when 4 bytes x (ceil(max_M/128) + 2 max_R) x ceil(max_N/128)
 *     counters plus 128 KiB per SM stay under 24 MiB (on a 152-SM GB300:
 *     plans of up to about a million output tiles). Where the configuration
 *     is the plan's own (gemm_shard_describe reports it), the result is
 *     bit-identical to gemm_ar's.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) and keeps it for that device's context; make
 *     that first call before any stream capture begins. The lookup is
 *     repeated only when the device's context has changed (after a
 *     cudaDeviceReset, the library image and its array are loaded again) or
 *     on a thread where no context is current yet.
 *   - Every call on a device shares the one array and starts by clearing its
 *     status word and counters (a stream-ordered memset). Calls that may
 *     overlap on the GPU (different streams, or different host threads without
 *     ordering) race on it and must not be issued.
 *   - A bounded in-kernel wait that runs out leaves its code in the array's
 *     status word: gemm_ar_noalloc_check_status reads it. The next call
 *     clears it, so read it before the next call.
 * Arguments, validation and results are those of gemm_ar.
 */
gsr_status gemm_ar_noalloc(const gemm_shard_plan *plan, int64_t M, int64_t N, int R,
                           const int64_t *K_r, const void *const *X_r,
                           const void *const *W_r, void *Y, gsr_stream_t stream);

/*
 * gemm_shard_check_status for gemm_ar_noalloc: synchronise `stream`, read the
 * built-in scratch's status word on the plan's device, clear it and return
 * GSR_OK or GSR_ERR_TIMEOUT (the code of the first wait that ran out is in
 * gsr_last_error_string). It reports on the last gemm_ar_noalloc call on that
 * device, whichever plan made it. (The pages have no counterpart.)
 * GSR_ERR_INVALID_VALUE for a NULL plan, GSR_ERR_UNSUPPORTED on a host plan,
 * GSR_ERR_CUDA if the copy fails.
 */
gsr_status gemm_ar_noalloc_check_status(const gemm_shard_plan *plan, gsr_stream_t stream);

/*
 * Packed gather of per-shard states (the pages' "Kimi K3 SP: pack the per-layer
 * all-gathers into one", PR #51070 summary, implementation steps 2-3 and its
 * model.py snippet: each rank concatenates its hidden state and auxiliary
 * states along the last dimension, one all-gather stacks the ranks' packed
 * rows, and the result keeps the first full_num_tokens rows; splitting it by
 * the hidden size gives the gathered states back). Here the ranks are R sets of
 * buffers on this GPU and the whole thing is one pass of copies:
 *     P[g, t*H : (t+1)*H] = S[r*T + t][g - row_begin_r, :]      for g < rows_out,
 * where row_begin_r = M_0 + ... + M_{r-1} and g lies in [row_begin_r,
 * row_begin_r + M_r). Bits are copied unchanged (bf16 in, bf16 out).
 *   R         shards, 1..the plan's max_R
 *   M_r       host array of R row counts (>= 0; the sequence-parallel shards)
 *   T         states per shard, 1..16 (the hidden state, then the aux states)
 *   H         columns of every state (the hidden size), a positive multiple of 8
 *   S         host array of R*T device pointers, S[r*T + t] = shard r's state t,
 *             M_r x H row-major bf16, 16-byte aligned; read in place. A shard
 *             with no kept row (all of its rows at or past rows_out) is not
 *             read and its pointers may be NULL.
 *   rows_out  rows kept (full_num_tokens), 0..sum of M_r
 *   P         device output, rows_out x (T*H) row-major bf16, 16-byte aligned,
 *             caller-owned; every element is written, nothing else is. The
 *             split-back state t is the strided view P[:, t*H : (t+1)*H].
 *   ws        the plan's workspace (only its status word is used; a bounded
 *             wait that runs out is reported by gemm_shard_check_status)
 * Errors: GSR_ERR_INVALID_VALUE for the shapes and pointers above,
 * GSR_ERR_WORKSPACE for a NULL, misaligned or too small workspace,
 * GSR_ERR_UNSUPPORTED on a host plan (after validation), GSR_ERR_CUDA when the
 * launch fails. rows_out == 0 returns GSR_OK with no launch. Stream-ordered.
 */
gsr_status gemm_shard_pack_gather(const gemm_shard_plan *plan, int R, const int64_t *M_r, int T,
                                  int64_t H, const void *const *S, int64_t rows_out, void *P,
                                  void *ws, size_t ws_bytes, gsr_stream_t stream);

/* ------------------------------------------------------- routed projections
 * Products whose weights the ROW picks: rows grouped by expert, and rows that
 * carry a low-rank adapter beside a shared projection. (The pages this library
 * restates have no counterpart; a tensor-parallel model runs these between the
 * projections above, e.g. the experts between AG and AR.) Conventions as
 * above, and:
 *   - Routing data (ids, offsets, rows, positions, adapters) lives on the device
 *     and is read there: no call waits for the host to see it. The host cannot
 *     check it, so the kernels do: a value out of range never makes a read or
 *     write out of bounds. What it gives instead is said at each call.
 *   - Workspace: these calls share a workspace of their own, of
 *     gemm_routed_workspace_size bytes, initialised once with
 *     gemm_routed_workspace_init and left ready for the next call by every
 *     call. gemm_shard_check_status reads its status word. gemm_group_route and
 *     gemm_group_combine need none.
 *   - Options: GSR_OPT_TIMEOUT_NS and GSR_OPT_MAX_CTAS (in whole CTA pairs, one at
 *     least) apply to the products (not to gemm_expert_layer's own two kernels); the
 *     others do not.
 *   - Results are reproducible: sums run in an order that depends on the shapes
 *     and the group sizes alone.
 *   - Graphs: the calls may be recorded in a CUDA graph; a replay reads the
 *     routing data's current contents.
 */

/* Limits of one call. */
#define GSR_MAX_GROUPS 1024     /* E, experts                                  */
#define GSR_MAX_TOPK 128        /* entries of one token                        */
#define GSR_MAX_RANK 128        /* columns of an adapter                       */
#define GSR_MAX_ADAPTERS 65536  /* L                                           */
#define GSR_MAX_LAYER_TOKENS 64    /* T of gemm_expert_layer                   */
#define GSR_MAX_LAYER_ENTRIES 1024 /* its T * topk                             */

/* Bytes of workspace for every routed call under the plan; 0 for a NULL plan. One size
 * serves them all: it holds gemm_expert_layer's rows too, 4 * min(max_M,
 * GSR_MAX_LAYER_ENTRIES) * max_N bytes, so a plan for routed calls takes the max_N that
 * these need and a plan of its own serves a wider projection. */
size_t gemm_routed_workspace_size(const gemm_shard_plan *plan);

/* Zero its status word and counters (stream-ordered), once after allocating it
 * and after a GSR_ERR_TIMEOUT. ws: 256-byte aligned, at least
 * gemm_routed_workspace_size bytes. */
gsr_status gemm_routed_workspace_init(const gemm_shard_plan *plan, void *ws, size_t ws_bytes,
                                      gsr_stream_t stream);

/*
 * Route: group the entries of T tokens by expert, in a stable order.
 *   ids       device, T x topk integers of id_bytes (4 or 8) bytes: entry i =
 *             t * topk + j names the expert of token t's j-th entry. A value
 *             outside 0..E-1 drops the entry.
 *   offsets   device out, E + 1 int32: group e is the sorted rows
 *             [offsets[e], offsets[e+1]); offsets[E] entries are kept
 *   source    device out, T * topk int32: the token of each sorted row (i /
 *             topk), -1 at and past offsets[E]
 *   position  device out, T x topk int32: the sorted row of each entry, -1 for a
 *             dropped one
 * Within a group rows keep the entries' order. T * topk may not exceed the
 * plan's max_M. The outputs overlap neither one another nor ids (position is
 * scratch meanwhile). T == 0 writes offsets (zeros) alone.
 */
gsr_status gemm_group_route(const gemm_shard_plan *plan, int64_t T, int topk, int E,
                            const void *ids, int id_bytes, int32_t *offsets, int32_t *source,
                            int32_t *position, gsr_stream_t stream);

/*
 * Grouped product: Y[i] = X[row(i)] . W[e]^T for the rows i of group e,
 * offsets[e] <= i < offsets[e+1], row(i) = rows ? rows[i] : i.
 *   E, M      groups (1..GSR_MAX_GROUPS) and rows of Y (<= max_M); M == 0 returns
 *             GSR_OK with no launch
 *   N, K      multiples of 8, <= max_N and max_K
 *   offsets   device, E + 1 int32, non-decreasing; clamped to 0..M
 *   T, X      X is T x K bf16; T >= M without `rows`
 *   rows      device, M int32, or NULL; an index outside 0..T-1 reads as a row of
 *             zeros
 *   W         device, E x N x K bf16
 *   Y         device, M x N bf16; rows of no group are not written
 * Groups may have any size, 0 and M among them. The accumulation is fp32, the
 * output rounded once. Only the weights of groups that have rows are read.
 */
gsr_status gemm_grouped(const gemm_shard_plan *plan, int E, int64_t M, int64_t N, int64_t K,
                        const int32_t *offsets, int64_t T, const void *X, const int32_t *rows,
                        const void *W, void *Y, void *ws, size_t ws_bytes, gsr_stream_t stream);

/*
 * Gated grouped product: Y[i] = silu(g) * u elementwise, with g and u the
 * products of row(i) with the first and the last N rows of W[e]
 * (W: E x 2N x K; silu(x) = x / (1 + exp(-x))). Both products, the activation
 * and the product of the two stay in fp32; Y is rounded once. Otherwise as
 * gemm_grouped.
 */
gsr_status gemm_grouped_gated(const gemm_shard_plan *plan, int E, int64_t M, int64_t N,
                              int64_t K, const int32_t *offsets, int64_t T, const void *X,
                              const int32_t *rows, const void *W, void *Y, void *ws,
                              size_t ws_bytes, gsr_stream_t stream);

/*
 * Combine: Y[t] = base[t] + sum_j weights[t, j] * Z[position[t, j]].
 *   H         columns (a multiple of 8, <= max_N)
 *   Z         device, z_rows x H bf16
 *   position  device, T x topk int32; an entry outside 0..z_rows-1 adds nothing,
 *             whatever its weight holds
 *   weights   device, T x topk fp32
 *   base      device, T x H bf16, or NULL (0); may be Y
 *   Y         device, T x H bf16
 * fp32, j ascending after base, rounded once.
 */
gsr_status gemm_group_combine(const gemm_shard_plan *plan, int64_t T, int topk, int64_t H,
                              int64_t z_rows, const void *Z, const int32_t *position,
                              const float *weights, const void *base, void *Y,
                              gsr_stream_t stream);

/*
 * Expert layer of a few tokens: what gemm_group_route, gemm_grouped_gated,
 * gemm_grouped and gemm_group_combine do together, in one call:
 *     Y[t] = base[t] + sum_j weights[t, j] * W_down[e] . h_tj,
 *     h_tj = silu(G[e] . X[t]) * (U[e] . X[t]),  e = ids[t, j],
 * G[e] and U[e] the first and the last N rows of W_up[e].
 *   T, topk   tokens and entries of each: T <= GSR_MAX_LAYER_TOKENS, T * topk <=
 *             GSR_MAX_LAYER_ENTRIES and max_M; T == 0 returns GSR_OK with no launch
 *   E, N, K   experts, their inner and the outer width: multiples of 8, at most max_N and
 *             max_K and 2^20, 2 N K below 2^38
 *   ids       device, T x topk integers of id_bytes (4 or 8) bytes; a value outside
 *             0..E-1 drops the entry, whatever its weight holds. A token may name an
 *             expert twice.
 *   weights   device, T x topk fp32
 *   X, base   device, T x K bf16; base may be NULL (0)
 *   W_up      device, E x 2N x K bf16; W_down: E x K x N bf16
 *   Y         device, T x K bf16; may be base or X
 * Up to 64 entries (T * topk), and up to 8 E, run in two kernels of their own, whose
 * weighted sum is fp32 (experts ascending, the entries of one in order, in parts of k whose
 * number depends on the shapes); more run in the kernels of the calls named above,
 * with the down products rounded to bf16 before they are weighted, as there. In both the
 * products accumulate in fp32, h is rounded to bf16 between them and Y once. Only the
 * weights of named experts are read.
 */
gsr_status gemm_expert_layer(const gemm_shard_plan *plan, int64_t T, int topk, int E, int64_t N,
                             int64_t K, const void *ids, int id_bytes, const float *weights,
                             const void *X, const void *W_up, const void *W_down,
                             const void *base, void *Y, void *ws, size_t ws_bytes,
                             gsr_stream_t stream);

/*
 * AR with low-rank adapters: gemm_ar's sum plus each row's own adapter,
 *     Y[m] = sum_r X_r[m] . W_r^T + scale[a] * (sum_r X_r[m] . A_r[a]^T) . B[a]^T,
 * a = adapter[m].
 *   L, rank   adapters (1..GSR_MAX_ADAPTERS) and their columns, a multiple of 8 up
 *             to GSR_MAX_RANK (an adapter of a lower rank: zero rows of A_r)
 *   A_r       host array of R device pointers, A_r[r] is L x rank x K_r bf16
 *   B         device, L x N x rank bf16
 *   adapter   device, M int32; a value outside 0..L-1 (e.g. -1): no adapter
 *   scale     device, L fp32, or NULL (1)
 * The low-rank rows (scale included) are rounded to bf16 between the two
 * products; both products accumulate in fp32 in one accumulator with the base
 * product, and Y is rounded once. Only adapters that some row names are read.
 * Values that are not finite give what the formula gives, in the rows and columns
 * that it uses them in, and change no other.
 * M <= max_M; Y must not overlap an input. Other arguments as gemm_ar, with
 * the routed workspace.
 */
gsr_status gemm_ar_lora(const gemm_shard_plan *plan, int64_t M, int64_t N, int R,
                        const int64_t *K_r, const void *const *X_r, const void *const *W_r,
                        int L, int rank, const void *const *A_r, const void *B,
                        const int32_t *adapter, const float *scale, void *Y, void *ws,
                        size_t ws_bytes, gsr_stream_t stream);

/* ------------------------------------------------------- 8-bit projections
 * The AR and AG products on 8-bit operands, and what feeds them: the residual's
 * addition with the RMS norm, and the quantisation. (The pages this library
 * restates have no counterpart; a serving model stores the weights and sends the
 * activations this way.) Conventions as above, and:
 *   - 8 bits are e4m3 (1, 4, 3 bits; finite up to 448), one byte an element, rows
 *     dense. A group of elements shares an fp32 scale; an element stands for q *
 *     scale. Groups of activations are 128 columns of one row, groups of weights
 *     blocks of 128 x 128; a last group may be short. A K-shard starts its own.
 *   - Scales of rows are stored by column block: element (b, m) of a dense
 *     ceil(K / 128) x M array belongs to columns 128 b .. of row m. Scales of blocks
 *     are row-major, ceil(N / 128) x ceil(K / 128). Pointers 4-byte aligned. A product
 *     takes a row's scale times a block's in fp32 before it meets the block's sum, so the
 *     two may be any fp32 values whose product is a normal number or 0. Past the largest
 *     number the product is an infinity (and NaN with a sum of 0), below 2^-126 it has
 *     the bits that fp32 has left there.
 *   - K, K_r (and H with Q) are multiples of 16.
 *   - Quantising a group of values v: scale = max(max|v| / 448, 2^-126), q = v * (1 /
 *     scale) to the nearest e4m3, ties to even, at most 448 in magnitude. A group
 *     that holds NaN has scale NaN, one that holds an infinity scale infinity, and
 *     what it stands for is NaN.
 *   - Options: GSR_OPT_TIMEOUT_NS and GSR_OPT_MAX_CTAS (in whole CTA pairs, one at
 *     least) apply to the products; the others do not.
 *   - The workspace is gemm_shard_workspace_size's; the products use its status word
 *     alone. The norm and the quantisation need none.
 *   - Graphs, streams and errors as for gemm_ar.
 */

/*
 * Residual sum and RMS norm, for rows of H columns:
 *     h = X + residual,  y = h * (mean(h^2) + eps)^-1/2 * gamma.
 *   H         a multiple of 8 (of 16 with Q), at most 32768 and the larger of max_N and
 *             max_K
 *   X         M x H bf16; M <= max_M, 0 returns GSR_OK with no launch
 *   residual  M x H bf16, or NULL (0)
 *   gamma     H bf16, or NULL (1)
 *   eps       finite, >= 0
 *   sum       M x H bf16 out: h, or NULL
 *   Y         M x H bf16 out: y, or NULL
 *   Q, scale  M x H e4m3 and ceil(H / 128) x M fp32 out: y in 8 bits, or both NULL
 * One output at least. Everything is fp32 in between, the squares' sum too: a row of
 * finite h where it passes the largest number has y = 0, and where it vanishes, with eps
 * 0, y is infinite (NaN for h = 0). sum, Y and Q are each rounded
 * once from the unrounded values. sum and Y may each be X or residual itself (not one
 * another's buffer); otherwise the outputs overlap nothing.
 */
gsr_status gemm_shard_rms_norm(const gemm_shard_plan *plan, int64_t M, int64_t H, const void *X,
                               const void *residual, const void *gamma, float eps, void *sum,
                               void *Y, void *Q, float *scale, gsr_stream_t stream);

/*
 * Quantise a matrix of rows x cols bf16 to e4m3.
 *   block_rows  1: a scale for each row and 128 columns (activations; rows <=
 *               max_M, scale ceil(cols / 128) x rows); 128: for each block of 128 x
 *               128 (weights; rows <= max_N, scale ceil(rows / 128) x ceil(cols / 128))
 *   cols        a multiple of 16, at most max_K
 *   Q, scale    out, overlapping nothing; rows == 0 returns GSR_OK with no launch
 */
gsr_status gemm_shard_quantize(const gemm_shard_plan *plan, int64_t rows, int64_t cols,
                               int block_rows, const void *X, void *Q, float *scale,
                               gsr_stream_t stream);

/*
 * AR on 8-bit operands: Y = sum_r X_r . W_r^T over what the operands stand for.
 *   X_r, SX_r  host arrays of R device pointers: X_r[r] is M x K_r e4m3, SX_r[r] its
 *              row scales, ceil(K_r / 128) x M
 *   W_r, SW_r  W_r[r] is N x K_r e4m3, SW_r[r] its block scales, ceil(N / 128) x
 *              ceil(K_r / 128)
 *   Y          M x N bf16
 * The products of a block of 128 columns are summed in the tensor cores, times the
 * product of its two scales added up in fp32, blocks ascending, and Y is rounded once.
 * A value that is not finite reaches the rows and columns that use it and no other.
 * The sums' order depends on the shapes alone. Other arguments as gemm_ar.
 */
gsr_status gemm_ar_fp8(const gemm_shard_plan *plan, int64_t M, int64_t N, int R,
                       const int64_t *K_r, const void *const *X_r, const float *const *SX_r,
                       const void *const *W_r, const float *const *SW_r, void *Y, void *ws,
                       size_t ws_bytes, gsr_stream_t stream);

/*
 * AG on 8-bit operands: Y = concat_r(A_r) . W^T over what the operands stand for.
 *   A_r, SA_r  host arrays of R device pointers: A_r[r] is M_r x K e4m3, SA_r[r] its
 *              row scales, ceil(K / 128) x M_r (both ignored when M_r[r] == 0)
 *   W, SW      N x K e4m3 and its block scales
 * Otherwise as gemm_ar_fp8 and gemm_ag.
 */
gsr_status gemm_ag_fp8(const gemm_shard_plan *plan, int64_t N, int64_t K, int R,
                       const int64_t *M_r, const void *const *A_r, const float *const *SA_r,
                       const void *W, const float *SW, void *Y, void *ws, size_t ws_bytes,
                       gsr_stream_t stream);

/*
 * Synchronise `stream`, read the workspace status word, clear it and return
 * GSR_OK or GSR_ERR_TIMEOUT (the code of the first wait that ran out is
 * available through gsr_last_error_string). After a timeout, re-run
 * gemm_shard_workspace_init before the next call.
 */
gsr_status gemm_shard_check_status(const gemm_shard_plan *plan, void *ws,
                                   gsr_stream_t stream);

/* Text of the last error on the calling thread ("" if none). Never NULL. */
const char *gsr_last_error_string(void);

/* Kernel configuration of a call, as gemm_shard_describe reports it. */
typedef struct {
    int block_n;            /* output tile width: 128, 192 or 256 (the small-M
                               kernel: W rows per tile, a multiple of 16 <= 256)  */
    int cta_group;          /* 1: a CTA per 128-row tile; 2: a CTA pair per 256 rows */
    int schedule;           /* 1 = uniform pieces, 2 = stream-K hybrid, 3 = the
                               small-M kernel (one CTA pair per tile of block_n
                               W rows over the whole K range, split = 1),
                               4 = split tail (split = pieces per tail tile)      */
    int split;              /* uniform schedule: pieces per tile                    */
    int64_t tiles;          /* output tiles                                         */
    int64_t dp_tiles;       /* stream-K: tiles run whole                            */
    int64_t sk_iters;       /* stream-K: k-blocks shared out over the workers       */
    int ctas;               /* persistent CTAs launched                             */
    size_t workspace_bytes; /* workspace this call needs                           */
    int kblocks;            /* small-M kernel: k-blocks of 64 per copy (1 to 4);
                               1 for the main kernel                              */
    int l2_hints;           /* the TMA L2 hints taken: 1 = none, 2 = A evict-last /
                               B evict-first, 3 = A evict-first / B evict-last    */
} gsr_config;

/* The kernel configuration the plan chooses for a call, for logging and tests:
 * mode 0 = AR, 1 = RS, 2 = AG. AR/RS use M (>= 0) and sizes = K_r (positive
 * multiples of 8; K is ignored); AG uses K (a positive multiple of 8) and
 * sizes = M_r (>= 0; M is ignored). The plan's maxima are not checked. The
 * configuration depends on the shape, the device and the plan's options, never
 * on the mode, except that AG counts tiles per shard. GSR_ERR_INVALID_VALUE
 * for a NULL plan, out or sizes, a mode outside 0..2, R outside 1..16 or a
 * size that breaks the rules above. */
gsr_status gemm_shard_describe(const gemm_shard_plan *plan, int mode, int64_t M,
                               int64_t N, int64_t K, int R, const int64_t *sizes,
                               gsr_config *out);

#ifdef __cplusplus
}
#endif

#endif /* GSR_H */
