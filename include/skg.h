/*
 * skg.h -- C ABI of the skinny decode projection library (libskg.so).
 *
 * The library computes the projection of low-batch LLM decode,
 *
 *     y[m,n] = sum_k x[m,k] * W[n,k]   (+ residual[m,n])     0 <= m < M <= 64
 *
 * with bfloat16 W, x and residual, fp32 accumulation and a bf16 (or fp32)
 * output, on one NVIDIA GB300 (sm_103a).  Every step runs in the library's
 * own CUDA kernels; there is no CPU path and no fallback to another kernel.
 *
 * Where the operations come from.  The method is described, at paragraph
 * level and without formulas, by "Hyper Optimizing Kimi K3 in vLLM: Moving
 * Fast and Responsibly" (vLLM blog, NVIDIA), read here through its deep-notes
 * page (papercache.org) and its French translation (spke.com, "Hyper
 * optimisation de Kimi K3 dans vLLM : aller vite et responsablement"):
 *   [TS] method details 1 / Partie 1 section 1, "Tune shapes for the
 *        workload": small-matrix kernels at batch 1-2, split-K kernels at
 *        larger batch, each projection tuned to block sizes that fill the GPU.
 *   [OC] method details 2 / Partie 1 section 2, "Overlap computation and
 *        communication": the output projection fused with the attention
 *        residual add.
 *   [PF] method details 4 / Partie 1 section 4, "Prefetching upcoming weights
 *        into cache": small-batch decode is bound by streaming weights from
 *        HBM; a side-stream kernel preloads the next operation's weights.
 *   [VC] background 2 "Validate correctness systematically" / Partie 2
 *        section 3: an activation read was once hoisted above a
 *        synchronisation wait; early loads were restricted to static weights.
 *
 * Conventions shared by every entry point
 *   - Layouts are dense row-major: W is [N,K] (an nn.Linear weight), x is
 *     [M,K], residual and y are [M,N].  bf16 tensors are raw 16-bit patterns.
 *   - Device pointers are CUDA device (or managed) addresses on the current
 *     device.  x and W must be 16-byte aligned (they are read with TMA and
 *     16-byte vector loads); residual and y need their element alignment.
 *   - Streams are cudaStream_t handles passed as void* (NULL = legacy default
 *     stream).  Launches are asynchronous and stream-ordered.
 *   - The caller owns every tensor and stream.  The library owns each plan,
 *     the plan's split-K workspace and counters, and its TMA descriptors.
 *   - Every call returns a status; none throws across the ABI.  On failure,
 *     skg_last_error() returns a message for the calling thread.  A rejected
 *     call launches nothing.
 */
#ifndef SKG_H
#define SKG_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SKG_VERSION 3

/* Symbols of the ABI are exported; everything else in the library is hidden. */
#if defined(__GNUC__)
#define SKG_API __attribute__((visibility("default")))
#else
#define SKG_API
#endif

typedef enum skg_status {
    SKG_OK = 0,
    SKG_ERR_INVALID_ARG = 1,    /* bad size, NULL where a tensor is needed, bad enum */
    SKG_ERR_UNSUPPORTED = 2,    /* legal request outside what the library implements */
    SKG_ERR_ALIGNMENT = 3,      /* a pointer misses its required alignment */
    SKG_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed (message says which) */
    SKG_ERR_DEVICE_TIMEOUT = 5  /* a kernel's bounded wait ran out (see skg_plan_check) */
} skg_status;

typedef enum skg_epilogue {
    SKG_EPI_BF16 = 0,           /* y = bf16(x.W^T) */
    SKG_EPI_BF16_RESIDUAL = 1,  /* y = bf16(x.W^T + residual), one rounding [OC] */
    SKG_EPI_FP32 = 2            /* y = fp32(x.W^T), e.g. router scores */
} skg_epilogue;

typedef enum skg_kernel_kind {
    SKG_KERNEL_GEMV = 1,        /* M <= 2: CUDA-core kernel; weights by 16-byte loads or bulk copies [TS] */
    SKG_KERNEL_SPLITK_TC = 2    /* M > 2: TMA + tcgen05 split-K kernel [TS] */
} skg_kernel_kind;

/* Canonical number of K chunks.  Both kernels cut K into this many chunks
 * (in 16-byte vectors for GEMV, in 64-wide k-blocks for SPLITK_TC), sum each
 * chunk from a fresh fp32 accumulator, and combine the chunk sums with one
 * fixed balanced binary tree.  A split only decides which CTA or warp owns
 * which subtree, so every allowed split gives bit-identical results. */
#define SKG_CANONICAL_CHUNKS 16

/* What a plan will launch.  Filled by skg_plan_query and skg_plan_info. */
typedef struct skg_plan_desc {
    int kernel_kind;        /* skg_kernel_kind */
    int M, N, K, epilogue;
    int split_k;            /* S: CTAs (TC) or warps (GEMV) sharing one output's K range; power of 2 dividing 16 */
    int tile_n;             /* W rows per output tile: 128 (TC) or rows per CTA group (GEMV) */
    int m_pad;              /* MMA N (TC: M rounded up to 16) or M (GEMV) */
    int stages;             /* TC: shared-memory ring stages; GEMV split > 1: weight-ring slots per
                               warp; GEMV split 1: 0 = 16-byte loads into registers, 2 = each warp's
                               weight batches moved by bulk copies through a shared-memory slot,
                               whole rows per warp; 3 = the same in one balanced wave (CTAs own row
                               runs, warps equal runs of chunks, rows combined in shared memory) */
    int tma_burst;          /* TC: k-blocks the TMA producer requests back to back; GEMV split 1
                               with bulk copies: strips (512 bytes each) per copy, 4 or 8 */
    int grid;               /* CTAs launched */
    int threads;            /* threads per CTA */
    int smem_bytes;         /* dynamic shared memory per CTA */
    int from_table;         /* 1 if (M,N,K,epilogue) hit the measured picker table */
    size_t workspace_bytes; /* split-K partials + counters owned by the plan */
    size_t prefetch_bytes;  /* bytes skg_prefetch_l2 touches for this plan's W */
    int pdl;                /* 1: launched with programmatic dependent launch */
    int l2_ahead;           /* weights requested into L2 ahead of use: TC k-blocks after the
                               ring, before the wait for the previous kernel; GEMV (split 1)
                               batches of the row; 0 = none */
    int reducers;           /* TC: the last `reducers` CTAs to finish a tile share its final
                               reduction (1, 2, 4 or 8; a launch uses fewer where the split is
                               smaller, and 1 where its grid is more than one wave); GEMV: 0 */
    int ctas_per_sm;        /* CTAs one SM holds at once: TC, from the kernel's registers, shared
                               memory, threads and TMEM columns at this launch shape; GEMV, the
                               count the plan sizes one-wave grids from.  Filled by skg_plan_info;
                               0 from skg_plan_query */
} skg_plan_desc;

typedef struct skg_plan_s *skg_plan_t;

/*
 * skg_plan_query -- the kernel choice and launch shape for (M,N,K,epilogue)
 * on a GPU with num_sms SMs and l2_bytes of L2, without touching any GPU.
 * [TS]: M <= 2 -> SKG_KERNEL_GEMV, M > 2 -> SKG_KERNEL_SPLITK_TC, except that
 * an M <= 2 shape runs the tensor-core kernel where the table of measured
 * timings holds a tensor-core row for exactly that (M,N,K,epilogue) (written
 * only where it was faster on GB300), where K is too long for the GEMV to
 * stage x in shared memory (M = 1: K > 115,200), or at M = 2 from N = 2048
 * unless the table holds a GEMV row for exactly that shape; inside each kind
 * the split and pipeline depth come from that table (nearest M for a listed
 * (N,K,epilogue)), else from a rule measured on GB300 (split-K: the finest
 * split, at most 8, whose grid is one wave at the ring's occupancy).
 * Constraints: 1 <= M <= 64, N >= 1, K >= 8 and K % 8 == 0, epilogue valid.
 * Errors: SKG_ERR_INVALID_ARG (sizes, enum, NULL out), SKG_ERR_UNSUPPORTED.
 */
SKG_API skg_status skg_plan_query(int M, int N, int K, int epilogue, int num_sms,
                          size_t l2_bytes, skg_plan_desc *out);

/*
 * skg_plan -- build a plan for (M,N,K,epilogue) on the current CUDA device.
 * Picks the kernel as skg_plan_query does and allocates a mapped host word for
 * device-side error reports; a tensor-core plan also allocates its split-K
 * workspace, S x ceil(N/128) x M x 128 fp32 partials plus one zeroed
 * counter per 128-row tile.  The plan must be
 * freed with skg_plan_destroy.  One skg_run of a plan may be in flight at a
 * time (the workspace is shared); concurrent streams need separate plans.
 * Errors: as skg_plan_query, plus SKG_ERR_CUDA.  *out is NULL on failure.
 */
SKG_API skg_status skg_plan(int M, int N, int K, int epilogue, skg_plan_t *out);

/*
 * skg_plan_force -- override of the picker inside the plan's kernel kind
 * (used by tests and by the tuning sweep): split_k (power of 2 dividing 16;
 * TC needs 2..16, GEMV 1..8); for TC, stages (2..16, limited by shared
 * memory) and tma_burst (1..stages); for GEMV, grid (CTAs, >= 1), and at
 * split 1 the load path: stages 1 = 16-byte loads into registers, stages 2 =
 * bulk copies of tma_burst (4 or 8) strips per warp batch, stages 3 = the
 * same batches in one balanced wave (grid <= N, at most 256 rows per CTA)
 * (K % 256 == 0 only; SKG_ERR_UNSUPPORTED otherwise); at split > 1, stages =
 * ring slots (2..9).  A 0 keeps the current value; a field that does not apply must be 0.
 * If the workspace must grow, a new one is allocated and the old one is kept
 * until skg_plan_destroy, because a CUDA graph that captured skg_run of this
 * plan earlier still launches with the captured split, descriptors and
 * workspace.  Used by tests to run every allowed split.  Errors: SKG_ERR_INVALID_ARG, SKG_ERR_UNSUPPORTED, SKG_ERR_CUDA.
 */
SKG_API skg_status skg_plan_force(skg_plan_t plan, int split_k, int stages, int grid,
                                  int tma_burst);

/*
 * skg_plan_force_kernel -- run the plan on the given kernel kind
 * (SKG_KERNEL_GEMV: M <= 2 only; SKG_KERNEL_SPLITK_TC: any M), its launch
 * shape re-picked as skg_plan_query picks it for that kind; earlier
 * skg_plan_force overrides are dropped, the PDL setting is kept.  The two
 * kinds accumulate in different orders, so their results may differ in the
 * last bits (each within the same error bound).  Workspace as skg_plan_force.
 * Used by the tuner and the tests.  Errors: SKG_ERR_INVALID_ARG (NULL plan,
 * unknown kind), SKG_ERR_UNSUPPORTED (GEMV at M > 2, a shape the kind cannot
 * run), SKG_ERR_CUDA.
 */
SKG_API skg_status skg_plan_force_kernel(skg_plan_t plan, int kind);

/*
 * skg_plan_set_k_shard -- [OC] row-parallel projection: the plan computes
 * rank `rank` of `ranks` (1, 2, 4 or 8) of a K split across ranks.  Rank r
 * owns canonical chunks [16r/R, 16(r+1)/R) of K, i.e. columns [rK/R,
 * (r+1)K/R) (K % 1024 == 0 when ranks > 1).  After this call skg_run takes
 * x as that shard [M, K/R] and W as [N, K/R] (dense, row stride K/R) and
 * leaves in y (fp32 [M, N]: the plan's epilogue must be SKG_EPI_FP32) the
 * value of the rank's subtree of the canonical tree, so that
 * skg_combine_partials over the R ranks gives exactly the bits of one
 * launch of the split-K kernel over the whole K.  The plan switches to the
 * split-K kernel if needed and splits a rank's chunks at most 16/R ways;
 * skg_prefetch_l2 then covers the shard.  ranks == 1 restores the whole K.
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_UNSUPPORTED (epilogue, K), SKG_ERR_CUDA.
 */
SKG_API skg_status skg_plan_set_k_shard(skg_plan_t plan, int rank, int ranks);

/*
 * skg_combine_partials -- the cross-rank step of a row-parallel projection
 * [OC]: y[m,n] = the R rank partials (fp32 [M, N] each; `partials` is a host
 * array of R device pointers) combined in rank order by the top levels of
 * the canonical tree, + residual (bf16 [M, N], given iff epilogue is
 * SKG_EPI_BF16_RESIDUAL) in fp32, rounded once to bf16 (stored as fp32 for
 * SKG_EPI_FP32).  The caller brings the partials to this device first (an
 * all-gather, or peer pointers).  ranks: 1, 2, 4 or 8.  One kernel on
 * `stream`; allocates nothing.
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_ALIGNMENT, SKG_ERR_CUDA.
 */
SKG_API skg_status skg_combine_partials(int M, int N, int ranks, const float *const *partials,
                                        const void *residual, void *y, int epilogue, void *stream);

/*
 * skg_plan_set_pdl -- 1 (default): launch with programmatic dependent launch,
 * so a kernel's prologue and its first WEIGHT loads overlap the previous
 * kernel in the stream; x and residual are read, and y written, only after
 * griddepcontrol.wait [VC].  0: plain stream-ordered launch.
 */
SKG_API skg_status skg_plan_set_pdl(skg_plan_t plan, int enable);

/*
 * skg_run -- y = x.W^T (+ residual) on `stream`, one kernel launch.
 *   x        device, bf16 [M,K], 16-byte aligned; read-only
 *   W        device, bf16 [N,K], 16-byte aligned; read-only (static weight)
 *   residual device, bf16 [M,N], or NULL; non-NULL iff the plan's epilogue
 *            is SKG_EPI_BF16_RESIDUAL [OC]
 *   y        device, [M,N], bf16 (fp32 for SKG_EPI_FP32); must not overlap
 *            the inputs
 * Allocates nothing.  Results are bit-identical across runs and across every
 * allowed split of the plan (see SKG_CANONICAL_CHUNKS).
 * Errors: SKG_ERR_INVALID_ARG (NULL plan/tensor, residual mismatch),
 * SKG_ERR_ALIGNMENT, SKG_ERR_DEVICE_TIMEOUT (reported by an earlier launch of
 * this plan), SKG_ERR_CUDA (descriptor encode or launch failure).
 */
SKG_API skg_status skg_run(skg_plan_t plan, const void *x, const void *W,
                   const void *residual, void *y, void *stream);

/*
 * skg_prefetch_l2 -- [PF] on `side_stream`, ask the L2 to fetch the first
 * min(2*N*K, f * L2size) bytes of W_next, the weight of the plan `next`, so
 * that next's skg_run finds them cached.  f = 0.5 unless changed with
 * skg_plan_set_prefetch_fraction; the L2 size is queried from the device
 * when the plan is built.  The kernel only issues bulk L2 prefetches (no
 * data is written); it may run concurrently with any kernel.
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_ALIGNMENT (W_next), SKG_ERR_CUDA.
 */
SKG_API skg_status skg_prefetch_l2(skg_plan_t next, const void *W_next, void *side_stream);

/*
 * skg_plan_set_l2_ahead -- [PF] applied inside a kernel, without shared
 * memory or registers.  TC: before waiting for the previous kernel in the
 * stream, each CTA also requests the `ahead` weight tiles (128 x 64
 * k-blocks) that follow its ring into L2, so the previous kernel's tail
 * keeps HBM busy with this launch's weights.  GEMV split 1 with 16-byte
 * loads (stages 0) or in one wave (stages 3): each batch is also requested
 * into L2 `ahead` batches before it is loaded (the first ones before the
 * wait).  0..64; 0 turns it off.  The GEMV ring kernel (split > 1) and the
 * whole-row bulk-copy form (stages 2) ignore it.
 */
SKG_API skg_status skg_plan_set_l2_ahead(skg_plan_t plan, int ahead);

/*
 * skg_plan_set_reducers -- [TS] the split-K kernel's final reduction of a
 * 128-row tile (its S partial sums combined by the top levels of the
 * canonical tree, the residual added, one rounding) is done by the last R
 * CTAs of the tile to finish, each taking 1/R of the tile's outputs; all but
 * the last wait, with the plan's bounded wait, for the others.  R = 1, 2, 4
 * or 8.  The output bits do not depend on R.  A launch uses min(R, split_k),
 * and 1 at split 16 or while its grid is more than one wave of the CTAs the
 * SMs hold at once (within one wave the waiting CTAs always leave the CTAs
 * they wait for a place); the plan's description reports that count for its
 * current launch shape.  Errors: SKG_ERR_INVALID_ARG (R),
 * SKG_ERR_UNSUPPORTED (a GEMV plan), SKG_ERR_CUDA.
 */
SKG_API skg_status skg_plan_set_reducers(skg_plan_t plan, int reducers);

/*
 * skg_plan_set_next_weight -- [PF] inside the launch instead of on a side
 * stream: every later skg_run of this plan also asks the L2 (evict-last) for
 * the first `bytes` of W_next, the weight of the projection that runs next,
 * each CTA taking its slice once it has requested all of its own weight
 * tiles -- so the next launch finds its first tiles cached and this launch's
 * tail keeps HBM busy.  No extra kernel, stream or dependency is involved.
 * bytes is rounded down to a multiple of 16 and capped at the L2 size;
 * W_next must be 16-byte aligned and stay allocated while the plan runs.
 * W_next == NULL or bytes == 0 turns it off.
 */
SKG_API skg_status skg_plan_set_next_weight(skg_plan_t plan, const void *W_next, size_t bytes);

/* Fraction f in [0, 1] of the L2 that skg_prefetch_l2 fills for this plan. */
SKG_API skg_status skg_plan_set_prefetch_fraction(skg_plan_t plan, double fraction);

/* Copy the plan's launch description into *out. */
SKG_API skg_status skg_plan_info(skg_plan_t plan, skg_plan_desc *out);

/*
 * skg_plan_check -- synchronise the plan's last stream and report whether
 * any of its kernels ran out of a bounded wait since the last check
 * (SKG_ERR_DEVICE_TIMEOUT; the report is then cleared) or a CUDA error is
 * pending (SKG_ERR_CUDA).
 */
SKG_API skg_status skg_plan_check(skg_plan_t plan);

/* Free the plan, its workspace and descriptors (after its work finished). */
SKG_API skg_status skg_plan_destroy(skg_plan_t plan);

/*
 * skg_debug_wait_timeout -- failure-detection self test: launch one CTA that
 * waits on a shared-memory barrier that nothing ever arrives at, bounded by
 * timeout_ns of %globaltimer; on expiry the kernel records the timeout in
 * the plan's error word and returns normally, leaving the context usable.
 * A following skg_plan_check returns SKG_ERR_DEVICE_TIMEOUT.  With plan
 * NULL the timeout is recorded in the word of skg_run_noalloc's fixed array
 * instead, and skg_noalloc_check reports it.
 */
SKG_API skg_status skg_debug_wait_timeout(skg_plan_t plan, unsigned long long timeout_ns,
                                  void *stream);

/*
 * skg_run_noalloc -- the split-K projection (M = 3..64) for callers that may
 * not allocate device memory: runtimes that own the whole device-memory
 * budget, code that must not enter the CUDA allocator, or hosts that cannot
 * create plans (skg_plan allocates).  It takes no plan, allocates nothing, and
 * keeps the kernel's fp32 partials, arrival counters and timeout word in a
 * fixed 16 MiB array inside the library that every GPU loading the library
 * holds until the process exits.  The pages describe no such entry point; it
 * exists only for these callers.
 *   M, N, K, epilogue, x, W, residual, y, stream: as for skg_plan + skg_run.
 *   Limits: M must be 3..64 (M <= 2 needs no scratch: use skg_run); the
 *   partials at the picker's split, split * ceil(N/128) * 128 * M * 4 bytes,
 *   must fit 16 MiB - 64 KiB - 256 bytes, else SKG_ERR_UNSUPPORTED (at
 *   M = 64 that admits N up to 32512, where the picker splits K in 2).
 *   The first call on each device resolves the array's device address
 *   (cudaGetSymbolAddress) and keeps it for the life of the process: make
 *   that first call before any stream capture, and do not reset the device
 *   (cudaDeviceReset) after it.
 *   Every call clears the counters (cudaMemsetAsync on `stream`) and then
 *   launches one kernel, with the same L2 look-ahead as the plan path;
 *   results are bit-identical to skg_run's.  All calls share the one array,
 *   so calls that overlap on the GPU (other streams, or other threads) race:
 *   serialise them.  A bounded wait that runs out stops the kernel, leaves y
 *   incomplete and sets the array's timeout word, which skg_noalloc_check
 *   reports.
 * Errors: as skg_run, except that an earlier timeout is reported only by
 * skg_noalloc_check.
 */
SKG_API skg_status skg_run_noalloc(int M, int N, int K, int epilogue, const void *x, const void *W,
                                   const void *residual, void *y, void *stream);

/*
 * skg_noalloc_check -- synchronise `stream`, then report whether any kernel
 * launched by skg_run_noalloc on the current device ran out of a bounded
 * wait since the last check (SKG_ERR_DEVICE_TIMEOUT: the output of that call
 * is incomplete; the word is then cleared), or a CUDA error is pending
 * (SKG_ERR_CUDA).  Allocates nothing (a 4-byte device-to-host copy and, after
 * a timeout, a 4-byte clear).
 */
SKG_API skg_status skg_noalloc_check(void *stream);

/* Message of the last failed call on this thread ("" if none). */
SKG_API const char *skg_last_error(void);

/* SKG_VERSION of the loaded library. */
SKG_API int skg_version(void);

/*
 * Groups -- several projections of the same M (1..64) in one persistent
 * split-K launch.  [OC] fuses producer and consumer in one kernel across
 * GPUs; this is the one-GPU form of that idea: the launch's CTAs take the
 * work units (projection, 128-row tile, split) from a counter in projection
 * order (so the launch completes with any part of its grid resident), keep
 * their TMA ring, TMEM and barriers from one unit to the next, and stream
 * the next projection's weights while the previous one is still being
 * reduced, so consecutive projections pay no launch head or tail between
 * them.  Each projection's output has the bits of skg_run on the split-K
 * kernel at the same split (splits above 8 are lowered to 8: any split gives
 * the same bits; at M <= 2 that is the plan after
 * skg_plan_force_kernel(SKG_KERNEL_SPLITK_TC)).
 *
 * skg_group -- plan n (1..8) projections: N[i], K[i] and epilogue[i] as for
 * skg_plan; dep[i] (i >= 1; dep may be NULL for none) = 1: projection i
 * reads its x and residual only after projection i - 1 has written all of
 * its y (an on-device counter, bounded wait) -- set it whenever projection
 * i consumes projection i - 1's output.  Projections without dep read their
 * inputs with no ordering against the rest of the group, so their x,
 * residual and y must not be written by another projection of the group.
 * Projection 0 reads x only after the previous kernel in the stream
 * (programmatic dependent launch, as skg_run).  Allocates the partials and
 * counters of every projection.  Errors: SKG_ERR_INVALID_ARG,
 * SKG_ERR_UNSUPPORTED (n, M or a shape outside the limits), SKG_ERR_CUDA.
 */
typedef struct skg_group_s *skg_group_t;
SKG_API skg_status skg_group(int n, int M, const int *N, const int *K, const int *epilogue, const int *dep,
                             skg_group_t *out);

/*
 * skg_group_run -- enqueue the group on `stream`: x[i] bf16 [M, K[i]], W[i]
 * bf16 [N[i], K[i]], residual[i] bf16 [M, N[i]] or NULL (the residual array
 * itself may be NULL when no epilogue takes one), y[i] [M, N[i]] bf16 (fp32
 * for SKG_EPI_FP32); x[i] and W[i] 16-byte aligned.  Allocates nothing.
 * One run of a group may be in flight at a time.  After a device timeout
 * (SKG_ERR_DEVICE_TIMEOUT from a later run or skg_group_check) the group's
 * counters are inconsistent: destroy it.
 */
SKG_API skg_status skg_group_run(skg_group_t group, const void *const *x, const void *const *W,
                                 const void *const *residual, void *const *y, void *stream);

/* Launch shape: CTAs, ring stages, work units, and each projection's split (n ints). */
SKG_API skg_status skg_group_info(skg_group_t group, int *grid, int *stages, int *units, int *split);

/* Synchronize the group's last stream and report a device timeout, if any. */
SKG_API skg_status skg_group_check(skg_group_t group);

/* Free the group (after its work finished). */
SKG_API skg_status skg_group_destroy(skg_group_t group);

/*
 * The 8-bit path -- W8A8 projections of a decode layer or a prompt: weights and
 * activations as 8-bit integers, half the weight bytes of skg_run.
 *
 *   rows:        q[m,k] in [-127, 127] (int8) with one fp32 scale per row m;
 *                q[m,k] * scale[m] is the value it stands for.
 *   projection:  y[m,n] = x_scale[m] * w_scale[n] * sum_k x[m,k] W[n,k]  (+ residual[m,n])
 *
 * Activations are rows per token (skg_rmsnorm_q8, skg_quantize_q8); a weight
 * [N,K] is quantised once, rows per output channel, by skg_quantize_q8 too.
 * These are serving operators: they have no gradients.
 *
 * Quantising a row v: scale = max|v| / 127, q = v * (127 / max|v|) rounded to
 * the nearest integer, half to even.  A row of zeros has scale 0 and q = 0.  A
 * row with a value that is not finite (NaN, infinity) has scale NaN and q = 0:
 * a projection of that row is NaN, and no other row is affected.
 * Rows of any length can be quantised; a projection takes K in multiples of 16, so
 * rows that are to be projected are made that long, with zeros, before.
 *
 * skg_rmsnorm_q8 -- residual addition, root-mean-square norm and quantisation
 * of M >= 0 rows of any length K >= 1, in one kernel on `stream`:
 *     h = x + residual (or x);   v = h / sqrt(mean(h^2) + eps) * gamma
 * h and v are fp32; where they are within its range the norm is right whatever
 * their squares are, for any eps >= 0.  (With eps = 0 a row of zeros is 0 / 0: scale
 * NaN, q = 0.)
 *   x        bf16 [M, K], row stride ldx >= K elements; read-only
 *   residual bf16 [M, K], row stride ldr >= K, or NULL
 *   gamma    bf16 [K], or NULL for ones
 *   h        bf16 [M, K], row stride ldh >= K, or NULL: the sum, rounded once
 *            (the norm goes on from the unrounded sum); only with a residual.
 *            May be the residual itself (same address and stride), or x
 *   y        bf16 [M, K] dense, or NULL: v rounded once, for a bf16 projection
 *   q, scale int8 [M, K] dense and fp32 [M]: the quantised rows of v
 *   Any alignment the element types allow; 16-byte aligned rows are fastest.
 *   M == 0 launches nothing.  Outputs must not overlap inputs except h as said.
 * Errors: SKG_ERR_INVALID_ARG (sizes, strides, NULL, eps negative or not
 * finite, h without residual), SKG_ERR_ALIGNMENT, SKG_ERR_CUDA.
 */
SKG_API skg_status skg_rmsnorm_q8(int M, int K, float eps, const void *x, size_t ldx, const void *residual,
                                  size_t ldr, const void *gamma, void *h, size_t ldh, void *y, void *q,
                                  float *scale, void *stream);

/*
 * skg_quantize_q8 -- the rows of x, or of silu(gate) * x with
 * silu(g) = g / (1 + exp(-g)), quantised as above: M >= 0 rows of any K >= 1.
 *   x, gate  bf16 [M, K], row strides ldx, ldg >= K; gate may be NULL.  Both may
 *            be halves of one [M, 2K] tensor
 *   q, scale int8 [M, K] dense and fp32 [M]
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_ALIGNMENT, SKG_ERR_CUDA.
 */
SKG_API skg_status skg_quantize_q8(int M, int K, const void *x, size_t ldx, const void *gate, size_t ldg, void *q,
                                   float *scale, void *stream);

typedef enum skg_q8_kernel_kind {
    SKG_Q8_KERNEL_STREAM = 1,   /* M <= 16: W streams into registers, warp-level fp16 MMA, exact */
    SKG_Q8_KERNEL_SPLIT = 2,    /* M > 8, few tiles: TMA + tcgen05 on integers widened to fp16, exact; K split
                                   over the CTAs of a cluster, joined in shared memory */
    SKG_Q8_KERNEL_WIDE = 3      /* M > 8, many tiles: the same arithmetic by pairs of CTAs, over whole tiles or
                                   with K split over the pairs of a cluster */
} skg_q8_kernel_kind;

/* What an 8-bit plan will launch. */
typedef struct skg_q8_plan_desc {
    int kernel_kind;            /* skg_q8_kernel_kind */
    int M, N, K, epilogue;
    int static_weights;         /* see skg_q8_plan */
    int m_tile;                 /* tokens per tile (STREAM: 8 or 16; SPLIT: 32 or 64; WIDE: 128) */
    int n_tile;                 /* output channels per tile (STREAM: 16 or 32; SPLIT: 128; WIDE: 256, a pair's) */
    int tiles;                  /* output tiles */
    int split_k;                /* parts of a tile's K: CTAs of a cluster (SPLIT: 1..8) or pairs of them (WIDE: 1..4); STREAM: 1 */
    int grid, threads, smem_bytes, stages, ctas_per_sm;
    size_t workspace_bytes;     /* SPLIT: sums put away where a CTA has more than 2048 k; else 0 */
} skg_q8_plan_desc;

typedef struct skg_q8_plan_s *skg_q8_plan_t;

/*
 * skg_q8_plan_query -- the launch of an 8-bit projection on a GPU with num_sms
 * SMs, without touching any GPU.  1 <= M <= 262144 tokens, N >= 1, K a multiple
 * of 16 in [16, 131056] (so that no sum of K products of 8-bit integers can
 * leave 32 bits), epilogue as for skg_plan.
 * Errors: SKG_ERR_INVALID_ARG (M, N, num_sms, epilogue, NULL),
 * SKG_ERR_UNSUPPORTED (K, M above the limits, or more than 2^27 tiles).
 */
SKG_API skg_status skg_q8_plan_query(int M, int N, int K, int epilogue, int num_sms, skg_q8_plan_desc *out);

/*
 * skg_q8_plan -- build a plan for (M,N,K,epilogue) on the current device.
 * static_weights != 0 promises that W and w_scale of every skg_q8_run were
 * written long before it: by work that had completed before the kernel that
 * precedes the run in its stream was launched.  The run may then request weight
 * bytes while that kernel still finishes.  0: everything is read after it.
 * Allocates the launch's workspace and a mapped host word for device-side error
 * reports; free the plan with skg_q8_plan_destroy.
 * Errors: as skg_q8_plan_query, plus SKG_ERR_CUDA.  *out is NULL on failure.
 */
SKG_API skg_status skg_q8_plan(int M, int N, int K, int epilogue, int static_weights, skg_q8_plan_t *out);

/*
 * skg_q8_run -- the 8-bit projection on `stream`.
 *   x        int8 [M,K] dense, 16-byte aligned; x_scale fp32 [M]
 *   W        int8 [N,K] dense, 16-byte aligned; w_scale fp32 [N]
 *   residual bf16 [M,N], non-NULL iff the epilogue is SKG_EPI_BF16_RESIDUAL
 *   y        [M,N] bf16 (fp32 for SKG_EPI_FP32); must not overlap the inputs
 * The sum over k is the exact integer, so the result does not depend on the
 * launch shape; it is scaled in fp32 as (sum * x_scale) * w_scale, the residual
 * is added in fp32, and the result is rounded once.
 * Allocates nothing.  One run of a plan may be in flight at a time (the
 * workspace is shared); concurrent streams need separate plans.
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_ALIGNMENT, SKG_ERR_DEVICE_TIMEOUT
 * (reported by an earlier launch of this plan), SKG_ERR_CUDA.
 */
SKG_API skg_status skg_q8_run(skg_q8_plan_t plan, const void *x, const float *x_scale, const void *W,
                              const float *w_scale, const void *residual, void *y, void *stream);

/*
 * skg_q8_plan_force -- override of the kernel choice (tests and measurements):
 * kind (an skg_q8_kernel_kind, 0 keeps; STREAM: M <= 16), m_tile (SPLIT: 32, 64;
 * WIDE: 128; 0 = chosen) and split_k (SPLIT: 1..8, WIDE: 1..4, no finer than
 * K / 128; 0 = chosen).  Results do not change.  A larger workspace is allocated where
 * needed and the old one kept until the plan is destroyed, as by skg_plan_force.
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_UNSUPPORTED, SKG_ERR_CUDA.
 */
SKG_API skg_status skg_q8_plan_force(skg_q8_plan_t plan, int kind, int m_tile, int split_k);

/* Copy the plan's launch description into *out. */
SKG_API skg_status skg_q8_plan_info(skg_q8_plan_t plan, skg_q8_plan_desc *out);

/* Synchronise the plan's last stream and report a bounded wait that ran out
 * since the last check (SKG_ERR_DEVICE_TIMEOUT, then cleared) or a pending CUDA
 * error, as skg_plan_check.  skg_q8_run reports such a timeout too. */
SKG_API skg_status skg_q8_plan_check(skg_q8_plan_t plan);

/* skg_debug_wait_timeout with the word of an 8-bit plan. */
SKG_API skg_status skg_q8_debug_wait_timeout(skg_q8_plan_t plan, unsigned long long timeout_ns, void *stream);

/* Free the plan (after its work finished). */
SKG_API skg_status skg_q8_plan_destroy(skg_q8_plan_t plan);

/*
 * The 8-bit floating point path -- projections of e4m3 numbers with an fp32 scale
 * for each block of 128: for tokens and weights whose range one scale a row does
 * not serve, of one weight or of the experts that the tokens go to.
 *
 *   activations:  q[m,k] e4m3, scale[m, k / 128]:          q * scale is the value
 *   weights:      q[n,k] e4m3, scale[n / 128, k / 128]
 *   projection:   y[m,n] = sum_b x_scale[m,b] w_scale[n / 128, b]
 *                          sum_(k in block b) x[m,k] W[n,k]   (+ residual[m,n])
 *
 * (Divisions of indexes round down; the last block of a row or column is short
 * where 128 does not divide it.)  These are serving operators: no gradients.
 *
 * These calls, and those of the experts' tokens below, launch on the current device,
 * on which the stream and every pointer have to be.  (The Python binding refuses
 * tensors of another device than the current one.)
 *
 * Quantising a block of values v (fp32): scale = max|v| / 448, q = e4m3(v * f) with
 * f = 448 / max|v|, each operation rounded to fp32 and the product to e4m3, half
 * to even.  A block of zeros has scale 0 and q = 0.  A block with a value that is
 * not finite has scale NaN and q = 0: a projection that reads it is NaN.
 *
 * skg_quantize_f8 -- M >= 0 rows of any K in [1, 2^30]: of x, or of silu(gate) * x with
 * silu(g) = g / (1 + exp(-g)); or row i of the output from row rows[i] of those.
 *   x, gate  bf16 rows of K, row strides ldx, ldg >= K; gate may be NULL.  Both may
 *            be halves of one [M, 2K] tensor
 *   rows     int32 [M], or NULL.  With rows, x and gate have x_rows >= 0 rows, and
 *            an index outside [0, x_rows) gives a row of q = 0, scale = 0.  Without,
 *            they have M, and x_rows is not read
 *   q, scale e4m3 [M, K] and fp32 [M, ceil(K / 128)], dense
 *   Any alignment the element types allow; 16-byte aligned rows are fastest.
 *   q and scale must not overlap the inputs.
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_UNSUPPORTED, SKG_ERR_ALIGNMENT, SKG_ERR_CUDA.
 */
SKG_API skg_status skg_quantize_f8(int M, int K, const void *x, size_t ldx, const void *gate, size_t ldg, const int *rows,
                                   int x_rows, void *q, float *scale, void *stream);

/*
 * skg_quantize_f8_weights -- weights W bf16 [experts, N, K] (experts = 1 for one
 * weight), dense, to q e4m3 of the same shape and scale fp32 [experts,
 * ceil(N / 128), ceil(K / 128)].
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_ALIGNMENT, SKG_ERR_UNSUPPORTED (more than
 * 2^31 - 1 blocks, K above 2^30), SKG_ERR_CUDA.
 */
SKG_API skg_status skg_quantize_f8_weights(int experts, int N, int K, const void *W, void *q, float *scale, void *stream);

typedef enum skg_f8_kernel_kind {
    SKG_F8_KERNEL_SPLIT = 1,    /* few tokens (of each expert): 128 channels x m_tile tokens, K split over the CTAs of
                                   a cluster, joined in shared memory */
    SKG_F8_KERNEL_WIDE = 2      /* many: 128 x 128, or 256 tokens x 256 channels by pairs of CTAs, K split in the same way */
} skg_f8_kernel_kind;

/* What a plan of the 8-bit floating point path will launch. */
typedef struct skg_f8_plan_desc {
    int kernel_kind;            /* skg_f8_kernel_kind */
    int M, N, K, epilogue;
    int experts;                /* 0: one weight */
    int static_weights;         /* see skg_f8_plan */
    int m_tile, n_tile;         /* tokens and channels of a tile */
    int tiles;                  /* output tiles; with experts the most that offsets can ask for */
    int split_k;                /* CTAs (or pairs of them) that share a tile's K: SPLIT 1..8, WIDE 1..4 */
    int grid, threads, smem_bytes, stages, ctas_per_sm;
} skg_f8_plan_desc;

typedef struct skg_f8_plan_s *skg_f8_plan_t;

/*
 * skg_f8_plan_query -- the launch of a projection on a GPU with num_sms SMs,
 * without touching any GPU.  1 <= M <= 2^20 rows, N >= 1, K a multiple of 16 in
 * [16, 131072], epilogue as for skg_plan, experts in [0, 1024].
 * Errors: SKG_ERR_INVALID_ARG (M, N, num_sms, experts, epilogue, NULL),
 * SKG_ERR_UNSUPPORTED (K, M or experts above the limits, more than 2^31 - 256
 * channels of all experts, or more than 2^27 tiles).
 */
SKG_API skg_status skg_f8_plan_query(int M, int N, int K, int epilogue, int experts, int num_sms, skg_f8_plan_desc *out);

/*
 * skg_f8_plan -- build a plan on the current device.  experts = 0: every row by one
 * weight.  experts = E > 0: rows sorted by expert, rows offsets[e] to
 * offsets[e + 1] by weight e.  static_weights as for skg_q8_plan (with experts it
 * changes nothing: which weight comes first is known from offsets).  Allocates a
 * mapped host word for device-side error reports and no device memory; free the
 * plan with skg_f8_plan_destroy.
 * Errors: as skg_f8_plan_query, plus SKG_ERR_CUDA.  *out is NULL on failure.
 */
SKG_API skg_status skg_f8_plan(int M, int N, int K, int epilogue, int experts, int static_weights, skg_f8_plan_t *out);

/*
 * skg_f8_run -- the projection on `stream`.
 *   x        e4m3 [M,K] dense, 16-byte aligned; x_scale fp32 [M, ceil(K / 128)]
 *   W        e4m3 [N,K], or [E,N,K], dense, 16-byte aligned; w_scale fp32
 *            [ceil(N / 128), ceil(K / 128)], or [E, ...] of that
 *   residual bf16 [M,N], non-NULL iff the epilogue is SKG_EPI_BF16_RESIDUAL
 *   offsets  int32 [E + 1] on the device, ascending within [0, M], non-NULL iff the
 *            plan has experts (as skg_experts_sort writes them).  Rows before the
 *            first and behind the last of them are left as they were in y.  Other
 *            numbers are taken as the nearest that are allowed, in order
 *   y        [M,N] bf16 (fp32 for SKG_EPI_FP32); must not overlap the inputs
 * Sums of products and over blocks are fp32, a block's two scales are multiplied in
 * fp32 before they meet its sum (their product should be a normal number), the
 * residual is added in fp32, and the result is rounded once.  The order of the sum
 * over blocks depends on the launch shape: a plan gives the same bits each time,
 * and a row's result does not depend on the other rows.
 * Allocates nothing and keeps no workspace: runs of a plan may be in flight at the
 * same time.  The plan's device must be the current one.
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_ALIGNMENT, SKG_ERR_DEVICE_TIMEOUT
 * (reported by an earlier launch of this plan), SKG_ERR_CUDA.
 */
SKG_API skg_status skg_f8_run(skg_f8_plan_t plan, const void *x, const float *x_scale, const void *W, const float *w_scale,
                              const void *residual, const int *offsets, void *y, void *stream);

/*
 * skg_f8_plan_force -- override of the kernel choice (tests and measurements):
 * kind (an skg_f8_kernel_kind, 0 keeps), m_tile (SPLIT: 16, 32, 64; WIDE: 128, 256;
 * 0 = chosen) and split_k (SPLIT: 1..8, WIDE: 1..4, no finer than K / 128; 0 =
 * chosen).
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_UNSUPPORTED.
 */
SKG_API skg_status skg_f8_plan_force(skg_f8_plan_t plan, int kind, int m_tile, int split_k);

/* Copy the plan's launch description into *out. */
SKG_API skg_status skg_f8_plan_info(skg_f8_plan_t plan, skg_f8_plan_desc *out);

/* As skg_q8_plan_check. */
SKG_API skg_status skg_f8_plan_check(skg_f8_plan_t plan);

/* skg_debug_wait_timeout with the word of this plan. */
SKG_API skg_status skg_f8_debug_wait_timeout(skg_f8_plan_t plan, unsigned long long timeout_ns, void *stream);

/* Free the plan (after its work finished). */
SKG_API skg_status skg_f8_plan_destroy(skg_f8_plan_t plan);

/*
 * Tokens to their experts and back.  T tokens choose k experts each; the T * k
 * choices become R = T * k rows, sorted by expert.  Outputs must not overlap
 * inputs except as said.
 *
 * skg_experts_sort -- from expert int32 [T, k]:
 *   offsets  int32 [experts + 1]: expert e has the sorted rows offsets[e] to offsets[e + 1]
 *   rows     int32 [T * k]: the token of each sorted row; -1 behind the last
 *   pos      int32 [T, k]: the sorted row of each choice; -1 where expert[t, j] is
 *            outside [0, experts), a choice that goes nowhere
 * Rows of an expert are in the order of their choices (t, then j).  The same expert
 * twice makes two rows.  One launch.  T >= 0, k >= 1, 1 <= experts <= 1024, T * k
 * <= 2^24.
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_UNSUPPORTED, SKG_ERR_ALIGNMENT, SKG_ERR_CUDA.
 */
SKG_API skg_status skg_experts_sort(int T, int k, int experts, const int *expert, int *offsets, int *rows, int *pos,
                                    void *stream);

/*
 * skg_experts_gather -- out[p] = x[rows[p]] for R >= 0 rows, zeros where rows[p] is
 * outside [0, T).  Its gradient is skg_experts_combine without weights.
 *   x bf16 [T, N], row stride ldx >= N; rows int32 [R]; out bf16 [R, N] dense; N <= 2^30
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_UNSUPPORTED, SKG_ERR_ALIGNMENT, SKG_ERR_CUDA.
 */
SKG_API skg_status skg_experts_gather(int R, int T, int N, const void *x, size_t ldx, const int *rows, void *out, void *stream);

/*
 * skg_experts_combine -- out[t] = residual[t] + sum_j weight[t,j] y[pos[t,j]], in
 * fp32 in the order of j, rounded once.  A choice whose pos is outside [0, R) is
 * left out, whatever its weight; a token without any has its residual, or zeros.
 *   y bf16 [R, N], row stride ldy >= N; pos int32 [T, k]; weight fp32 [T, k], or
 *   NULL for ones; residual bf16 [T, N] dense, or NULL; out bf16 [T, N] dense, which
 *   may be the residual.  N <= 2^30, T * k < 2^31
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_UNSUPPORTED, SKG_ERR_ALIGNMENT, SKG_ERR_CUDA.
 */
SKG_API skg_status skg_experts_combine(int T, int k, int R, int N, const void *y, size_t ldy, const int *pos,
                                       const float *weight, const void *residual, void *out, void *stream);

/*
 * skg_experts_combine_grad -- gradients of skg_experts_combine with weights:
 *   grad_y[pos[t,j]] = weight[t,j] grad_out[t], rounded once; rows that no choice
 *                    goes to are left as they were.  bf16 [R, N] dense
 *   grad_weight[t,j] = <grad_out[t], y[pos[t,j]]>, fp32, 0 where a choice was left out
 *   grad_out bf16 [T, N] dense; the others as for skg_experts_combine.  (The
 *   residual's gradient is grad_out itself.)  grad_y may be y where ldy = N
 * From grad_y a program goes on through the projections that it trains; the 8-bit
 * ones above have no gradients.
 * A sorted row belongs to one choice: where pos has the same row twice, each element
 * of grad_y is of one of the two (and where grad_y is y, their grad_weight may be of
 * a row that has been written already).
 * Errors: SKG_ERR_INVALID_ARG, SKG_ERR_UNSUPPORTED, SKG_ERR_ALIGNMENT, SKG_ERR_CUDA.
 */
SKG_API skg_status skg_experts_combine_grad(int T, int k, int R, int N, const void *grad_out, const void *y, size_t ldy,
                                            const int *pos, const float *weight, void *grad_y, float *grad_weight,
                                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SKG_H */
