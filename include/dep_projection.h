/*
 * dep_projection.h -- C ABI of the GB300 (sm_103a) decode projection library.
 *
 * The operation.  One decode-time linear layer at tensor-parallel degree 1:
 *
 *     y[B,N] = BF16( x[B,K] . W[N,K]^T ),  BF16 inputs, FP32 accumulation.
 *
 * Source: vllm.models.kimi_k3.nvidia.specialized_decode.runtime.dep (the
 * "runtime.dep page"), class DepProjection: a TP1 linear that runs split-K at the
 * batches its tactic table names and the stock FP32-accumulated BF16 GEMM
 * (torch.mm(x, W.t(), out=out)) otherwise; the module overview's precision
 * paragraph: BF16 outputs, FP32 accumulation, a split-K order that differs from
 * the stock one.  The weights it serves are the packed DSA input projection
 * (14560 x 7168), o_proj (7168 x 12288) and the packed KDA input projection
 * (49376 x 7168), streamed whole once per decode step.
 *
 * Plans.  A plan is built once per weight shape (N, K) and set of batch sizes,
 * like DepProjection.__init__ (runtime.dep page), and holds a tactic table keyed
 * by "max rows" (runtime.dep page, _bins and dep_policies).  At run time a batch
 * of B rows takes the entry with the smallest key >= B, else the entry with the
 * largest key.  Every tactic accepts any B >= 1 (wider batches run in passes).
 *
 * Layouts.  x is [B,K], W is [N,K] (the nn.Linear weight), y is [B,N]; all three
 * are row-major, contiguous, BF16, in device memory of the plan's device, and
 * 16-byte aligned.  K must be a multiple of 8 (16-byte rows).  N is any value
 * >= 1.  y must not overlap x or W.  The caller owns x, W and y; the library
 * neither retains nor repacks W.
 *
 * Determinism.  Each tactic sums in one fixed order with a fixed-order
 * cross-block split-K reduction and no floating-point atomics: the same call on
 * the same plan gives the same bits every time.
 *
 * Errors.  Every call returns a dep_status_t; nothing aborts or throws across
 * the ABI.  Launch failures are reported as DEP_ERR_CUDA.
 *
 * Concurrency.  A plan owns one split-K workspace.  Two runs of the same plan
 * must not overlap on the GPU (use one plan per stream).  Runs are asynchronous
 * on the given stream, allocate nothing and do not synchronise, so they can be
 * captured in CUDA graphs (the runtime package page, specialized_decode_config:
 * the deployment's decode batches are its CUDA-graph capture sizes).
 */
#ifndef DEP_PROJECTION_H
#define DEP_PROJECTION_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque plan handle, owned by the library (free with dep_projection_plan_destroy). */
typedef struct dep_plan_s *dep_plan_t;

typedef enum {
    DEP_OK = 0,
    DEP_ERR_INVALID_ARG = 1,  /* null pointer, bad size, unknown tactic, wrong device */
    DEP_ERR_UNSUPPORTED = 2,  /* shape or plan kind this build cannot run */
    DEP_ERR_MISALIGNED = 3,   /* a pointer not 16-byte aligned, or K % 8 != 0 */
    DEP_ERR_CUDA = 4,         /* a CUDA runtime/driver call or a launch failed */
    DEP_ERR_OOM = 5,          /* plan-time device allocation failed */
    DEP_ERR_TIMEOUT = 6,      /* a kernel gave up a bounded wait (device status) */
    DEP_ERR_INTERNAL = 7,     /* an invariant of the library was broken */
    DEP_ERR_IO = 8            /* plan file could not be read or written, or is malformed */
} dep_status_t;

/* Tactic kinds. */
#define DEP_KIND_SPLITK_FMA 1 /* warp split-K on the FP32 FMA pipe, TMA-staged W */
#define DEP_KIND_TC 2         /* tcgen05 MMA, TMEM accumulators, TMA-staged W and x */
#define DEP_KIND_ROWS 3       /* warp split-K over whole weight rows, dynamic tiles, no
                                 cross-block fix-up; x resident in shared memory */
#define DEP_KIND_TC_SPLIT 4   /* tcgen05 MMA over (tile, K piece) items taken
                                 dynamically; tiles of tile_n = 64 or 128 weight rows
                                 (MMA M), each cut into `splits` fixed K pieces whose
                                 FP32 partials are added in piece order */
#define DEP_KIND_TC_WIDE 5    /* tcgen05 MMA for wide batches: each block streams a
                                 group of tile_n / 128 = 2 or 4 weight tiles of 128
                                 rows against every x slice (one MMA per tile, the
                                 same x operand), stream-K over (group, k-tile)
                                 units; split groups are reduced by the blocks
                                 that share them, each a part of the columns, adding
                                 the blocks' FP32 partials in block order */
#define DEP_KIND_TC_CLUSTER 6 /* tcgen05 MMA for wide batches: a thread-block cluster
                                 of `splits` = k CTAs per group of weight tiles --
                                 tile_n = 256 or 512 rows (2 or 4 tiles of 128), or
                                 192 rows (a 128-row and a 64-row tile) -- one MMA
                                 per tile with the same x operand, CTA rank r
                                 streaming K piece r; the K
                                 pieces are added in rank order through distributed
                                 shared memory (no global workspace); `stages` =
                                 weight stages (x has its own 2-4 stage ring);
                                 `ctas` = a multiple of k; tile_k = 64 */
#define DEP_KIND_TC_XM 7      /* tcgen05 MMA for wide batches with x on the MMA's M
                                 side: blocks of 128 batch rows (cols = 128 or 256:
                                 one or two per pass) against tiles of tile_n weight
                                 rows (MMA N, a multiple of 16 up to 256), dealt out
                                 statically over `ctas` blocks; splits = 0: each
                                 block sums its tiles' whole K; splits = 2: a
                                 thread-block cluster of two per tile (tile_n a
                                 multiple of 32, ctas even), each half of K, the
                                 halves added in order through distributed shared
                                 memory; no workspace either way; `stages` of
                                 tile_k = 64, 128 or 256 columns of the weight and
                                 of x */
#define DEP_KIND_WARP_MMA 8   /* warp-level mma.sync for small weights at up to 16
                                 rows: one block per tile of tile_n = 16 weight
                                 rows and whole K (splits = 0 or 1), or a cluster of
                                 splits = 2 or 4 blocks per tile, each a K piece,
                                 added in rank order in the first block's shared
                                 memory; cols = 16 batch rows per pass, stages of
                                 tile_k = 64, 128 or 256 columns; no tensor memory,
                                 a small ring, so several blocks (of one call and
                                 of the next) share an SM; `ctas` is not used */

/* One table entry: the tactic that serves batches of up to max_rows rows. */
typedef struct {
    int32_t max_rows; /* table key (binning rule above) */
    int32_t kind;     /* DEP_KIND_* */
    int32_t ctas;     /* persistent blocks launched (FMA/TC/TC_WIDE: work split
                         evenly, stream-K; ROWS/TC_SPLIT: work items taken
                         dynamically) */
    int32_t tile_n;   /* weight rows per tile (TC_WIDE: per group, 256 or 512;
                         TC_CLUSTER: per group, 192, 256 or 512; TC_XM: MMA N) */
    int32_t tile_k;   /* reduction columns per pipeline stage */
    int32_t stages;   /* pipeline depth (shared-memory stages) */
    int32_t cols;     /* batch rows per pass (FMA/ROWS: x rows held; TC: MMA N;
                         TC_XM: 128 or 256, MMA M = 128 per block of rows) */
    int32_t splits;   /* TC_SPLIT: K pieces per tile, 1..64 (capped at the tile's
                         k-tiles, ceil(K / tile_k)); TC_CLUSTER: CTAs per cluster;
                         TC_XM: 0, or 2 for pairs of blocks; WARP_MMA: K pieces
                         per tile, 0/1, 2 or 4; 0 for the other kinds */
} dep_tactic_t;

/* Plan flags. */
#define DEP_PLAN_DEFAULT 0u /* fixed rule: FMA split-K for small batches, TC past them */
#define DEP_PLAN_TUNE 1u    /* time candidate tactics per batch on scratch data; keep the fastest */
/* Programmatic dependent launch: each run may start while the preceding kernel
 * in its stream finishes, streaming its first weight tiles early and waiting for
 * that kernel before it reads x or writes y.  The caller promises that no work
 * enqueued before a run on the same stream writes W (decode weights are
 * read-only).  Consecutive runs then overlap one kernel's tail with the next
 * one's ramp-up, also inside CUDA graphs. */
#define DEP_PLAN_PDL 2u
/* Inspection: the wide-batch kernel (DEP_KIND_TC_WIDE) also stores the partials
 * each block reduces itself, so that dep_projection_plan_partials returns every
 * block's piece of every split group (extra writes; same results). */
#define DEP_PLAN_KEEP_PIECES 4u

/*
 * Build a plan for weights of shape [N,K] on the current CUDA device.
 *   batches/n_batches: the batch sizes the caller will run (the table's keys);
 *                      n_batches == 0 takes 1,2,4,8,16,32,64,128,256.
 *   flags:             DEP_PLAN_DEFAULT, or DEP_PLAN_TUNE and/or DEP_PLAN_PDL.
 * Allocates the plan's workspace, counters and status word on the device.
 * Errors: INVALID_ARG (N < 1, K < 8, batch < 1, null out), MISALIGNED (K % 8),
 * OOM, CUDA.  On error *out is set to NULL.
 */
dep_status_t dep_projection_plan(int64_t N, int64_t K, const int32_t *batches,
                                 int32_t n_batches, uint32_t flags, dep_plan_t *out);

/*
 * Build the default table for an explicit SM count without touching any GPU:
 * for inspection, saving, and host-side tests.  Running such a plan returns
 * DEP_ERR_UNSUPPORTED.  Errors as dep_projection_plan, plus INVALID_ARG for
 * sm_count < 1.
 */
dep_status_t dep_projection_plan_host(int64_t N, int64_t K, const int32_t *batches,
                                      int32_t n_batches, int32_t sm_count,
                                      dep_plan_t *out);

/*
 * y[B,N] = BF16(x[B,K] . W[N,K]^T) on `stream` (a cudaStream_t; NULL = legacy
 * default stream).  The tactic is the plan's table entry for B (binning rule).
 * B == 0 launches nothing and returns DEP_OK; B < 0 is INVALID_ARG.
 * Asynchronous: returns after enqueueing.  Errors: INVALID_ARG (null pointer,
 * overlap of y with x or W, current device is not the plan's), MISALIGNED,
 * UNSUPPORTED (host-only plan), CUDA (launch failure).
 */
dep_status_t dep_projection_run(dep_plan_t plan, const void *x, const void *W, void *y,
                                int32_t B, void *stream);

/*
 * The same with an explicit tactic instead of the table's (tests and tuning).
 * Errors as dep_projection_run, plus INVALID_ARG for a tactic this build does
 * not implement or whose split-K workspace exceeds the plan's, and UNSUPPORTED
 * for a grid the device cannot hold at once in a kind whose blocks wait on one
 * another (DEP_KIND_TC, DEP_KIND_TC_SPLIT, DEP_KIND_TC_WIDE: at most
 * (blocks resident per SM) x (SM count) blocks).
 */
dep_status_t dep_projection_run_tactic(dep_plan_t plan, const dep_tactic_t *tactic,
                                       const void *x, const void *W, void *y,
                                       int32_t B, void *stream);

/*
 * End-to-end call with the activations in host memory: brings x_host [B,K] to
 * the plan's device staging buffer, runs the projection against the resident
 * device weight W, and puts y back to y_host [B,N], all enqueued on `stream`.
 * The caller synchronises the stream before reading y_host.  B must not exceed
 * the plan's largest table key (the staging capacity).  Errors as
 * dep_projection_run.
 *   - Pinned host buffers (mapped into the device's address space, 16-byte
 *     aligned): a small kernel reads x_host directly (zero-copy) into the
 *     staging buffer, chained to the projection by programmatic dependent
 *     launch, so the projection streams its first weight stages while x
 *     arrives and consecutive calls leave no launch gap.  The projection
 *     stores y straight into y_host, except the cluster and x-on-M kinds
 *     (DEP_KIND_TC_CLUSTER, DEP_KIND_TC_XM), whose y a second small kernel
 *     copies back from the staging buffer.
 *     Stream order holds as for memcpys: each copy reads only after the
 *     preceding work in the stream has completed, so one call's y_host may be
 *     the next call's x_host.
 *   - Any other host memory: cudaMemcpyAsync both ways.
 *   Both give the same bits as dep_projection_run.  The environment variable
 *   DEP_STAGING=copy forces the copy path, DEP_STAGING=stage the copy-back of
 *   y for every kind (both for comparisons).
 */
dep_status_t dep_projection_run_host(dep_plan_t plan, const void *x_host, const void *W,
                                     void *y_host, int32_t B, void *stream);

/*
 * No counterpart in the pages: an addition of this library for callers that
 * must not allocate device memory -- code running inside a device-memory
 * allocator or pool (allocating there would re-enter it), hosts that reserve
 * all device memory up front and allow no other allocation, and latency-bound
 * paths that cannot afford cudaMalloc's implicit synchronisation.  They cannot
 * build a plan, since a plan allocates its workspace.
 *
 * y[B,N] = BF16(x[B,K] . W[N,K]^T) with the split-K FMA kernel, no plan, and no
 * allocation: the kernel's scratch (status word, tile counters, split-K
 * partials) is one 1 MiB array compiled into the library, which every GPU that
 * loads the library holds until the process exits.  Limits: N <= 262144 rows
 * (the counters) and at most 383 SMs (the partials); larger shapes return
 * DEP_ERR_UNSUPPORTED.  Same layouts, alignment and argument errors as
 * dep_projection_run; B == 0 does nothing.  The first call on a device looks up
 * the array's device address (cudaGetSymbolAddress) with that device current;
 * make that first call before any stream capture.  Every call clears the
 * counters and status word on `stream` before its kernel.  All calls share the
 * one array: calls that overlap on the GPU (other streams, other threads) race
 * and give wrong results.  Give-ups of the kernel's bounded waits are not
 * reported by this entry point.
 */
dep_status_t dep_projection_run_static(const void *x, const void *W, void *y, int64_t N,
                                       int64_t K, int32_t B, void *stream);

/*
 * No counterpart in the pages: a measurement aid.  Reads `bytes` of device
 * memory at p once with a read-only streaming kernel (16-byte loads, four in
 * flight per thread, four 512-thread blocks per SM) and XORs a fold of what it
 * read into the 64-bit word *sink (device memory), so that timing it on
 * `stream` gives the device's read-only bandwidth: the ceiling of a call that
 * streams a weight and writes almost nothing (a device-to-device copy also
 * writes as many bytes as it reads).  p 16-byte aligned, bytes a multiple of
 * 16, sink 8-byte aligned (else MISALIGNED); INVALID_ARG for null pointers or
 * zero bytes; CUDA if the launch fails.  Asynchronous.
 */
dep_status_t dep_projection_probe_read(const void *p, size_t bytes, void *sink, void *stream);

/* The tactic the plan uses for a batch of B >= 1 rows. */
dep_status_t dep_projection_plan_query(dep_plan_t plan, int32_t B, dep_tactic_t *out);

/* Copy up to `cap` table entries (sorted by max_rows) to `out`; *n = entry count. */
dep_status_t dep_projection_plan_table(dep_plan_t plan, dep_tactic_t *out, int32_t cap,
                                       int32_t *n);

/* Replace (or insert) the table entry with key tactic->max_rows.  The tactic is
 * validated (INVALID_ARG if not; UNSUPPORTED, as for dep_projection_run_tactic,
 * for a grid the device cannot hold at once); if it needs more workspace, counters or
 * staging than the plan owns, the plan's device block is re-allocated (after a
 * device synchronisation; OOM leaves the plan unchanged). */
dep_status_t dep_projection_plan_set(dep_plan_t plan, const dep_tactic_t *tactic);

/*
 * Inspection: copy the plan's split-K partial area (FP32) to host memory after
 * synchronising the device; *written = bytes copied (at most `bytes`).  Layout
 * for a stream-K launch of C blocks: partial (block c, slot s, batch column j,
 * tile row r) at float index ((c * 2 + s) * cols + j) * tile_n + r, slot 0 for
 * the block's first tile and 1 for its last.  Lets a test re-add the partials
 * of every split tile in block order and check the kernel's fix-up bit for bit.
 * For a DEP_KIND_TC_WIDE launch of C blocks with MMA width NT on groups of
 * R = tile_n rows: block c's piece of a split group sits in slot s (1 for the
 * group the block starts in, 0 for its last group when it has more than one)
 * at float offset (c * 2 + s) * R * NT; inside it, epilogue warp e (0..7, TMEM
 * lane quadrant (e + 2) % 4, column half e / 4 of the G * NT accumulator
 * columns) owns 32 * G * NT / 2 floats, accumulator column j of TMEM lane l
 * at (j / 4 * 32 + l % 32) * 4 + j % 4.  Without DEP_PLAN_KEEP_PIECES the
 * columns a block reduces itself are not stored.
 */
dep_status_t dep_projection_plan_partials(dep_plan_t plan, void *host, size_t bytes, size_t *written);

/*
 * Inspection: copy the plan's K-piece exchange region (64-bit words) to host
 * memory after synchronising the device; *written = bytes copied (at most
 * `bytes`).  For a K-piece launch (TC_SPLIT, S > 1 pieces in effect) the word of
 * (tile t, piece p, batch column j, tile row r) is at index
 * ((t * S + p) * cols + j) * tile_n + r; its low 32 bits are the piece's FP32
 * partial, its high 32 bits the "full" flag (0 once the launch has finished).
 * Lets a test re-add the pieces in order and check y bit for bit.
 */
dep_status_t dep_projection_plan_exchange(dep_plan_t plan, void *host, size_t bytes, size_t *written);

/* Bytes of device workspace the plan owns (split-K partials, counters, status). */
dep_status_t dep_projection_plan_workspace(dep_plan_t plan, size_t *bytes);

/*
 * Save the table as text keyed by (device name, SM count, N, K), and load it
 * back onto the current device (tuning need not be repeated).  Files are
 * written in format 2 (eight fields per entry); format 1 files (seven fields,
 * no K pieces) still load.  Load checks the
 * shape (INVALID_ARG if it differs) and the SM count (UNSUPPORTED if the file
 * was made for another GPU, or holds a grid this device cannot hold at once).  Errors: IO for unreadable or malformed files.
 */
dep_status_t dep_projection_plan_save(dep_plan_t plan, const char *path);
dep_status_t dep_projection_plan_load(const char *path, int64_t N, int64_t K,
                                      dep_plan_t *out);

/* Free the plan and its device memory (synchronises its device).  NULL is a no-op. */
void dep_projection_plan_destroy(dep_plan_t plan);

/*
 * Read and clear the plan's device status word (synchronises `stream`).
 * *code = 0 if every kernel since the last read finished its waits; otherwise
 * the first nonzero code a kernel recorded (see DEP_DEV_* below), and the
 * return value is DEP_ERR_TIMEOUT; the plan's split-K counters and K-piece
 * exchange flags, which a give-up may leave mid-protocol, are then cleared
 * (synchronises the device) so that later runs start clean.
 */
dep_status_t dep_projection_device_status(dep_plan_t plan, void *stream, int32_t *code);

#define DEP_DEV_TIMEOUT_PRODUCER 1 /* the load warp gave up waiting for a free stage */
#define DEP_DEV_TIMEOUT_CONSUMER 2 /* a compute warp gave up waiting for a stage's data */
#define DEP_DEV_TIMEOUT_MMA 3      /* the MMA warp gave up waiting */
#define DEP_DEV_TIMEOUT_EPILOGUE 4 /* an epilogue warp gave up waiting for an accumulator */
#define DEP_DEV_BOUNDS 5           /* bounds-checked (DEP_DEBUG) builds only: a kernel
                                      computed an index past one of its buffers and
                                      skipped that access */

/*
 * Bounded-wait self-test: launches one block whose waits can never be satisfied
 * (an mbarrier that nothing arrives on) with a wait limit of `limit_us`
 * microseconds, synchronises, and reports the code the kernel recorded in
 * *code (expected: DEP_DEV_TIMEOUT_CONSUMER).  Returns DEP_OK if the kernel
 * came back by itself.  Exercises the give-up path without faulting the GPU.
 */
dep_status_t dep_projection_selftest_timeout(int32_t limit_us, int32_t *code);

/*
 * Give-up self-test of the split-K exchange, on a plan's own workspace: enqueues
 * on `stream` one warp that publishes ("full") exchange words of two pieces,
 * as publishers would, then runs the exchange's reducer over two pieces of
 * which one is never published, with a wait limit of `limit_us` microseconds.
 * The reducer gives up and records DEP_DEV_TIMEOUT_EPILOGUE in the plan's
 * status word; the unreduced piece's flags and a nonzero word at the start of
 * the counters are left behind.  dep_projection_device_status then reports the code and clears the
 * counters and exchange words, after which the plan's runs give the same bits
 * as a fresh plan's.  Exercises the give-up path without faulting the GPU.
 * Errors: INVALID_ARG (null plan, limit outside 1 us..10 s), UNSUPPORTED
 * (host-only plan, or a plan whose table has no tensor-core tactic and so no
 * exchange region), CUDA.
 */
dep_status_t dep_projection_plan_selftest_exchange(dep_plan_t plan, int32_t limit_us, void *stream);

/* ------------------------------------------------------------------------
 * Around the projections of a delta-attention layer: the norm that feeds a
 * projection, the projection with 8-bit integers on both sides, and the gated
 * delta rule between the packed input projection (96 heads of 128 channels in
 * 49376 rows) and the output projection.  No counterpart in the pages.
 *
 * These calls are asynchronous on `stream`, allocate nothing, do not
 * synchronise and can be captured in CUDA graphs (dep_int8_plan and
 * dep_int8_device_status excepted).  Tensors lie in device memory of the
 * current device; strides are in elements; nothing is retained.  Status codes
 * as above; a null `args`, a null required pointer or a bad size is
 * INVALID_ARG.
 * ------------------------------------------------------------------------ */

/* Formats of a stored row. */
#define DEP_QUANT_NONE 0 /* BF16, no scales */
#define DEP_QUANT_INT8 1 /* int8, one scale for each row */
#define DEP_QUANT_E4M3 2 /* e4m3, one scale for each group of 128 columns (the last
                            group of a row may be shorter) */
#define DEP_QUANT_GROUP 128
#define DEP_NORM_MAX_COLS 65536

/*
 * Root-mean-square norm of `rows` rows of `cols` columns, after the residual's
 * addition:
 *
 *     h = BF16(x + residual)            (h = x where residual is null)
 *     y = h / sqrt(mean(h^2) + eps) * weight
 *
 * h is stored to residual_out (which may be `residual` itself, with the same
 * stride) and the norm is taken of h as stored.  y is stored in one format:
 *   NONE  BF16 [rows, cols], one rounding.
 *   INT8  q = rint(127 p / P) with p = h * weight (exact in FP32) and P the
 *         row's largest |p|: 1/rms cancels out of q.  scale[row] = P/rms/127.
 *   E4M3  q = e4m3(448 p / P), P the group's largest |p|;
 *         scale[row, group] = P/rms/448, scales contiguous [rows, ceil(cols/128)].
 * Both quotients are rounded as if they were exact (ties to even), up to the
 * largest values (a p beyond FP32's range counts as an infinity), so q is the
 * same on every run and machine.  A row (group) whose P is below 2^-100 is
 * stored as zeros with a scale of zero; one that holds an infinity or a NaN has
 * a scale that is infinite or NaN.
 * Sums and scales are FP32; a row whose squares leave FP32's range is added up
 * times a power of two, so 1/rms is right for any finite h (up to 2^127, what
 * FP32 holds).  Any alignment and strides >= cols; 16-byte aligned
 * rows (8-byte for q) are moved in wide loads and stores.  `out` may be x
 * itself (format NONE, same stride).  Errors: INVALID_ARG also for an output
 * that overlaps an input or another output in any other way; UNSUPPORTED for
 * cols > DEP_NORM_MAX_COLS.  rows == 0 does nothing.
 */
typedef struct {
    const void *x;        /* BF16 [rows, cols] */
    const void *residual; /* BF16 [rows, cols] or null */
    const void *weight;   /* BF16 [cols] or null (ones) */
    void *residual_out;   /* BF16 [rows, cols]; required with `residual`, else null */
    void *out;            /* [rows, cols] of `quant`'s type */
    float *scale;         /* scales of an 8-bit format, else null */
    int64_t x_stride, residual_stride, residual_out_stride, out_stride;
    int64_t rows, cols;
    int32_t quant; /* DEP_QUANT_* */
    float eps;     /* >= 0 */
} dep_norm_args_t;

dep_status_t dep_add_rms_norm(const dep_norm_args_t *args, void *stream);

/* The rows of x in 8 bits, by the same rules without a norm: p = x, rms = 1.
 * residual, weight and residual_out must be null, quant INT8 or E4M3; eps is
 * not used.  Prepares the input of a projection that no norm feeds, and the
 * weight of dep_int8_run (a scale for each output channel). */
dep_status_t dep_quantize_rows(const dep_norm_args_t *args, void *stream);

/*
 * The gated delta rule over sequences packed one after another.  For each
 * sequence and value head, with a state S [Dv, Dk] and for every token
 *
 *     S <- S diag(exp(g)),   S <- S + beta (v - S k) k^T,   o = scale * S q
 *
 * q, k: BF16 [tokens, Hq, Dk]; v: BF16 [tokens, Hv, Dv]; o: BF16 [tokens, Hv, Dv];
 * heads contiguous in a token, tokens q_stride etc. apart, so that slices of a
 * packed projection are read in place.  Hv is a multiple of Hq; value head h
 * takes query and key head h / (Hv / Hq).  g: FP32 natural logarithm of the
 * decay, one for each head [tokens, Hv] or (DEP_DELTA_CHANNEL) for each key
 * channel [tokens, Hv, Dk]; minus infinity empties the state, and values above
 * zero count as zero (a decay is at most one).  beta: FP32 [tokens, Hv].
 * With DEP_DELTA_L2NORM q and k are first divided by
 * sqrt(sum of squares + 1e-6) over their Dk channels.
 * Sequences: cu_seqlens, int32 [n_seq + 1] in device memory, first tokens and
 * the end (never decreasing, so lengths may be zero; clipped to 0..tokens), or null for
 * n_seq sequences of tokens / n_seq each.
 * States: FP32 [n_states, Hv, Dv, Dk], contiguous.  Sequence s starts from
 * state_in[i] and leaves state_out[i], i = slots[s] (int32, device memory) or s
 * where slots is null.  state_in null: from zeros.  state_out may be state_in.
 * A slot outside 0..n_states-1 (padding) has no state read or written and zeros
 * for its outputs.  Two sequences of a call may not share a slot.
 * States stay in FP32; o is rounded once.  Fixed order, no atomics.  By chunks (see
 * below) the operands of products are split into FP16 parts: they keep 22 bits, and
 * what a chunk's outputs and state lose is counted against the largest that the state's
 * row held within the chunk.  Rows of a state that are below 2^-92 altogether keep fewer.
 * A chunk whose tokens are too far apart in size for that, or not all finite, goes token by
 * token: an infinity or a NaN reaches no output of an earlier token, and a decay to
 * nothing leaves nothing of the state before it, however large.  With L2NORM the sums
 * of squares are FP32: |q| and |k| up to 2^63.  Tokens that belong to no sequence of the
 * table (before its first entry, from its last on) keep what their rows of o hold.
 * Dk is 64 or 128, Dv a multiple of 16 up to 256 (else UNSUPPORTED).
 * Workspace: device memory that the call overwrites.  With it, sequences of eight
 * tokens and more on average go by chunks of sixteen tokens, whose shares that do
 * not depend on the state are worked out there first, as many at once as it holds;
 * without it, or with less than one chunk of every head takes, all go token by token.
 * dep_delta_workspace gives the bytes that help: 0 for short sequences, else what
 * holds all chunks, but at most 2 GiB (or one chunk, where that is more).  It reads
 * tokens, n_seq, Hv and Dk alone.
 * MISALIGNED unless q, k, v, g (per channel), o, the states and the workspace are 16-byte
 * aligned, the strides of q, k, v and o multiples of 8 and g's of 4 (per channel),
 * and cu_seqlens, slots, beta and a per-head g 4-byte aligned.
 */
#define DEP_DELTA_CHANNEL 1u /* g for each key channel */
#define DEP_DELTA_L2NORM 2u  /* normalise q and k */

typedef struct {
    const void *q, *k, *v;
    const float *g, *beta;
    const float *state_in; /* or null */
    float *state_out;
    void *o;
    const int32_t *cu_seqlens; /* or null */
    const int32_t *slots;      /* or null */
    int64_t q_stride, k_stride, v_stride, g_stride, beta_stride, o_stride; /* between tokens */
    int64_t tokens, n_states;
    int32_t n_seq, Hq, Hv, Dk, Dv;
    uint32_t flags;
    float scale;
    void *workspace; /* or null */
    int64_t workspace_bytes;
} dep_delta_args_t;

dep_status_t dep_delta_rule(const dep_delta_args_t *args, void *stream);
dep_status_t dep_delta_workspace(const dep_delta_args_t *args, int64_t *bytes);

/*
 * y[B,N] = BF16(x_scale[b] * w_scale[n] * sum_k x[b,k] * W[n,k]) with x and W
 * int8: the projection at half the weight bytes.  The sum is exact (32-bit
 * integers; K <= 131056, so that it cannot overflow); the two scales are
 * multiplied in FP32, then with the sum, and the product is rounded to BF16.
 * x [B,K], W [N,K], y [B,N] row-major, contiguous and 16-byte aligned, K a
 * multiple of 16 (else MISALIGNED); x_scale [B] and w_scale [N] FP32.  y must
 * not overlap an input.  B == 0 does nothing.
 * A plan owns the workspace of one weight shape and batches of up to max_rows
 * rows (wider ones run in passes); two runs of one plan must not overlap on
 * the GPU.
 */
typedef struct dep_int8_plan_s *dep_int8_plan_t;

dep_status_t dep_int8_plan(int64_t N, int64_t K, int32_t max_rows, dep_int8_plan_t *out);
dep_status_t dep_int8_run(dep_int8_plan_t plan, const void *x, const float *x_scale, const void *W,
                          const float *w_scale, void *y, int32_t B, void *stream);
/* Bytes of device workspace the plan owns. */
dep_status_t dep_int8_plan_workspace(dep_int8_plan_t plan, size_t *bytes);
/* As dep_projection_device_status, for the plan's own status word. */
dep_status_t dep_int8_device_status(dep_int8_plan_t plan, void *stream, int32_t *code);
/* Free the plan (synchronises its device).  NULL is a no-op. */
void dep_int8_plan_destroy(dep_int8_plan_t plan);

/* ------------------------------------------------------------------------
 * The core of a softmax-attention layer between the packed input projection
 * and the output projection (7168 x 12288: 96 heads of 128 channels): the
 * norm and rotation of the heads of q and k, the paged cache, and attention
 * over it.  No counterpart in the pages.  The calls keep the rules of the
 * group above (asynchronous, nothing allocated, capturable).
 * ------------------------------------------------------------------------ */

/*
 * For every token t and every head of q and of k, D channels x:
 *
 *     y = x / sqrt(mean(x^2) + eps) * weight     (DEP_HEADS_NORM; else y = x)
 *     (a, b) <- amplitude * (a cos u - b sin u, b cos u + a sin u),
 *                                                u = positions[t] * freqs[i]
 *
 * for the pairs i = 0 .. rot/2 - 1 of the channels [first, first + rot): channels
 * first + i and first + rot/2 + i, or with DEP_HEADS_INTERLEAVED first + 2i and
 * first + 2i + 1.  The other channels keep y.  FP32 throughout, one rounding to
 * BF16 at the end; the angle is reduced as a 64-bit fraction of a turn, so far
 * positions lose nothing (2^-53 of position * frequency) before it is rounded to FP32.  freqs: FP64 radians a
 * position, rot/2 of them (not read where rot is 0).  1/rms is right for any
 * finite x (up to 2^128).
 *
 * dep_norm_rotate stores the heads to q_out and k_out (each may be its input, with
 * the same stride); k may be null (Hk is then 0).
 * dep_append_kv stores k's heads, and v's as they are, to a cache of pages:
 * token t's to slot slots[t] % page_size of page slots[t] / page_size.  A slot below
 * 0 or at or past n_pages * page_size is padding: nothing of the token is stored to
 * the cache.  Two tokens of a call may not share a slot.  q and q_out may both be null
 * (Hq is then 0); where given, q is normed and rotated as in dep_norm_rotate, for every
 * token.
 *
 * q [tokens, Hq, D], k and v [tokens, Hk, D] BF16, heads contiguous in a token and
 * tokens q_stride etc. apart, so that columns of a packed projection are read in
 * place.  Caches: BF16, channel c of head h at slot s of page p at
 * p * page_stride + s * slot_stride + h * head_stride + c, so that a page may hold
 * the heads of each token or the tokens of each head.  D, rot and first are multiples
 * of 8, D at most 256 (else UNSUPPORTED).  q, k, v, outputs and caches are 16-byte
 * aligned and their strides multiples of 8; the weights are 16-byte, freqs 8-byte and
 * positions and slots 4-byte aligned (else MISALIGNED).  INVALID_ARG also for an
 * output that overlaps an input or another output in any other way, and for a cache
 * whose strides let two of its rows share bytes.
 */
#define DEP_HEADS_INTERLEAVED 1u /* pairs of neighbours, not of halves */
#define DEP_HEADS_NORM 2u        /* RMS norm of each head */
#define DEP_HEADS_MAX_D 256

typedef struct {
    const void *q, *k, *v;
    const void *q_weight, *k_weight; /* BF16 [D], or null (ones); only with DEP_HEADS_NORM */
    const double *freqs;             /* [rot / 2] */
    const int32_t *positions;        /* [tokens], or null where rot is 0 */
    const int32_t *slots;            /* [tokens]; dep_append_kv */
    void *q_out, *k_out;             /* k_out: dep_norm_rotate */
    void *k_cache, *v_cache;         /* dep_append_kv */
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride; /* between tokens */
    int64_t k_page_stride, k_slot_stride, k_head_stride, v_page_stride, v_slot_stride, v_head_stride;
    int64_t tokens, n_pages;
    int32_t Hq, Hk, D, rot, first, page_size;
    uint32_t flags;
    float eps, amplitude;
} dep_heads_args_t;

dep_status_t dep_norm_rotate(const dep_heads_args_t *args, void *stream);
dep_status_t dep_append_kv(const dep_heads_args_t *args, void *stream);

/*
 * Attention of the new tokens of several sequences over a paged cache.  For token t
 * of sequence s and query head h (key and value head h / (Hq / Hk))
 *
 *     o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q . k_j),
 *     lse = log(sum_j p_j)
 *
 * over the positions j that the token sees.  The sequence has kv_lens[s] positions in
 * the cache, position j in slot j % page_size of page page_table[s, j / page_size];
 * the last n of them are those of its own n tokens, token i's at kv_lens[s] - n + i
 * (they are stored before the call, as by dep_append_kv).  All its tokens see the
 * positions before these.  Of these a token sees
 *   tree null:  those up to its own (a decode token, a piece of a prompt; any n);
 *   tree given: token i' of the sequence where bit i' of tree[t] is set (a tree of
 *               drafted tokens: a node's ancestors and, to see itself, its own bit).
 *               Tokens from the 64th on of a sequence are seen by none.
 * What a token does not see does not reach its output, whatever the cache holds there.
 * A token that sees nothing (or nothing but scores of minus infinity) has zeros and
 * lse minus infinity.  Positions on a page outside 0..n_pages-1 are seen by none, and
 * kv_lens is clipped to 0..table_width * page_size; a sequence may be shorter than its
 * n tokens (those before position 0 are not in the cache).
 *
 * q, o: BF16 [tokens, Hq, D], heads contiguous, tokens q_stride and o_stride apart.
 * lse: FP32 [tokens, Hq], contiguous, or null.  Caches as for dep_append_kv (rows may
 * share bytes here).  cu_seqlens: int32 [n_seq + 1] in device memory (never decreasing;
 * clipped to 0..tokens), or null for n_seq sequences of tokens / n_seq each.  Tokens
 * that belong to no sequence keep what their rows of o and lse hold.  kv_lens int32
 * [n_seq], page_table int32 [n_seq, table_width], rows table_stride apart, tree 64-bit
 * words [tokens]: device memory.  Hq is a multiple of Hk, D 64 or 128 (else
 * UNSUPPORTED, as are Hq D, tokens Hq, n_seq, n_pages and table_width page_size from
 * about 2^31 on), scale finite and not negative.
 * Scores, sums and o's accumulators are FP32 (q . k and scale q . k of any size in FP32's
 * range; from about 2^27 on the latter is rounded to FP32 before anything else); the p_j,
 * taken relative to the row's largest, are rounded to BF16 for the product with v, which
 * puts o 0.0023 (rms) off where its own rounding alone puts it 0.0017.  The order of sums is fixed for given sizes and lengths.  No atomics.
 * Workspace: device memory that the call overwrites, at least dep_attention_workspace
 * bytes (of tokens, n_seq, Hq, Hk and D alone; else INVALID_ARG).
 * Every wait in the kernel is bounded (1 s); if one gives up, a DEP_DEV_* code is stored to
 * *status where that holds 0, and every row of o and lse that is not complete is NaN
 * (complete ones may be).
 * MISALIGNED unless q, o, the caches and the workspace are 16-byte aligned, the strides
 * of q, o and the caches multiples of 8, tree 8-byte and the rest 4-byte aligned.
 */
typedef struct {
    const void *q, *k_cache, *v_cache;
    const int32_t *page_table, *kv_lens;
    const int32_t *cu_seqlens; /* or null */
    const uint64_t *tree;      /* or null */
    void *o;
    float *lse; /* or null */
    int64_t q_stride, o_stride;
    int64_t k_page_stride, k_slot_stride, k_head_stride, v_page_stride, v_slot_stride, v_head_stride;
    int64_t table_stride, tokens, n_pages;
    int32_t n_seq, Hq, Hk, D, page_size, table_width;
    float scale;
    void *workspace;
    int64_t workspace_bytes;
    int32_t *status; /* or null; device memory */
} dep_attention_args_t;

dep_status_t dep_paged_attention(const dep_attention_args_t *args, void *stream);
dep_status_t dep_attention_workspace(const dep_attention_args_t *args, int64_t *bytes);

/*
 * Give-up self-test of the attention: dep_paged_attention in which waits of the kind
 * `code` (a DEP_DEV_TIMEOUT_* code) are held up for good.  A block that comes to one
 * gives up after the second that a wait may take, ends its copies and products in
 * flight and returns; the first wait of the call that gave up (of this kind, or for what it
 * holds up) stores its code to *status.  A call in which no such wait is needed (a ring that
 * is never full) ends as ever.  The workspace serves later calls as it is.  Exercises the
 * give-up path without faulting the GPU.  Errors: as dep_paged_attention; INVALID_ARG
 * also for another code.
 */
dep_status_t dep_attention_selftest_timeout(const dep_attention_args_t *args, int32_t code, void *stream);

/* The binning rule on its own: index into keys[0..n_keys) of the entry serving
 * B rows -- smallest key >= B, else the largest key; -1 if n_keys < 1.  The keys
 * need not be sorted.  Pure host function. */
int32_t dep_bins_index(const int32_t *keys, int32_t n_keys, int32_t B);

/* Static description of a status code.  Never NULL. */
const char *dep_status_string(dep_status_t status);

/* Library version, as MAJOR * 10000 + MINOR * 100 + PATCH. */
int32_t dep_projection_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DEP_PROJECTION_H */
