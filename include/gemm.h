/*
 * gemm.h -- C ABI of the GB300 (sm_103a) dense GEMM / GEMV library
 * (libdgemm_gb300.so).
 *
 * Operation (one call):
 *
 *     C <- act(alpha * op(A) @ op(B) + beta * C)
 *
 * op(A) is M x K, op(B) is K x N and C is M x N, following the BLAS naming of
 * "Matrix Multiplication Background User's Guide", section 2 (Math and Memory
 * Bounds); every output is a K-long dot product, 2*M*N*K floating-point
 * operations in all.  The guide's display formula for GEMM is lost in the
 * extracted text: the BLAS form above is the reading taken.  act is the
 * identity, LeakyReLU (the fused output transform of "OpenAI open-sources the
 * Triton GPU language (part 2)", section Matrix multiplication), ReLU, GELU
 * or SiLU.  Operands are bf16, fp16 or TF32 (fp32 words), products are
 * accumulated in fp32, C is fp32 or the operand type (gemm_run_ex: a separate
 * D, and a C of its own type).
 *
 * Storage is row-major ("Learning Triton One Kernel at a Time: Matrix
 * Multiplication", section Memory coalescing: a row is contiguous, a
 * transpose changes the strides, not the memory):
 *   transA = GEMM_OP_N: A is stored M x K,  op(A)(i,k) = A[i*lda + k]
 *   transA = GEMM_OP_T: A is stored K x M,  op(A)(i,k) = A[k*lda + i]
 *   transB = GEMM_OP_N: B is stored K x N,  op(B)(k,j) = B[k*ldb + j]
 *   transB = GEMM_OP_T: B is stored N x K,  op(B)(k,j) = B[j*ldb + k]
 *   C is stored M x N,                      C(i,j)     = C[i*ldc + j]
 * Leading dimensions count elements.  Entries of a row beyond its logical
 * width (the ld padding) are never read or written.
 *
 * Execution: gemm_run is asynchronous and stream-ordered on the caller's CUDA
 * stream; it returns after enqueueing its kernels.  All device pointers are
 * owned by the caller and must stay valid until the stream has run the call.
 * The plan owns its workspace (split-K partials, GEMV partials, the watchdog
 * word) and frees it in gemm_plan_destroy.  One plan must not be used by two
 * host threads, or on two streams whose work may overlap, at the same time.
 * The GEMM and GEMV kernels launch as programmatic dependents of the previous
 * kernel on the stream (CUDA programmatic dependent launch): their launch
 * and setup may overlap that kernel's last moments, but they touch no memory
 * before it has completed, so stream order holds as for a plain launch.  The
 * GEMM kernel lets its own dependents start early; a caller's kernel launched
 * after a gemm_run with the programmatic stream-serialization attribute must
 * therefore call cudaGridDependencySynchronize() (griddepcontrol.wait) before
 * it reads the result, as that attribute requires.  Set GEMM_PDL=0 in the
 * environment before gemm_plan_create for plain launches.
 *
 * Errors: argument problems are reported synchronously, before anything is
 * launched, as a gemm_status_t; nothing aborts or throws across this ABI.
 * There is no CPU fallback: without a usable sm_100-family GPU,
 * gemm_plan_create returns GEMM_ERR_NO_DEVICE.
 */
#ifndef DGEMM_GB300_GEMM_H
#define DGEMM_GB300_GEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gemm_plan* gemm_plan_t;

typedef enum {
  GEMM_OK = 0,
  GEMM_ERR_INVALID_ARG = 1,   /* null pointer, negative size, ld too small, bad enum  */
  GEMM_ERR_ALIGNMENT = 2,     /* pointer or leading dimension breaks the rules below */
  GEMM_ERR_UNSUPPORTED = 3,   /* size beyond what the kernels index (see gemm_run)   */
  GEMM_ERR_NO_DEVICE = 4,     /* no CUDA device, or not compute capability 10.x      */
  GEMM_ERR_OUT_OF_MEMORY = 5, /* workspace allocation failed                         */
  GEMM_ERR_CUDA = 6,          /* a CUDA runtime/driver call or a launch failed       */
  GEMM_ERR_TIMEOUT = 7,       /* a kernel's bounded wait ran out (watchdog)          */
  GEMM_ERR_DEBUG_CHECK = 8    /* debug build: a kernel's bounds or copy-rule check
                                 failed and the access was skipped (see below)    */
} gemm_status_t;

typedef enum { GEMM_OP_N = 0, GEMM_OP_T = 1 } gemm_op_t;

/* operand type _ C type */
typedef enum {
  GEMM_BF16_F32 = 0,
  GEMM_BF16_BF16 = 1,
  GEMM_F16_F32 = 2,
  GEMM_F16_F16 = 3,
  /* A and B are fp32 words read as TF32 by the tensor core: sign, exponent and
   * the 10 highest fraction bits (the 13 lowest are dropped), fp32
   * accumulation, C fp32 ("Matrix Multiplication Background User's Guide",
   * section 2.2, Table 1).  Every shape runs on the tensor cores, M = 1 or
   * N = 1 included.  Operands stored M/N-major (transA = T, transB = N) are
   * read by the MMAs where they are, except where the call is large enough
   * that copying one or both K-major into plan workspace first is estimated
   * faster (the in-place MMAs run ~10% longer with one such operand, ~44%
   * with both; a copy reads and writes the operand): 8192^3, for instance.
   * GEMM_TF32_TRANSPOSE=1 in the environment copies every M/N-major TF32
   * operand, =0 none (read at every call). */
  GEMM_TF32_F32 = 4
} gemm_dtype_t;

typedef enum {
  GEMM_ACT_NONE = 0,
  GEMM_ACT_LEAKY_RELU = 1, /* x < 0 ? slope*x : x  (the pages' example: "OpenAI open-sources the
                              Triton GPU language (part 2)", section Matrix multiplication) */
  GEMM_ACT_RELU = 2,       /* x < 0 ? 0 : x  (-0 and NaN pass unchanged)                    */
  GEMM_ACT_GELU = 3,       /* x * Phi(x), Phi the standard normal distribution function,
                              evaluated as erfc(-x / sqrt(2)) / 2 in fp32                    */
  GEMM_ACT_SILU = 4        /* x * sigmoid(x) = x / (1 + exp(-x)), in fp32                     */
} gemm_act_t;

/* The activation is applied in fp32 to alpha*acc + beta*C, before the
 * rounding to the output type; slope is read for GEMM_ACT_LEAKY_RELU only. */
typedef struct {
  int32_t act;
  float slope;
} gemm_epilogue_t;

/* Which kernels a call used. */
typedef enum {
  GEMM_PATH_NONE = 0,          /* M == 0 or N == 0: nothing launched                    */
  GEMM_PATH_TC = 1,            /* tcgen05 tensor-core GEMM, epilogue fused               */
  GEMM_PATH_TC_SPLITK = 2,     /* tcgen05 GEMM over K slices + fixed-order reduction     */
  GEMM_PATH_GEMV_ROWDOT = 3,   /* GEMV: one warp per contiguous row                      */
  GEMM_PATH_GEMV_COLSTREAM = 4,/* GEMV: threads own 8 contiguous columns, K split       */
  GEMM_PATH_GEMV_GENERIC = 5,  /* GEMV with strided operands (no 128-bit loads)          */
  GEMM_PATH_SCALE = 6,         /* K == 0 or alpha == 0: C <- act(beta*C)                 */
  GEMM_PATH_TC_SPLITK_CLUSTER = 7, /* tcgen05 GEMM, K in two halves on a cluster of two CTAs
                                  whose partial sums are added on chip: one launch, no
                                  workspace (the reduction of section 2.3 done in place) */
  GEMM_PATH_TC_TAIL_SPLIT = 8, /* tcgen05 GEMM: whole tiles for the full waves; only the
                                  tiles of the last, partly filled wave are split along K
                                  (section 3.2's tail wave), + reduction of those tiles  */
  GEMM_PATH_SCALED = 9,        /* block-scaled product (8 or 4 bits), whole output tiles */
  GEMM_PATH_SCALED_SLICED = 10 /* block-scaled product with few rows or few tiles:       */
                               /* K slices on a cluster of CTAs, added on chip           */
} gemm_path_t;

/* Plan decisions and the tile/wave quantization they imply ("Matrix
 * Multiplication Background User's Guide", section 3, Dimension Quantization
 * Effects: section 3.1 tile quantization, section 3.2 wave quantization). */
typedef struct {
  int32_t path;            /* gemm_path_t                                              */
  int32_t tile_m;          /* output tile rows (tensor-core paths)                     */
  int32_t tile_n;          /* output tile columns                                      */
  int32_t tile_k;          /* K elements per pipeline stage                            */
  int32_t cta_per_tile;    /* CTAs that work on one tile (1; 2 = a cluster of two: a    */
                           /* 256-row CTA pair, or the K halves of a split-K cluster)  */
  int32_t splitk;          /* K slices (1 = none)                                      */
  int32_t stages;          /* shared-memory pipeline depth                             */
  int32_t raster_group;    /* output-tile rows per rasterisation group                 */
  int32_t grid;            /* CTAs launched for the main kernel (gemm_choose_config:  */
                           /* 0 for the row-dot and generic GEMVs, whose grid comes   */
                           /* from the device's occupancy at launch)                  */
  int32_t sms;             /* streaming multiprocessors used for the wave size         */
  int64_t tiles;           /* output tiles = ceil(M/tile_m) * ceil(N/tile_n)           */
  int64_t units;           /* work units = tiles - tail_tiles + tail_tiles * splitk    */
                           /* (a 256-row pair tile is one unit of two CTAs; a K pair  */
                           /* tile is two units, its halves)                          */
  double waves;            /* units / wave size                                        */
  double tail_fraction;    /* (units mod wave) / wave: SMs busy in the last wave, 0=full */
  double useful_fraction;  /* M*N / (tiles*tile_m*tile_n): share of tile area in C     */
  int32_t launches;        /* kernels the call launched                                */
  int32_t tail_tiles;      /* tiles split along K and reduced by a second launch:      */
                           /* all tiles (split-K), the last wave's (tail split) or 0   */
  int64_t workspace_bytes; /* plan workspace the call used                             */
} gemm_config_info_t;

/* Create a plan bound to CUDA device `device` (the caller's current device is
 * restored before returning).  Queries the SM count and allocates the
 * watchdog word.  Returns GEMM_ERR_NO_DEVICE if the device does not exist or
 * is not compute capability 10.x, GEMM_ERR_INVALID_ARG if plan is NULL.
 * With GEMM_LOG=1 in the environment at creation, every successful call of the
 * plan that launches kernels prints one line on stderr: its name, sizes and types, and for
 * products the decisions of gemm_config_info_t (gemm_choose_config does the same).
 * With GEMM_NVTX=1 at creation, every such call is
 * an NVTX range ("gemm MxNxK types opA opB", "gemm_quantize RxK types", ...) on the calling thread, for a
 * profiler's timeline (no cost beyond the range calls; none without a tool). */
gemm_status_t gemm_plan_create(gemm_plan_t* plan, int device);

/* C <- act(alpha * op(A) @ op(B) + beta * C), enqueued on `stream` (a
 * cudaStream_t; NULL means the legacy default stream).  Calls may be captured
 * into a CUDA graph and add only kernel launches to it: workspace that a captured
 * call has to add is allocated at once, outside the graph (the host waits for that; a call of the
 * same sizes before the capture avoids it), and what a captured call uses stays where it is
 * until gemm_plan_destroy, so that a graph may be replayed after later calls have grown
 * the workspace.  Replays are subject to the rule on streams at the top like calls.  See the top of this
 * file for the layout of A, B and C; all three are device pointers.
 *
 * Dispatch: M == 0 or N == 0 launches nothing; K == 0 or alpha == 0 gives
 * C <- act(beta*C) without reading A or B; M == 1 or N == 1 takes the
 * memory-bound GEMV kernels (no tensor cores: "Matrix Multiplication
 * Background User's Guide", section 2 notes that matrix-vector products are
 * always memory-bound); everything else takes the tcgen05 tensor-core kernel,
 * split along K when the output has too few tiles to fill the GPU (section
 * 2.3 mentions splitting along K followed by a reduction).  With beta == 0,
 * C is not read (NaN in C does not propagate).
 *
 * Rules, checked before any launch:
 *  - M, N, K >= 0 and each < 2^31; lda >= stored columns of A (K for N, M
 *    for T), ldb >= stored columns of B (N for N, K for T), ldc >= N; all >= 1.
 *  - A and B may be NULL only if M*N == 0 or K == 0 or alpha == 0; C may be
 *    NULL only if M*N == 0.
 *  - When A and B are read (M*N > 0, K > 0, alpha != 0), no byte of C (its
 *    M rows of N elements, ldc apart) may lie in A or B (their stored rows,
 *    lda / ldb apart).  Slices of one parent whose rows interleave without
 *    sharing a byte are accepted; with different leading dimensions and more
 *    than 2^20 rows on both sides, overlapping address ranges are rejected.
 *  - Every pointer is aligned to its element size.
 *  - Tensor-core path (M >= 2 and N >= 2): A, B and C are 16-byte aligned and
 *    lda, ldb, ldc times the element size are multiples of 16 bytes -- the
 *    rule of Table 1 of the guide's section 2.2 for FP16 (multiples of 8
 *    elements), which the Tensor Memory Accelerator requires here.
 *  - GEMM_TF32_F32 (always the tensor-core path): A and B 16-byte aligned with
 *    lda, ldb multiples of 4 elements (Table 1's TF32 row); C 4-byte aligned,
 *    and 16-byte aligned with ldc a multiple of 4 when N >= 4.
 * Violations return GEMM_ERR_INVALID_ARG or GEMM_ERR_ALIGNMENT.
 *
 * Split-K and GEMV with K split use the plan's workspace; the first call that
 * needs more than the plan holds grows it (stream-ordered allocation on
 * `stream`) and can return GEMM_ERR_OUT_OF_MEMORY.  Launch failures return
 * GEMM_ERR_CUDA.  A kernel whose bounded wait ran out sets the plan's
 * watchdog word (see gemm_plan_poll_error); the call itself still returns
 * GEMM_OK because it does not wait for the kernel.
 *
 * Results are deterministic: the same call on the same device gives the same
 * bits every time (split-K sums its slices in a fixed order). */
gemm_status_t gemm_run(gemm_plan_t plan, int64_t M, int64_t N, int64_t K,
                       const void* A, int64_t lda, const void* B, int64_t ldb,
                       void* C, int64_t ldc, float alpha, float beta,
                       gemm_dtype_t dtype, gemm_op_t transA, gemm_op_t transB,
                       gemm_epilogue_t epilogue, void* stream);

/* Free the plan and its workspace (synchronises the plan's device).  NULL is
 * accepted and ignored. */
gemm_status_t gemm_plan_destroy(gemm_plan_t plan);

/* Static, human-readable text for a status code. */
const char* gemm_status_string(gemm_status_t status);

/* Element types of gemm_run_ex's matrices. */
typedef enum { GEMM_TYPE_BF16 = 0, GEMM_TYPE_F16 = 1, GEMM_TYPE_F32 = 2,
               GEMM_TYPE_TF32 = 3, /* operands only (ab_type): fp32 words read as TF32 */
               GEMM_TYPE_E4M3 = 4, /* 8-bit, 4 exponent and 3 fraction bits, no infinity, largest 448   */
               GEMM_TYPE_E5M2 = 5, /* 8-bit, 5 and 2, largest 57344; both: block-scaled products only */
               GEMM_TYPE_E2M1 = 6  /* 4-bit, 2 and 1, largest 6, no infinity or NaN, two to a byte: gemm_dequantize only
                                      (the _mx calls imply it) */ } gemm_type_t;

/* D <- act(alpha * op(A) @ op(B) + beta * C) with a separate output D: the
 * gemm_run operation where the C that beta scales is read from one matrix and
 * the result written to another, each with its own leading dimension and
 * element type (e.g. fp32 C in, bf16 D out).
 *   ab_type  GEMM_TYPE_BF16, GEMM_TYPE_F16 or GEMM_TYPE_TF32: A and B, as in gemm_run.
 *   d_type   GEMM_TYPE_F32 or ab_type (GEMM_TYPE_F32 with TF32 operands): D (M x N,
 *            row stride ldd >= N), held to
 *            gemm_run's rules for C (device pointer, alignment, NULL only
 *            if M*N == 0).
 *   c_type   GEMM_TYPE_BF16, GEMM_TYPE_F16 or GEMM_TYPE_F32: C (M x N, row
 *            stride ldc >= N), read only when beta != 0 (it may then be NULL
 *            and ldc is ignored); it needs only its element alignment.  C may
 *            be D itself (same pointer, ldc == ldd, c_type == d_type: that is
 *            gemm_run); otherwise the two must not share a byte.  C may
 *            overlap A or B (all three are only read); D may not.
 * Violations return GEMM_ERR_INVALID_ARG or GEMM_ERR_ALIGNMENT before any
 * launch.  Paths, workspace, streams and errors as in gemm_run; the plan's
 * last configuration is updated the same way.  The pages fuse input and
 * output transforms into the product ("OpenAI open-sources the Triton GPU
 * language (part 2)", section Matrix multiplication); a separate D is the
 * output side of that with C left intact. */
gemm_status_t gemm_run_ex(gemm_plan_t plan, int64_t M, int64_t N, int64_t K, const void* A,
                          int64_t lda, const void* B, int64_t ldb, const void* C, int64_t ldc,
                          gemm_type_t c_type, void* D, int64_t ldd, gemm_type_t d_type, float alpha,
                          float beta, gemm_type_t ab_type, gemm_op_t transA, gemm_op_t transB,
                          gemm_epilogue_t epilogue, void* stream);

/* Decisions of the plan's most recent gemm_run (path, tile, split-K, grid,
 * waves, tail fraction, kernels launched).  GEMM_ERR_INVALID_ARG on NULL. */
gemm_status_t gemm_plan_last_config(gemm_plan_t plan, gemm_config_info_t* out);

/* Wait for `stream`, then read and clear the plan's watchdog word: returns
 * GEMM_ERR_TIMEOUT if any kernel of this plan gave up on a bounded wait since
 * the last poll, GEMM_ERR_DEBUG_CHECK if (debug build) a device-side check
 * failed, GEMM_OK otherwise, GEMM_ERR_CUDA if the stream failed. */
gemm_status_t gemm_plan_poll_error(gemm_plan_t plan, void* stream);

/* The word the last gemm_plan_poll_error read, before it was cleared (0:
 * nothing happened).  Bits 0-15: the bounded waits that ran out (producer,
 * MMA, epilogue, exchange, ...); bit 30: a debug-build check failed, and bit
 * 16 + s for each failing site s: 0 a TMA copy's coordinates (innermost
 * coordinate times the element size not a multiple of 16 bytes, or a store
 * starting at a negative coordinate), 1 an epilogue store, 2 an epilogue load
 * of the C that beta scales, 3 the in-kernel split-K reduction, 4 the tile
 * reduction kernel, 5 a GEMV kernel, 6 the K == 0 / alpha == 0 kernel, 7 the
 * TF32 operand transpose, 8 a block-scaled product's load or store of D, 9 the
 * quantisers, 10 routing and its balance, 11 the weighted sum, 12 the norm.  GEMM_ERR_INVALID_ARG on NULL. */
gemm_status_t gemm_plan_last_error_bits(gemm_plan_t plan, int64_t* bits);

/* 1 in the debug build of the library (libdgemm_gb300_debug.so, compiled
 * with DG_DEBUG), 0 in the release build.  The debug build checks, on the
 * device, every plain global load and store of every kernel against the
 * byte ranges of the call's own buffers (operands, output, the C that beta
 * scales, plan workspace and counters; a GEMV matrix row or a column strip
 * as a whole) and every TMA copy's coordinates against the copy rules,
 * before the access; a failed check skips the access (no trap, no fault)
 * and sets the plan's error word, which gemm_plan_poll_error reports as
 * GEMM_ERR_DEBUG_CHECK.  A skipped TMA load leaves its barrier incomplete,
 * so the bounded waits behind it run out as well.  gemm_gemv_noalloc has no
 * plan to report through and is not checked.  For its own tests the debug
 * build reads GEMM_DEBUG_SHRINK=n once per process: the output's byte
 * range is taken n bytes shorter than it is, so that the checks of the last
 * output elements fail while every access stays inside the buffer.
 * GEMM_DEBUG_SHRINK_INPUT=n does that for the groups' starts and counts and for codes that
 * are copied before a product. */
int gemm_debug_build(void);

/* Limit, in nanoseconds, of every bounded wait inside this plan's kernels
 * (default 2e9; the environment variable GEMM_WATCHDOG_NS overrides the
 * default at plan creation).  Values < 1000 are rejected. */
gemm_status_t gemm_plan_set_watchdog(gemm_plan_t plan, uint64_t timeout_ns);

/* Benchmark mode ("Matrix Multiplication Background User's Guide", section
 * 2.3: some frameworks time every implementation option once, before the
 * real work, and keep the fastest).  With enable != 0, the first
 * tensor-core gemm_run of each (M, N, K, lda, ldb, ldc, dtype, transA,
 * transB, beta != 0) on this plan times the planner's leading candidates
 * (its pick and up to five more estimated within 15% of the best): one
 * warm-up and three timed runs each, on the call's stream, writing into a
 * scratch copy of C (stream-ordered allocation the size of C; C, A and B
 * are not modified).  The fastest is kept for every later call of that
 * shape on this plan, whatever the pointers.  That first call blocks the
 * host until the trials have run (a one-time cost per shape); if anything
 * fails the planner's pick is kept.  enable = 0 (the default; the
 * environment variable GEMM_AUTOTUNE=1 turns it on at plan creation)
 * uses the planner's estimate alone.  Not applied while `stream` is being
 * captured into a CUDA graph (the planner's estimate decides there).
 * Ignored while any GEMM_FORCE_* /
 * GEMM_RASTER_GROUP / GEMM_SPLITK_CLUSTER / GEMM_TAIL_SPLIT override is set.
 * GEMM_ERR_INVALID_ARG on NULL. */
gemm_status_t gemm_plan_set_autotune(gemm_plan_t plan, int enable);

/* Number of shapes benchmark mode has timed on this plan (bounded: the
 * record is cleared past 4096 shapes).  GEMM_ERR_INVALID_ARG on NULL. */
gemm_status_t gemm_plan_tuned_count(gemm_plan_t plan, int64_t* count);

/* Watchdog self-test: launch one CTA that waits on a barrier nothing will
 * ever arrive on, with this plan's limit, then wait for `stream`.  Returns
 * GEMM_ERR_TIMEOUT when the wait ran out and the kernel returned on its own
 * (the expected result; the context stays usable), GEMM_OK if it did not. */
gemm_status_t gemm_plan_selftest_watchdog(gemm_plan_t plan, void* stream);

/* The argument checks of gemm_run without a plan or a device: returns the
 * status gemm_run would return before launching anything. */
gemm_status_t gemm_check_args(int64_t M, int64_t N, int64_t K,
                              const void* A, int64_t lda, const void* B, int64_t ldb,
                              const void* C, int64_t ldc, float alpha,
                              gemm_dtype_t dtype, gemm_op_t transA, gemm_op_t transB,
                              gemm_epilogue_t epilogue);

/* The argument checks of gemm_run_ex without a plan or a device. */
gemm_status_t gemm_check_args_ex(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                                 const void* B, int64_t ldb, const void* C, int64_t ldc,
                                 gemm_type_t c_type, const void* D, int64_t ldd, gemm_type_t d_type,
                                 float alpha, float beta, gemm_type_t ab_type, gemm_op_t transA,
                                 gemm_op_t transB, gemm_epilogue_t epilogue);

/* The planner of gemm_run as a pure host function: the decisions it would
 * make for this problem on a GPU with `sms` multiprocessors.  Does not need a
 * device.  Honours the GEMM_FORCE_TILE / GEMM_FORCE_SPLITK overrides.
 * `launches` counts the GEMM's own kernels: with TF32 operands stored
 * M/N-major, gemm_run may launch a K-major copy of one or both first (see
 * GEMM_TF32_F32), which its own record (gemm_plan_last_config) counts. */
gemm_status_t gemm_choose_config(int64_t M, int64_t N, int64_t K, gemm_dtype_t dtype,
                                 gemm_op_t transA, gemm_op_t transB, int32_t sms,
                                 gemm_config_info_t* out);

/* Tile and wave quantization of an M x N output cut into tile_m x tile_n
 * tiles, each split into `splitk` K slices, on `sms` multiprocessors running
 * `ctas_per_sm` tiles at a time ("Matrix Multiplication Background User's
 * Guide", sections 3.1 and 3.2).  Fills tiles, units, waves, tail_fraction,
 * useful_fraction, tile_m, tile_n, splitk and sms.  Pure host arithmetic. */
gemm_status_t gemm_quantization(int64_t M, int64_t N, int32_t tile_m, int32_t tile_n,
                                int32_t splitk, int32_t sms, int32_t ctas_per_sm,
                                gemm_config_info_t* out);

/* GEMV that allocates nothing.  The pages have no counterpart: this entry
 * point exists for callers that may not call cudaMalloc where they run a
 * GEMV -- a plugin inside a framework or inference server that owns all
 * device memory through its own pool allocator, or a latency-critical loop
 * that cannot take cudaMalloc's implicit device synchronisation -- and so
 * cannot create a plan (gemm_plan_create allocates) or let one grow.
 *
 * Same arguments as gemm_run, without the plan; same results as gemm_run for
 * the shapes it accepts: the column-stream GEMV, i.e. M == 1 with B stored
 * K x N (transB = GEMM_OP_N) and N >= 2, or N == 1 with A stored K x M
 * (transA = GEMM_OP_T); K >= 1, alpha != 0; the matrix operand 16-byte
 * aligned with ld * 2 a multiple of 16 bytes.  Other shapes, and outputs
 * longer than 2,097,152 elements (the fixed scratch), return
 * GEMM_ERR_UNSUPPORTED before anything is launched; argument errors are
 * those of gemm_run.
 *
 * Runs on the calling thread's current device; `stream` must belong to it.
 * Its scratch is a fixed 4 MiB device array of the library; the call zeroes
 * the part that must start at zero.  CUDA loads the library's device code
 * lazily: the first call on a device looks up that array's address
 * (cudaGetSymbolAddress), which loads it there and takes its 4 MiB from the
 * device's free memory until the process exits (GEMM_ERR_OUT_OF_MEMORY if no
 * room is left).  Make that first call before a pool allocator reserves the
 * device's memory, and before any stream capture; later calls allocate
 * nothing.  All calls on a device share the array: calls whose kernels may
 * overlap on the GPU race and must be ordered by the caller (one stream, or
 * events).  No cudaMalloc, cudaFree or other allocating call is made. */
gemm_status_t gemm_gemv_noalloc(int64_t M, int64_t N, int64_t K,
                                const void* A, int64_t lda, const void* B, int64_t ldb,
                                void* C, int64_t ldc, float alpha, float beta,
                                gemm_dtype_t dtype, gemm_op_t transA, gemm_op_t transB,
                                gemm_epilogue_t epilogue, void* stream);

/* ------------------------------------------------------------------------
 * Products of 8 and 4 bits with scales for blocks of values, and what goes round them:
 * the quantisers, the norm, the experts' products, routing and its balance, and the weighted sum.
 *
 * A block-scaled matrix of R rows and K columns is two buffers:
 *   codes   R x K bytes, row-major, rows `ld` bytes apart: GEMM_TYPE_E4M3 or GEMM_TYPE_E5M2
 *   scales  one E8M0 byte b (the scale 2^(b - 127)) for each row and block of 128
 *           columns, packed: the matrix is cut into tiles of 128 rows and
 *           four blocks (512 columns); tile (r / 128, k / 512) is 512 bytes at
 *           512 * ((r / 128) * ceil(K / 512) + k / 512), and in it row r, block
 *           c = k / 128 is byte (r % 32) * 16 + (r % 128) / 32 * 4 + c % 4.
 *           gemm_scale_bytes(R, K) bytes in all; bytes of rows and blocks past the matrix
 *           are 0 as gemm_quantize writes them and must not be 255 (255 is NaN).
 * Element (r, k) stands for code * scale.  A 128 x 128 block's scale is the same
 * byte in its 128 rows.
 *
 * The calls below are asynchronous on `stream` (a cudaStream_t), ordered like
 * gemm_run's, may be captured into a CUDA graph as gemm_run may, and keep no result
 * between calls.  Some of them use plan workspace, which grows as gemm_run's does: gemm_route_map for more than 2,048
 * slots, products of codes that have to be copied first, gemm_norm_backward with dgain, and gemm_balance for more
 * than 16 tokens.  Row counts that depend on the data (counts, starts, pos, rowmap) are
 * read on the device: no call waits for them.  Errors are those of gemm_run: argument
 * problems come back before anything is launched.  Results are deterministic.
 * ------------------------------------------------------------------------ */

/* Bytes of the packed scales of a rows x cols matrix (a multiple of 512, at least 512);
 * -1 if a size is negative or past 2^31 - 1. */
int64_t gemm_scale_bytes(int64_t rows, int64_t cols);

/* Quantise X (GEMM_TYPE_BF16, F16 or F32; row r of the result is row r of X, rows
 * ldx elements apart) to codes and scales:
 *   block_rows = 1    a scale for each row and block of 128 columns
 *   block_rows = 128  a scale for each 128 x 128 block (weights)
 *   Q, SQ    the matrix as it stands (rows x cols, ldq bytes between rows); both or neither
 *   QT, SQT  the transposed matrix (cols x rows, ldqt), its blocks along rows: an operand
 *            of a gradient product; both or neither, and one of the pairs at least
 * A scale is the least power of two, 2^-127 at least, with which the block's largest
 * finite magnitude stays within the type's largest value; a code is the value over
 * the scale, rounded to nearest, ties to even.  Infinities and NaN become NaN codes and
 * do not count for the scale.  A block of zeros has the scale byte 0.
 * rowmap (device, `rows` int32; NULL: none): row r of the result is row rowmap[r] /
 * map_div of X, which has src_rows rows; where rowmap[r] is negative or leads past
 * X there is no row: the row of Q is left as it is, its scales are 0, and the column of
 * QT is zero.  With gemm_route_map's rowmap and map_div = top_k this orders tokens by expert.
 * Q, SQ, QT, SQT 16-byte aligned, ldq and ldqt multiples of 16, X and rowmap
 * aligned to their elements; no result may share a byte with an input or another result.
 * rows up to 8,388,096. */
gemm_status_t gemm_quantize(gemm_plan_t plan, int64_t rows, int64_t cols, const void* X, int64_t ldx,
                            gemm_type_t x_type, const int32_t* rowmap, int64_t map_div, int64_t src_rows,
                            gemm_type_t q_type, int32_t block_rows, void* Q, int64_t ldq, void* SQ, void* QT,
                            int64_t ldqt, void* SQT, void* stream);

/* D <- act(alpha * A @ B^T + beta * D) with block-scaled A (M x K, scales SA) and B
 * (N x K, scales SB), D M x N of GEMM_TYPE_BF16, F16 or F32.  The tensor core applies
 * the scales and accumulates in fp32; alpha, beta and act are applied in fp32 before the one
 * rounding to D's type.  A and B may be of different 8-bit types.
 *   forward            Y  = X  @ W^T      A = X  (tokens x in),   B = W   (out x in)
 *   input gradient     dX = dY @ W        A = dY (tokens x out),  B = W^T (in x out)
 *   weight gradient    dW = dY^T @ X      A = dY^T (out x tokens), B = X^T (in x tokens)
 * (W^T, dY^T and X^T are gemm_quantize's QT.)
 * M, N, K >= 0 and < 2^31; K == 0 gives D <- act(beta * D) without reading A or B; with
 * beta == 0, D is not read.  SA, SB and D 16-byte aligned; lda and ldb >= K.  A
 * matrix of codes that is 16-byte aligned with rows a multiple of 16 bytes apart is read where it is; another is copied
 * into plan workspace first (a launch more and the matrix read and written once more; the workspace grows
 * as gemm_run's does).  Rows a multiple of 32 bytes apart are read fastest: at an odd multiple of 16
 * a row's 128 bytes touch five 32-byte sectors of memory instead of four, which cost
 * 20 to 35% of a large product's time.  ldd elements between rows of D, a multiple of 16 bytes, >= N.  No byte of D may lie in A,
 * B or their scales.  D's columns past N are not written.
 * GEMM_SCALED_KERNEL=tile|pair|sliced and GEMM_SCALED_SLICES=n in the environment
 * (read at every call) override the choice of kernel. */
gemm_status_t gemm_run_scaled(gemm_plan_t plan, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                              const void* SA, gemm_type_t a_type, const void* B, int64_t ldb, const void* SB,
                              gemm_type_t b_type, void* D, int64_t ldd, gemm_type_t d_type, float alpha,
                              float beta, gemm_epilogue_t epilogue, void* stream);

/* The argument checks of gemm_run_scaled without a plan or a device. */
gemm_status_t gemm_check_scaled(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* SA,
                                gemm_type_t a_type, const void* B, int64_t ldb, const void* SB, gemm_type_t b_type,
                                const void* D, int64_t ldd, gemm_type_t d_type, float alpha, float beta,
                                gemm_epilogue_t epilogue);

/* Experts' products: for each group e, rows starts[e] .. starts[e] + counts[e] of A
 * (rows x K) times B_e^T (B_e N x K, b_group bytes after B_(e-1); its scales
 * gemm_scale_bytes(N, K) after the last group's) into the same rows of D (rows x N), as
 * gemm_run_scaled.  starts and counts (device, `groups` int32 each) are gemm_route_map's:
 * starts are multiples of 128, so that a group's rows begin a scale tile.  A group whose start is no
 * multiple of 128 or outside [0, rows) counts as empty, a count past the end of A is cut there.  D may share no byte
 * with starts or counts either.  Rows of D that are in no group are left as they are.  What A holds in rows between groups does not matter.
 * groups <= 1024; B is read where it is if b_group is a multiple of 16 too, else the groups that have rows
 * are copied. */
gemm_status_t gemm_run_grouped(gemm_plan_t plan, int64_t groups, int64_t rows, int64_t N, int64_t K,
                               const int32_t* starts, const int32_t* counts, const void* A, int64_t lda,
                               const void* SA, gemm_type_t a_type, const void* B, int64_t ldb, int64_t b_group,
                               const void* SB, gemm_type_t b_type, void* D, int64_t ldd, gemm_type_t d_type,
                               float alpha, float beta, gemm_epilogue_t epilogue, void* stream);

/* Experts' weight gradients: for each group e, columns starts[e] .. starts[e] + counts[e] of A
 * (M x rows) times the same columns of B (N x rows), summed over them, into D_e
 * (M x N, d_group elements after D_(e-1)): D_e <- act(alpha * A_e @ B_e^T + beta * D_e).
 * A and B are gemm_quantize's QT of rows in gemm_route_map's order; the columns from a group's end to
 * the next multiple of 128 are read and must be zero, as gemm_quantize leaves them.  An
 * empty group gives D_e <- act(beta * D_e). */
gemm_status_t gemm_run_grouped_k(gemm_plan_t plan, int64_t groups, int64_t M, int64_t N, int64_t rows,
                                 const int32_t* starts, const int32_t* counts, const void* A, int64_t lda,
                                 const void* SA, gemm_type_t a_type, const void* B, int64_t ldb, const void* SB,
                                 gemm_type_t b_type, void* D, int64_t ldd, int64_t d_group, gemm_type_t d_type,
                                 float alpha, float beta, gemm_epilogue_t epilogue, void* stream);

/* ---- 4 bits ----
 * A matrix of 4-bit values (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) of R rows and K columns is two buffers:
 *   codes   (K + 1) / 2 bytes a row, rows `ld` bytes apart: column 2i in the low, 2i + 1 in the high four bits of
 *           byte i.  With odd K the last byte's high four bits must be 0, as gemm_quantize_mx leaves them.
 *   scales  one E8M0 byte for each row and block of 32 columns, in the same tiles as above: 128 rows and four
 *           blocks (here 128 columns), tile (r / 128, k / 128) at 512 * ((r / 128) * ceil(K / 128) + k / 128), in it row r,
 *           block c = k / 32 at byte (r % 32) * 16 + (r % 128) / 32 * 4 + c % 4.  gemm_mx_scale_bytes(R, K) bytes in all;
 *           bytes of rows and blocks past the matrix are 0 as gemm_quantize_mx writes them and must not be 255.
 * The scale byte 255 is NaN, and so is every value of its block. */

/* Bytes of the packed scales of a rows x cols matrix of 4-bit values (a multiple of 512, at least 512);
 * -1 if a size is negative or past 2^31 - 1. */
int64_t gemm_mx_scale_bytes(int64_t rows, int64_t cols);

/* Quantise X as gemm_quantize does, to 4-bit codes with a scale for each row and block of 32 columns: Q and SQ the
 * matrix as it stands (rows of (cols + 1) / 2 bytes), QT and SQT the transposed one (rows of (rows + 1) / 2 bytes, blocks
 * of 32 rows of X); both or neither of a pair, one pair at least.
 * A scale is the least power of two, 2^-127 at least, with which the block's largest magnitude stays within 6; a code is
 * the value over the scale, rounded to nearest, ties to the even code.  A block of zeros has the scale byte 0, one
 * that holds an infinity or NaN the byte 255 and codes of 0.
 * Q and QT at any address, rows any number of bytes apart (16-byte boundaries are fastest, and spare the products a
 * copy); otherwise alignment, rowmap, map_div, src_rows, aliasing and limits as in gemm_quantize, but 2^31 - 1025 columns at most. */
gemm_status_t gemm_quantize_mx(gemm_plan_t plan, int64_t rows, int64_t cols, const void* X, int64_t ldx,
                               gemm_type_t x_type, const int32_t* rowmap, int64_t map_div, int64_t src_rows, void* Q,
                               int64_t ldq, void* SQ, void* QT, int64_t ldqt, void* SQT, void* stream);

/* X <- the values that a block-scaled matrix stands for: codes Q of q_type (GEMM_TYPE_E4M3 or E5M2 with scales of
 * gemm_quantize's tiles, GEMM_TYPE_E2M1 with those of 4 bits) times their scales, to GEMM_TYPE_BF16, F16 or F32.  Products with the
 * scale are exact in fp32 unless they leave its range; one rounding to X's type, which is exact too for bf16 and fp32 while the values
 * stay within their normal numbers.  The way back from weights kept in 8 or 4 bits to gemm_run's operands.
 * Q at any address, rows ldq bytes apart (8 codes on a boundary of their size are read fastest), SQ 16-byte aligned, X
 * aligned to its element (rows on 16-byte boundaries are faster); X may share no byte with Q or SQ.  2^31 - 1025 rows or
 * columns at most. */
gemm_status_t gemm_dequantize(gemm_plan_t plan, int64_t rows, int64_t cols, const void* Q, int64_t ldq, gemm_type_t q_type,
                              const void* SQ, void* X, int64_t ldx, gemm_type_t x_type, void* stream);

/* D <- act(alpha * A @ B^T + beta * D) with 4-bit A (M x K) and B (N x K): gemm_run_scaled with codes of 4 bits and
 * scales of blocks of 32; lda and ldb are bytes, >= (K + 1) / 2.  Everything else as there, but that GELU and SiLU of larger calls
 * with 16-bit results are computed to 2^-18 (GEMM_TYPE_F16) or 2^-16 (GEMM_TYPE_BF16) of the result before it is rounded: one
 * next to a rounding border may fall to either side with M, N, K and groups.  SiLU is 0 below -87.3, where it is less than 2^-119
 * in size. */
gemm_status_t gemm_run_mx(gemm_plan_t plan, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* SA,
                          const void* B, int64_t ldb, const void* SB, void* D, int64_t ldd, gemm_type_t d_type,
                          float alpha, float beta, gemm_epilogue_t epilogue, void* stream);

/* The argument checks of gemm_run_mx without a plan or a device. */
gemm_status_t gemm_check_mx(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* SA, const void* B,
                            int64_t ldb, const void* SB, const void* D, int64_t ldd, gemm_type_t d_type, float alpha,
                            float beta, gemm_epilogue_t epilogue);

/* Experts' products with 4-bit rows and weights: gemm_run_grouped with codes of 4 bits and scales of blocks of 32
 * (lda, ldb and b_group are bytes; a group's scales gemm_mx_scale_bytes(N, K) after the last one's).
 * gemm_quantize_mx with gemm_route_map's rowmap orders the tokens by expert. */
gemm_status_t gemm_run_grouped_mx(gemm_plan_t plan, int64_t groups, int64_t rows, int64_t N, int64_t K,
                                  const int32_t* starts, const int32_t* counts, const void* A, int64_t lda,
                                  const void* SA, const void* B, int64_t ldb, int64_t b_group, const void* SB, void* D,
                                  int64_t ldd, gemm_type_t d_type, float alpha, float beta, gemm_epilogue_t epilogue,
                                  void* stream);

/* ---- norm ----
 * Root-mean-square norm of a residual stream, row by row (rows x cols):
 *   h = X + residual      rstd = 1 / sqrt(mean(h^2) + eps)      y = h * rstd * gain
 *   residual, H  of h_type, which is X's type or GEMM_TYPE_F32; residual NULL: h = X; H (the stream for the next layer,
 *                and what the backward pass reads) NULL: not kept
 *   gain         cols values of g_type, X's type or GEMM_TYPE_F32; NULL: ones
 *   Y            the result in X's type, NULL: not wanted
 *   Q, SQ        the result as codes of q_type (GEMM_TYPE_E4M3 or E5M2) with scales for each row and block of 128
 *                columns, exactly what gemm_quantize makes of the 32-bit result: an operand for gemm_run_scaled
 *                and gemm_run_grouped; both or neither
 *   rstd         rows floats, NULL: not wanted
 * One of H, Y, Q and rstd at least.  Sums, rstd and products are fp32; Y and the codes are rounded once, from the unrounded h (H is
 * rounded on its own).  A row whose sum of squares is past fp32's largest number (4096 values of 3e17) has rstd 0; squares below 2^-149
 * add nothing, which shows where eps is 0 or next to it: a row of values below 2^-75 has the rstd of zeros.
 * H may be X or the residual themselves (the same address, stride and type), Y too, not both the same; results
 * share no byte with inputs or each other otherwise.  cols <= 32768.  Everything needs only its element's
 * alignment (rows and gain on 16-byte boundaries are faster), Q and SQ 16 bytes with ldq a multiple of 16.
 * eps is finite and not negative. */
gemm_status_t gemm_norm(gemm_plan_t plan, int64_t rows, int64_t cols, const void* X, int64_t ldx, gemm_type_t x_type,
                        const void* residual, int64_t ldr, gemm_type_t h_type, const void* gain, gemm_type_t g_type,
                        float eps, void* H, int64_t ldh, void* Y, int64_t ldy, gemm_type_t q_type, void* Q, int64_t ldq,
                        void* SQ, float* rstd, void* stream);

/* Gradients of gemm_norm from dY (rows x cols, x_type), the kept H (h_type) and rstd:
 *   dX = rstd * (g - xhat * mean(g * xhat)) + dH,  g = dY * gain,  xhat = H * rstd     dgain = sum over rows of dY * xhat
 * dX (h_type) is the gradient of X and of the residual alike; dH (h_type, NULL: none) is the gradient that reaches h past the
 * norm.  dgain: cols floats, overwritten (zeros for no rows), NULL: not wanted.
 * dX may be dY or dH themselves (the same address, stride and type); otherwise results share no byte with inputs
 * or each other.  Limits and alignment as in gemm_norm. */
gemm_status_t gemm_norm_backward(gemm_plan_t plan, int64_t rows, int64_t cols, const void* dY, int64_t lddy,
                                 gemm_type_t x_type, const void* H, int64_t ldh, gemm_type_t h_type, const void* gain,
                                 gemm_type_t g_type, const float* rstd, const void* dH, int64_t lddh, void* dX, int64_t lddx,
                                 float* dgain, void* stream);

/* ---- routing ---- */

typedef enum { GEMM_SCORE_SOFTMAX = 0, GEMM_SCORE_SIGMOID = 1 } gemm_score_t;

/* How tokens choose experts. */
typedef struct {
  int32_t score;       /* gemm_score_t: softmax over all experts, or each expert's sigmoid      */
  int32_t top_k;       /* experts a token goes to, 1 .. 32                                      */
  int32_t groups;      /* equal groups of consecutive experts, 1 .. 32                          */
  int32_t top_groups;  /* groups a token chooses from                                           */
  int32_t group_top;   /* a group ranks by its best key (1) or its two best keys' sum (2)       */
  int32_t renormalize; /* != 0: weights are scores over the sum of the chosen ones              */
  float scale;         /* factor of the weights                                                 */
} gemm_route_t;

/* Route tokens: logits (tokens x experts, GEMM_TYPE_F32, BF16 or F16, rows ldl
 * elements apart) -> the top_k experts of each token in descending order of their keys
 * (indices) and their weights (both tokens x top_k, contiguous).
 * Scores s are computed in fp32.  The key is s + bias (bias: device, `experts`
 * floats, for balance: it takes part in the choice, not in the weights), or without a
 * bias and with group_top = 1 the logit itself, whose order is the same.  Equal keys: the lowest index first, of
 * groups too.  A logit of minus infinity or NaN masks its expert: its score is 0 and its
 * key below every other of its group choice; where fewer than top_k experts are left, masked ones of
 * the chosen groups follow in order of index, with weight 0.  Experts of other groups are never chosen.
 * Renormalising a sum of 0 gives weights 0.
 * weights and indices may share no byte with each other, the logits or the bias.
 * experts <= 1024, a multiple of groups, and top_k <= experts of top_groups groups. */
gemm_status_t gemm_route(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ldl,
                         gemm_type_t l_type, const float* bias, gemm_route_t route, float* weights, int32_t* indices,
                         void* stream);

/* Gradient of gemm_route: dlogits (tokens x experts, of the logits' type, every entry written)
 * from dweights (tokens x top_k) and the choice it made (indices; one outside [0,
 * experts) takes no part).  The choice itself has no gradient.  Of `route`, score, top_k,
 * renormalize and scale are used.  dlogits may be the logits themselves (the same
 * address and stride), and may share no byte with an input otherwise. */
gemm_status_t gemm_route_backward(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ldl,
                                  gemm_type_t l_type, gemm_route_t route, const int32_t* indices,
                                  const float* dweights, void* dlogits, int64_t lddl, void* stream);

/* How evenly a choice (indices, tokens x top_k, gemm_route's or any other's) spreads the tokens over the experts.  With p[t, e] the
 * softmax of token t's logits, or each expert's sigmoid over the sum of them all; over the m tokens that have an index in [0,
 * experts) and the n such indices, counts[e] of them expert e's:
 *   shares[e] = mean over those tokens of p[t, e]      loss = scale * experts * sum over e of counts[e] / n * shares[e]
 *   factor[e] = scale * experts * counts[e] / (n * m), the derivative of the loss by p[t, e] (the counts have none)
 * (each `experts` long; loss one float).  An even router's loss is `scale`.  A token whose indices are all outside (padding,
 * marked with -1) takes no part, nor does one whose logits are all masked add to the shares; without any tokens all
 * results are 0.  Masked logits as in gemm_route.  Shares are ratios: sigmoids too small for fp32 have the shares of their ratio.
 * Results may share no byte with each other, the logits or indices.  experts <= 1024, top_k <= 32. */
gemm_status_t gemm_balance(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ldl,
                           gemm_type_t l_type, gemm_score_t score, int32_t top_k, const int32_t* indices, float scale,
                           int32_t* counts, float* shares, float* factor, float* loss, void* stream);

/* Gradient of gemm_balance's loss: dlogits (tokens x experts, of the logits' type) <- (accumulate != 0: dlogits +) dloss *
 * d loss / d logits, from its factor; every entry is written, 0 (or itself) for tokens that take no part.  dloss: device, one
 * float, NULL for 1.  accumulate adds in fp32 with one rounding, to gemm_route_backward's result for one.  dlogits may be
 * the logits themselves (the same address and stride) unless it accumulates, and may share no byte with an input otherwise. */
gemm_status_t gemm_balance_backward(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ldl,
                                    gemm_type_t l_type, gemm_score_t score, int32_t top_k, const int32_t* indices,
                                    const float* factor, const float* dloss, int32_t accumulate, void* dlogits, int64_t lddl,
                                    void* stream);

/* Rows that gemm_route_map's order may take: tokens * top_k, and up to 127 empty rows for each expert
 * that has one, rounded up to 128; -1 if a size is out of range. */
int64_t gemm_route_rows(int64_t tokens, int64_t top_k, int64_t experts);

/* The order of the slots (slot = token * top_k + choice) by expert: expert e's slots, in their
 * own order, take rows starts[e] .. starts[e] + counts[e], starts[e] the next multiple of 128
 * after the experts before.  pos[slot] is the slot's row (-1 where its index is outside [0, experts)),
 * rowmap[row] the row's slot (-1: none), for `rows` rows, gemm_route_rows(...) at least.
 * starts, counts, pos and rowmap may share no byte with each other or with indices. */
gemm_status_t gemm_route_map(gemm_plan_t plan, int64_t tokens, int64_t top_k, int64_t experts, const int32_t* indices,
                             int32_t* starts, int32_t* counts, int32_t* pos, int32_t* rowmap, int64_t rows,
                             void* stream);

/* out[t] <- sum over j of weights[t, j] * Y[pos[t, j]], in fp32 with one rounding: the experts' rows
 * (Y rows x cols) back into tokens (out tokens x cols).  A pos that is negative or >= rows adds
 * nothing.  Y and out are of any of GEMM_TYPE_F32, BF16, F16 and need only their element's alignment (rows
 * on 16-byte boundaries are faster); out may not share a byte with Y, pos or weights. */
gemm_status_t gemm_combine(gemm_plan_t plan, int64_t tokens, int64_t top_k, int64_t cols, int64_t rows, const void* Y,
                           int64_t ldy, gemm_type_t y_type, const int32_t* pos, const float* weights, void* out,
                           int64_t ldo, gemm_type_t out_type, void* stream);

/* Gradients of gemm_combine from dout (tokens x cols, out_type): dY[pos[t, j]] <-
 * weights[t, j] * dout[t] (dY of Y's type) and dweights[t, j] <- <dout[t], Y[pos[t, j]]> (0
 * where pos leads nowhere).  pos must name no row twice, as gemm_route_map's does not.  With rowmap (`rows`
 * int32; NULL: none) the rows of dY that hold no slot are set to zero; other rows are left as they are.
 * dweights may be the weights themselves (the same address); dY and dweights may share no byte with each
 * other or an input otherwise. */
gemm_status_t gemm_combine_backward(gemm_plan_t plan, int64_t tokens, int64_t top_k, int64_t cols, int64_t rows,
                                    const void* dout, int64_t ldo, gemm_type_t out_type, const void* Y, int64_t ldy,
                                    gemm_type_t y_type, const int32_t* pos, const float* weights,
                                    const int32_t* rowmap, void* dY, int64_t lddy, float* dweights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DGEMM_GB300_GEMM_H */
