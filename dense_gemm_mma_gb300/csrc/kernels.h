// kernels.h -- parameter blocks and launchers shared by the host planner
// (api.cpp) and the CUDA kernels.  Internal to the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dg {

// Output kinds of the tensor-core epilogue and of the GEMV / reduction kernels.
enum OutKind : int {
  OUT_F32 = 0,
  OUT_BF16 = 1,
  OUT_F16 = 2
};

// Debug build (compiled with DG_DEBUG into libdgemm_gb300_debug.so): every
// kernel checks each plain global load and store against the byte ranges of
// the call's own buffers (operands, output, the C that beta scales, plan
// workspace and counters), and each TMA copy's coordinates against the copy
// rules (innermost coordinate times the element size a multiple of 16 bytes;
// a store starts at non-negative coordinates), before the access.  A failed
// check skips the access and ORs DBG_FLAG and the site's bit (bit
// DBG_SITE_SHIFT + site) into the plan's error word, where
// gemm_plan_poll_error finds it.  A skipped TMA load never completes its
// barrier, so the waits behind it run out and add their own codes.  The
// release build compiles every check out.
enum DbgSite : int {
  DBG_TMA = 0,        // a TMA copy's coordinates break the copy rules
  DBG_EPI_STORE = 1,  // tensor-core epilogue: plain or bulk store of outputs
  DBG_EPI_LOAD = 2,   // tensor-core epilogue: plain load of the C that beta scales
  DBG_SPLIT = 3,      // K slices reduced inside the tensor-core kernel: partials, counters
  DBG_REDUCE = 4,     // tile reduction kernel
  DBG_GEMV = 5,       // GEMV kernels: matrix, vector, output, partials, counters
  DBG_SCALE = 6,      // the K == 0 / alpha == 0 kernel
  DBG_TRANSPOSE = 7,  // the TF32 operand transpose
  DBG_SCALED = 8,     // 8-bit products: plain loads and stores of D
  DBG_QUANTIZE = 9,   // the quantiser
  DBG_ROUTE = 10,     // routing, its map and its gradient
  DBG_COMBINE = 11,   // the weighted sum of rows and its gradients
  DBG_NORM = 12       // the norm and its gradients
};
constexpr int DBG_SITE_SHIFT = 16;
constexpr int DBG_FLAG = 1 << 30;
constexpr int kDbgSpans = 8;
struct DbgSpans {
  uint64_t lo[kDbgSpans], hi[kDbgSpans];  // [lo, hi) byte ranges; unused entries have lo == hi
  int* err;                               // the plan's error word
};
#ifdef DG_DEBUG
#define DG_DEBUG_FIELD DbgSpans dbg;
#else
#define DG_DEBUG_FIELD
#endif

// Codes OR-ed into the plan's error word by a wait that ran out.
enum WaitCode : int {
  WAIT_PRODUCER_EMPTY = 1,
  WAIT_MMA_FULL = 2,
  WAIT_MMA_TMEM_EMPTY = 4,
  WAIT_EPI_TMEM_FULL = 8,
  WAIT_EPI_C_LOAD = 16,
  WAIT_DRAIN = 32,
  WAIT_SELFTEST = 64,
  WAIT_EPI_EXCHANGE = 128,  // K pair: the peer CTA's partial sums or its free buffers
  WAIT_SPLIT_PEERS = 256,   // split-K reduced in the GEMM kernel: the tile's other K slices
  WAIT_SPLIT_LOAD = 512,    // ... or the bulk loads of the published slices
  WAIT_SLICES = 1024        // 8-bit products: the partial sums of a tile's other K slices
};

// Variants of the tensor-core kernel.
enum TcMode : int {
  TC_SOLO = 0,  // one CTA per 128-row tile (K optionally split over units + reduction kernel)
  TC_PAIR = 1,  // a cluster of two CTAs computes one 256-row tile with .cta_group::2 MMAs
  TC_KPAIR = 2  // a cluster of two CTAs splits the K loop of one 128-row tile in halves;
                // the halves' partial sums are exchanged through distributed shared
                // memory and each CTA finishes half of the tile's columns
};

constexpr int TC_BM = 128;       // output rows per tile (one tcgen05.mma M=128)
constexpr int TC_BK = 64;        // 16-bit K elements per stage: 64 x 2 B = one 128-B swizzle row
constexpr int TC_BK_TF32 = 32;   // TF32 (fp32 word) K elements per stage: the same 128 bytes
constexpr int TC_THREADS = 192;  // warp 0 TMA, warp 1 MMA, warps 2-5 epilogue
constexpr int TC_EPI_WARPS = 4;

// Output tile t (raster order) -> (m_blk, n_blk): groups of `group` tile rows,
// each group walked column by column, so that tiles running at the same time
// share A row-panels and B column-panels in L2.
__host__ __device__ inline void tile_coords(int t, int num_m_blocks, int num_n_blocks, int group,
                                            int* m_blk, int* n_blk) {
  const int per_group = group * num_n_blocks;
  const int g = t / per_group;
  const int first_m = g * group;
  const int rows = num_m_blocks - first_m < group ? num_m_blocks - first_m : group;
  const int r = t - g * per_group;
  *m_blk = first_m + r % rows;
  *n_blk = r / rows;
}

struct TcParams {
  int M, N, K;
  int num_m_blocks, num_n_blocks;
  int k_blocks;      // ceil(K / k-block elements): TC_BK (bf16/fp16) or TC_BK_TF32 per k-block
  int tf32;          // operands are TF32 (the kind::tf32 instantiation; both K-major)
  int raster_group;  // output-tile rows per rasterisation group
  // Work units, in this order: dp_units whole tiles (raster positions
  // 0 .. dp_units-1, all of K, final output); then `splitk` K slices of each of
  // the tail_tiles remaining tiles, slice-major, written as raw fp32 partial
  // sums to the workspace, tile-major [slice][tail tile][TILE_M rows][BN
  // columns], and summed in slice order by the tile reduction kernel.  Plain
  // split-K is dp_units = 0; no split is tail_tiles = 0.
  int dp_units;
  int tail_tiles;
  int splitk;        // K slices of a tail tile
  // fused_reduce (GEMM_FUSED_REDUCE=1): the slices are summed inside this
  // kernel instead of by the tile reduction kernel.  Then every partial unit is the last unit of its
  // CTA (tail_tiles * splitk <= CTAs or clusters) and all are resident at
  // once; the unit publishes its partials, arrives on the tile's counter
  // (counters[tail tile], zero on entry and left zero on exit), waits for
  // all splitk * CTAs-per-unit arrivals, then sums one share of the tile's
  // elements over slices 0 .. splitk-1 in order and applies the epilogue.
  int fused_reduce;
  unsigned* counters;
  const float* ws;   // the partial workspace (the memory tmW maps)
  int kb_per_split;  // k-blocks per slice (the last one may be shorter); a K pair: per half
  int units;         // dp_units + tail_tiles * splitk (a K pair: tiles)
  int out_kind;      // OutKind of C
  int n_tma;         // columns [0, n_tma) of the output go through TMA (a 16-byte multiple per row)
  void* c_ptr;       // the output (C, or D of gemm_run_ex), for columns [n_tma, N) written directly
  int64_t ldc;
  // The C that beta scales: the output itself (cin == c_ptr, read through the
  // output's tensor map) or, with cin_direct, a separate matrix of kind
  // cin_kind read with plain loads.
  const void* cin;
  int64_t ldcin;
  int cin_kind;
  int cin_direct;
  int a_mn_major;    // A stored K x M (M contiguous)
  int b_mn_major;    // B stored K x N (N contiguous)
  uint32_t idesc;    // tcgen05 instruction descriptor
  float alpha, beta, slope;
  int act;
  int* err;          // plan error word
  uint64_t timeout_ns;
  int pdl;           // launch as a programmatic dependent of the stream's previous kernel
  DG_DEBUG_FIELD     // (debug build) the byte ranges this launch may touch
};

// Ring depth of the tensor-core kernel for a tile width and TcMode (TC_PAIR and
// TC_KPAIR exist for bn 128 and 256); -1 if none.
int tc_stages(int bn, int mode);
// Bytes of the operand ring (A and B stages) of one CTA.
int tc_ring_bytes(int bn, int mode);
// Clusters of two CTAs of a TC_PAIR / TC_KPAIR kernel that fit on the device at once.
int tc_max_clusters(int bn, int mode);

// TC_KPAIR: p.units counts tiles (one per cluster), p.kb_per_split is half the
// k-blocks (rounded up), and no unit is a tail slice (tail_tiles = 0).
// c: C (box 32 rows x 128 bytes); ws: the fp32 partial workspace (box 32 x 32),
// used only when p.tail_tiles > 0.
// p.tf32 selects the TF32 instantiation (kind::tf32, 32 K elements per k-block).
cudaError_t launch_gemm_tc(int bn, int mode, const CUtensorMap& a, const CUtensorMap& b,
                           const CUtensorMap& c, const CUtensorMap& ws, const TcParams& p, int grid,
                           cudaStream_t s);



#ifdef __CUDACC__
// Programmatic dependent launch: a kernel launched with the programmatic
// stream-serialization attribute may be scheduled before the previous kernel
// in its stream has finished (once that kernel's CTAs have all started and
// signalled, or exited), so its launch and prologue overlap that kernel's
// tail.  It must call wait_prior_grid() before it reads or writes global
// memory: that returns once the previous kernel has completed and its writes
// are visible.  In a kernel launched normally it returns at once.
__device__ __forceinline__ void wait_prior_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets a dependent grid be scheduled once every CTA of this one has called it (or exited): its
// launch and prologue overlap this grid's tail.
__device__ __forceinline__ void allow_next_grid() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Debug-build checks (see DbgSite): true when the access may go ahead.
#ifdef DG_DEBUG
__device__ __forceinline__ bool dbg_in(const DbgSpans& d, const void* ptr, int64_t bytes, int site) {
  const uint64_t a = reinterpret_cast<uint64_t>(ptr);
#pragma unroll
  for (int i = 0; i < kDbgSpans; ++i)
    if (a >= d.lo[i] && a + uint64_t(bytes) <= d.hi[i]) return true;
  atomicOr(d.err, DBG_FLAG | (1 << (DBG_SITE_SHIFT + site)));
  return false;
}
__device__ __forceinline__ bool dbg_tma(const DbgSpans& d, int x, int y, int esize, bool store) {
  if ((x * esize) % 16 == 0 && (!store || (x >= 0 && y >= 0))) return true;
  atomicOr(d.err, DBG_FLAG | (1 << (DBG_SITE_SHIFT + DBG_TMA)));
  return false;
}
#define DG_IN(spans, ptr, bytes, site) ::dg::dbg_in(spans, ptr, bytes, site)
#define DG_TMA(spans, x, y, esize, store) ::dg::dbg_tma(spans, x, y, esize, store)
#else
#define DG_IN(spans, ptr, bytes, site) true
#define DG_TMA(spans, x, y, esize, store) true
#endif

// kern<<<grid, block, smem, s>>>(args...), as a programmatic dependent if pdl.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_k(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                            bool pdl, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Output transform (gemm_act_t), in fp32: 1 LeakyReLU, 2 ReLU, 3 GELU
// (x * Phi(x), Phi through erfc so the negative tail keeps its relative
// accuracy), 4 SiLU; anything else is the identity.
__device__ __forceinline__ float apply_act(float v, int act, float slope) {
  switch (act) {
    case 1: return v < 0.f ? v * slope : v;
    case 2: return v < 0.f ? 0.f : v;
    case 3: return 0.5f * v * erfcf(-v * 0.70710678118654752f);
    case 4: return v / (1.f + expf(-v));
    default: return v;
  }
}
#endif

struct EpiParams {
  float alpha, beta, slope;
  int act;
  int out_kind;  // OUT_F32 / OUT_BF16 / OUT_F16 of the output
  int cin_kind;  // of the C that beta scales
};

// Fixed-order sum of the K slices of the tail tiles of a tensor-core call
// (workspace layout: see TcParams), then the epilogue into C.
struct TileReduceArgs {
  const float* ws;
  int tail_tiles, splits;
  int tile0;  // raster position of the first tail tile (= dp_units)
  int tile_m, tile_n;
  int num_m_blocks, num_n_blocks, raster_group;
  int M, N;
  void* C;  // output
  int64_t ldc;
  const void* Cin;  // the C that beta scales (may be the output)
  int64_t ldcin;
  EpiParams e;
  int pdl;  // launch as a programmatic dependent of the GEMM that writes the partials
  DG_DEBUG_FIELD
};
cudaError_t launch_tile_reduce(const TileReduceArgs& a, cudaStream_t s, int sms);

// out (cols x rows, row stride ld_out) <- transpose of in (rows x cols, row
// stride ld_in), 32-bit elements: makes a TF32 operand K-major.
cudaError_t launch_transpose32(const void* in, int64_t ld_in, int rows, int cols, void* out, int64_t ld_out,
                               cudaStream_t s, const DbgSpans& dbg);

// D <- act(beta * C) (K == 0 or alpha == 0); C may be D.
// dbg: the byte ranges the kernel may touch (checked by the debug build only).
cudaError_t launch_scale(int M, int N, void* D, int64_t ldd, const void* C, int64_t ldc, EpiParams e,
                         cudaStream_t s, int sms, const DbgSpans& dbg);

// GEMV, operand type in_f16 (0 = bf16, 1 = fp16).
// rowdot:    out[r*inc_out] = epi(sum_k W[r*ldw + k] * x[k*incx]),  r < R
// colstream: out[c*inc_out] = epi(sum_k W[k*ldw + c] * x[k*incx]),  c < R
// generic:   out[r*inc_out] = epi(sum_k W[r*w_rs + k*w_cs] * x[k*incx])
struct GemvArgs {
  const void* W;
  int64_t ldw;
  int64_t w_rs, w_cs;  // generic strides (elements)
  int R, K;
  const void* x;
  int64_t incx;
  void* out;
  int64_t inc_out;
  const void* cin;  // the C that beta scales, element r at cin[r * inc_cin] (may be out)
  int64_t inc_cin;
  int in_f16;
  EpiParams e;
  int pdl;  // launch as a programmatic dependent of the stream's previous kernel
  DG_DEBUG_FIELD
};

int gemv_rowdot_max_k();
// grid_out (optional): the CTAs launched (one wave, sized from the occupancy query).
cudaError_t launch_gemv_rowdot(const GemvArgs& g, cudaStream_t s, int sms, int* grid_out = nullptr);

// Plan of the column-stream kernel: `ksplit` K slices of `kc` rows each.
struct ColstreamPlan {
  int cols;    // columns per CTA (panel width)
  int panels;  // ceil(R / cols)
  int ksplit;
  int kc;
  int64_t ws_bytes;  // fp32 partials, ksplit x panels x cols (0 when ksplit == 1)
};
ColstreamPlan plan_gemv_colstream(int R, int K, int sms);
// counters: `panels` words that are zero on entry and are left zero on exit.
cudaError_t launch_gemv_colstream(const GemvArgs& g, const ColstreamPlan& cp, void* ws,
                                  unsigned* counters, cudaStream_t s);

cudaError_t launch_gemv_generic(const GemvArgs& g, cudaStream_t s, int sms, int* grid_out = nullptr);

// One CTA waits on a barrier that nothing arrives on; gives up after timeout_ns.
cudaError_t launch_watchdog_selftest(int* err, uint64_t timeout_ns, cudaStream_t s);

// ------------------------------------------------ 8-bit block-scaled products

// How the rows of a product are grouped.
enum ScGroup : int {
  SC_DENSE = 0,  // one product
  SC_ROWS = 1,   // group e: rows starts[e] .. starts[e] + counts[e] of A and D, its own B
  SC_K = 2       // group e: those columns (along K) of A and B, its own D
};

constexpr int SC_BK = 128;           // K values per ring stage: one 128-byte swizzle row, one scale
constexpr int SC_MAX_GROUPS = 1024;  // groups whose tile counts fit the kernels' table
constexpr int SC_MAX_TILES = 1 << 30;  // output tiles of a call

struct ScParams {
  int M, N;        // rows of A and of B (of one group's B)
  int group;       // ScGroup
  int groups;
  const int* starts;  // device: multiples of 128
  const int* counts;
  int cap;            // rows (SC_ROWS: of A and D) or K values (SC_K) that starts / counts may reach
  int m_blocks, n_blocks;  // tiles (SC_ROWS: m_blocks is per group, in the kernel)
  int k_blocks;       // of one product (SC_K: of cap)
  int raster;         // output-tile rows per rasterisation group
  int units;          // tiles (SC_ROWS: counted in the kernel)
  // 512-byte scale tiles (128 rows x 4 k-blocks): tile of row block r, k-blocks
  // 4g .. 4g+3 is number r * sa_cols + g; group e's B scales start at e * sb_group
  int sa_cols, sb_cols, sb_group;
  int out_kind;
  int n_tma;          // columns [0, n_tma) of D go through TMA (a 16-byte multiple per row)
  void* d;
  int64_t ldd, d_group;  // elements between rows, between groups' D (SC_K)
  float alpha, beta, slope;
  int act;
  uint32_t idesc;     // tcgen05 instruction descriptor, scale ids zero
  int bn;             // sliced kernel: rows of A per tile at most (32, 64, 96 or 128; a call with several tiles of rows: 128)
  int stages;         // sliced kernel: ring depth
  int part_rows;      // sliced kernel: rows of A in the partial tile (bn; one slice: 32)
  int slices;         // sliced kernel: CTAs of a cluster, each with kb_per_slice k-blocks of the tile
  int kb_per_slice;
  int* err;
  uint64_t timeout_ns;
  int pdl;
  DG_DEBUG_FIELD
};

struct ScMaps {
  CUtensorMap a, b, d, sa, sb;
};

// Tile kernel: `pair` = 256 x 256 tiles on a cluster of two CTAs, else 128 x 128
// tiles; maps: a (box 128 values x 128 rows), b (box 128 values x 128 rows),
// d (box 128 bytes x 32 rows), sa and sb (box one scale tile).
cudaError_t launch_scaled_tile(bool pair, const ScMaps& m, const ScParams& p, int grid, cudaStream_t s);
int scaled_tile_clusters();  // pairs that can be resident at once
int scaled_tile_stages(bool pair);
// Sliced kernel: tiles of 128 rows of B x bn rows of A; maps: a (box 128 values x
// 32 rows), b (box 128 values x 128 rows).  idesc: N zero.
cudaError_t launch_scaled_sliced(const ScMaps& m, const ScParams& p, int grid, cudaStream_t s);
int scaled_sliced_smem(int bn, int stages, int part_rows);
int scaled_sliced_clusters(int slices);  // clusters of that many CTAs that can be resident at once, a CTA an SM

// The same for 4-bit operands (E2M1, scales of blocks of 32): maps a and b of bytes, two values each; sa and sb
// with a row block's scale tiles as their second coordinate and the row block as their third (box two tiles; sb for a pair: of two row blocks).
cudaError_t launch_mx4_tile(bool pair, const ScMaps& m, const ScParams& p, int grid, cudaStream_t s);
int mx4_tile_clusters();
int mx4_tile_stages(bool pair, const ScParams& p);
int mx4_tile_box_row(bool pair, const ScParams& p);  // bytes of a row of the boxes that results are stored in, and of their swizzle
cudaError_t launch_mx4_sliced(const ScMaps& m, const ScParams& p, int grid, cudaStream_t s);
int mx4_sliced_smem(int bn, int stages, int part_rows);
int mx4_sliced_clusters(int slices);

// Rows of `cols` bytes (groups x rows of them, `ld` bytes apart, groups `group` bytes apart) copied
// to rows of `ld_out` bytes, a multiple of 16: makes a code matrix whose rows the TMA cannot address one
// that it can.  With counts, groups that have none are left out.
struct RepackArgs {
  const uint8_t* in;
  int64_t ld, group;
  int cols, rows, groups;
  const int* counts;
  uint8_t* out;
  int64_t ld_out;
  int pdl;
  DG_DEBUG_FIELD
};
cudaError_t launch_repack(const RepackArgs& a, cudaStream_t s);

// --------------------------------------------------------------- quantiser

struct QuantArgs {
  const void* x;
  int64_t ldx;
  int x_kind;  // OutKind of X
  int rows, cols;  // of the result; row r is row rowmap[r] / map_div of X (no map: row r)
  int rows_padded, cols_padded;  // to whole scale tiles (multiples of 128)
  const int* rowmap;  // a negative entry, or one past src_rows: no row
  int map_div, src_rows;
  int block_rows;  // 1 or 128
  int e5m2;
  int vec;         // rows of X allow four values a load
  uint8_t *q, *sq, *qt, *sqt;  // q / sq or qt / sqt may be null
  int64_t ldq, ldqt;
  int q_groups, qt_groups;  // groups of four blocks along the rows of q / of qt
  int x_words, q_wide, qt_wide;  // 4 bits: rows of X allow words, of q too, of qt 16 bytes
  int pdl;
  DG_DEBUG_FIELD
};
cudaError_t launch_quantize(const QuantArgs& a, cudaStream_t s);

// The same into 4 bits (E2M1, a scale for each row and block of 32): cols values are (cols + 1) / 2 bytes;
// block_rows, e5m2 and cols_padded are not used, q_groups and qt_groups count blocks in fours as above.
cudaError_t launch_quantize_mx4(const QuantArgs& a, int sms, cudaStream_t s);

enum CodeKind : int { CODE_E4M3 = 0, CODE_E5M2 = 1, CODE_E2M1 = 2 };

// Values of a block-scaled matrix.
struct DequantArgs {
  const uint8_t* q;
  int64_t ldq;
  const uint8_t* sq;
  int code;      // CodeKind
  int rows, cols;
  int groups;    // groups of four blocks along a row
  void* x;
  int64_t ldx;
  int x_kind;
  int wide;      // rows of X on 16-byte boundaries
  int q_wide;    // eight codes of a row on a boundary of their size
  int pdl;
  DG_DEBUG_FIELD
};
cudaError_t launch_dequantize(const DequantArgs& a, cudaStream_t s);

// -------------------------------------------------------------------- norm

constexpr int NORM_MAX_COLS = 32768;  // a row stays in the registers of a CTA

struct NormArgs {
  int rows, cols;
  const void* x;
  int64_t ldx;
  int x_kind;       // OutKind of x and y
  const void* r;    // the residual, or null
  int64_t ldr;
  int h_kind;       // OutKind of r and h
  const void* gain; // or null: ones
  int g_kind;
  float eps;
  void* h;          // x + r, or null
  int64_t ldh;
  void* y;          // or null
  int64_t ldy;
  uint8_t *q, *sq;  // or null
  int64_t ldq;
  int e5m2, q_groups, rows_padded;
  float* rstd;      // or null
  int wide;         // bytes of a load that rows' and the gain's alignment allows: 16, 4 or 0 (by value)
  int warps, per;   // warps of a row, rows of a CTA (set by the launcher)
  int pdl;
  DG_DEBUG_FIELD
};
cudaError_t launch_norm(NormArgs a, int sms, cudaStream_t s);

struct NormBackArgs {
  int rows, cols;
  const void* dy;
  int64_t lddy;
  int x_kind;       // OutKind of dy
  const void* h;
  int64_t ldh;
  int h_kind;       // OutKind of h, dh and dx
  const void* gain;
  int g_kind;
  const float* rstd;
  const void* dh;   // gradient that reaches h past the norm, or null
  int64_t lddh;
  void* dx;
  int64_t lddx;
  float* dgain;     // or null
  float* parts;     // with dgain: a CTA's rows' sums of it, part_cols floats each
  int part_cols;    // (set by the launcher)
  int wide;
  int warps, per;
  int pdl;
  DG_DEBUG_FIELD
};
// Floats of a part: cols, rounded up to whole 32-byte pieces.
constexpr int norm_part_cols(int64_t cols) { return int((cols + 7) / 8 * 8); }
// CTAs of the gradients' first launch, each of which leaves one part of the gain's: those that are resident at once.
int norm_backward_grid(int x_kind, int h_kind, int64_t rows, int64_t cols, int sms);
cudaError_t launch_norm_backward(NormBackArgs a, int grid, cudaStream_t s);

// ----------------------------------------------------------------- routing

struct RouteArgs {
  int tokens, experts;
  const void* logits;
  int64_t ldl;
  int kind;  // OutKind of the logits
  const float* bias;
  int sigmoid, top_k, groups, top_groups, group_top, renormalize;
  float scale;
  float* weights;    // tokens x top_k
  int* indices;      // tokens x top_k
  // gradient
  const float* dweights;
  void* dlogits;
  int64_t lddl;
  int wide, wide_out;  // rows of the logits, of dlogits on 16-byte boundaries
  int pdl;
  DG_DEBUG_FIELD
};
constexpr int ROUTE_MAX_EXPERTS = 1024;
constexpr int ROUTE_MAX_K = 32;
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s);
cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t s);

// Balance of a router: tokens, experts, logits, ldl, kind, sigmoid, top_k, scale, indices, wide and pdl as in
// RouteArgs; for the gradient also dlogits, lddl, wide_out.
struct BalanceArgs : RouteArgs {
  int* counts;       // experts
  float* shares;     // experts
  float* factor;     // experts
  float* loss;       // one
  float* parts;      // several CTAs: balance_workspace bytes, [CTA][experts]
  unsigned* counters;  // several CTAs: experts + 2 words, zero on entry and left zero
  const float* dloss;  // gradient: null for 1
  int accumulate;      // gradient: added to what dlogits holds
};
int balance_ctas(int64_t tokens, int64_t experts, int sms);
cudaError_t launch_balance(const BalanceArgs& a, int ctas, cudaStream_t s);
cudaError_t launch_balance_backward(const BalanceArgs& a, cudaStream_t s);

struct RouteMapArgs {
  const int* indices;
  int slots;  // tokens x top_k
  int experts;
  int* starts;
  int* counts;
  int* pos;
  int* rowmap;
  int rows;  // length of rowmap
  int wide;  // rowmap on a 16-byte boundary
  int* block_counts;  // route_map_workspace bytes
  int run, warps;     // slots of a CTA, warps that share them (set by the launcher)
  int pdl;
  DG_DEBUG_FIELD
};
size_t route_map_workspace(int64_t slots, int64_t experts);
cudaError_t launch_route_map(RouteMapArgs a, cudaStream_t s);

// ----------------------------------------------------------------- combine

struct CombineArgs {
  int tokens, k, cols, rows;  // rows of Y
  const void* y;
  int64_t ldy;
  int y_kind;
  const int* pos;
  const float* weights;
  void* out;  // forward: sums; backward: their gradient (read)
  int64_t ldo;
  int o_kind;
  // backward
  const int* rowmap;
  void* dy;
  int64_t lddy;
  float* dweights;
  int wide;  // bytes of a load: 16 (whole pieces of eight columns on 16-byte boundaries in every row), 4, or 0: by element
  int pdl;
  DG_DEBUG_FIELD
};
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t s);
cudaError_t launch_combine_backward(const CombineArgs& a, cudaStream_t s);

}  // namespace dg
