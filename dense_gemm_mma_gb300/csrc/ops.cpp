// ops.cpp -- the C ABI of the block-scaled products of 8 and 4 bits, the quantisers, the routing
// to experts with its balance, and the weighted sum of their rows (include/gemm.h): argument checks,
// the choice of kernel, tensor maps and launches.
#include "gemm.h"

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <utility>

#include "ops.h"

using namespace dg;

namespace {

constexpr int kSmemMax = 232448;  // shared memory of a CTA; an SM holds 1 KB more for each CTA

// 3-D row-major tensor (inner contiguous, ld elements between rows, group elements
// between groups); boxes of box_inner x box_rows x box_groups.  Out-of-range reads give zero.
bool map3(CUtensorMap* m, CUtensorMapDataType t, int64_t esize, const void* ptr, int64_t inner, int64_t rows, int64_t groups,
          int64_t ld, int64_t group, int box_inner, int box_rows, CUtensorMapSwizzle swizzle, int box_groups = 1) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cuuint64_t(inner), cuuint64_t(rows), cuuint64_t(groups)};
  cuuint64_t strides[2] = {cuuint64_t(ld * esize), cuuint64_t(group * esize)};
  cuuint32_t box[3] = {cuuint32_t(box_inner), cuuint32_t(box_rows), cuuint32_t(box_groups)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, t, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A product as its callers give it.
struct Product {
  const char* name = "gemm_run_scaled";
  bool four = false;  // 4-bit operands (scales of blocks of 32), else 8-bit ones
  int group = SC_DENSE;
  int64_t groups = 1;
  int64_t M = 0, N = 0, K = 0;  // SC_ROWS: M = rows of A and D; SC_K: K = columns of A and B
  const int32_t* starts = nullptr;
  const int32_t* counts = nullptr;
  const void* A = nullptr;
  int64_t lda = 0;
  const void* SA = nullptr;
  gemm_type_t a_type = GEMM_TYPE_E4M3;
  const void* B = nullptr;
  int64_t ldb = 0, b_group = 0;
  const void* SB = nullptr;
  gemm_type_t b_type = GEMM_TYPE_E4M3;
  void* D = nullptr;
  int64_t ldd = 0, d_group = 0;
  gemm_type_t d_type = GEMM_TYPE_BF16;
  float alpha = 1.f, beta = 0.f;
  gemm_epilogue_t epi{};
  bool nothing() const { return M == 0 || N == 0 || groups == 0; }
  int64_t k_bytes() const { return four ? ceil_div(K, 2) : K; }  // of a row of codes
  int64_t tiles_of(int64_t rows) const { return four ? mx4_scale_tiles(rows, K) : scale_tiles(rows, K); }
};

// Do `groups` matrices, `group` elements from one to the next, share a byte with y?  What lies between
// them is not theirs.
bool groups_meet(const void* p, int64_t groups, int64_t rows, int64_t cols, int64_t ld, int64_t group, int64_t es,
                 const Region& y) {
  if (groups <= 1 || group == rows * ld) return overlaps(region(p, std::max<int64_t>(groups, 1) * rows, cols, ld, es), y);
  if (!overlaps(region(p, 1, (groups - 1) * group + (rows - 1) * ld + cols, 0, es), y)) return false;
  for (int64_t e = 0; e < groups; ++e)
    if (overlaps(region(static_cast<const char*>(p) + e * group * es, rows, cols, ld, es), y)) return true;
  return false;
}

gemm_status_t check_product(const Product& x) {
  if (!x.four && (!is_code_type(x.a_type) || !is_code_type(x.b_type))) return GEMM_ERR_INVALID_ARG;
  if (!is_float_type(x.d_type)) return GEMM_ERR_INVALID_ARG;
  if (x.epi.act < GEMM_ACT_NONE || x.epi.act > GEMM_ACT_SILU) return GEMM_ERR_INVALID_ARG;
  if (x.M < 0 || x.N < 0 || x.K < 0 || x.groups < 0) return GEMM_ERR_INVALID_ARG;
  if (!size_ok(x.M) || !size_ok(x.N) || !size_ok(x.K) || x.groups > SC_MAX_GROUPS) return GEMM_ERR_UNSUPPORTED;
  const int64_t one = 1, kb = x.k_bytes();
  if (x.lda < std::max(one, kb) || x.ldb < std::max(one, kb) || x.ldd < std::max(one, x.N)) return GEMM_ERR_INVALID_ARG;
  if (x.nothing()) return GEMM_OK;
  const bool rows = x.group == SC_ROWS, by_k = x.group == SC_K;
  if (rows && x.groups > 1 && x.b_group < (x.N - 1) * x.ldb + kb) return GEMM_ERR_INVALID_ARG;
  if (by_k && x.groups > 1 && x.d_group < (x.M - 1) * x.ldd + x.N) return GEMM_ERR_INVALID_ARG;
  if (x.group != SC_DENSE && (!x.starts || !x.counts)) return GEMM_ERR_INVALID_ARG;
  if (!x.D) return GEMM_ERR_INVALID_ARG;
  const int64_t es = type_bytes(x.d_type);
  const auto d_meets = [&](const Region& y) {
    return groups_meet(x.D, by_k ? x.groups : 1, x.M, x.N, x.ldd, x.d_group, es, y);
  };
  if (x.group != SC_DENSE && (d_meets(run_of(x.starts, x.groups * 4)) || d_meets(run_of(x.counts, x.groups * 4))))
    return GEMM_ERR_INVALID_ARG;
  if (x.K > 0) {
    if (!x.A || !x.B || !x.SA || !x.SB) return GEMM_ERR_INVALID_ARG;
    const int64_t nb = rows ? x.groups : 1;
    if (d_meets(region(x.A, x.M, kb, x.lda, 1)) || d_meets(run_of(x.SA, x.tiles_of(x.M) * 512)) ||
        d_meets(run_of(x.SB, nb * x.tiles_of(x.N) * 512)) ||
        (rows ? groups_meet(x.B, nb, x.N, kb, x.ldb, x.b_group, 1, region(x.D, x.M, x.N, x.ldd, es))
              : d_meets(region(x.B, x.N, kb, x.ldb, 1))))
      return GEMM_ERR_INVALID_ARG;
    if (!aligned(x.SA, 16) || !aligned(x.SB, 16)) return GEMM_ERR_ALIGNMENT;
    if (x.tiles_of(x.M) > kMaxDim || nb * x.tiles_of(x.N) > kMaxDim) return GEMM_ERR_UNSUPPORTED;
  }
  if (!aligned(x.D, 16) || (x.ldd * es) % 16 || (by_k && x.groups > 1 && (x.d_group * es) % 16)) return GEMM_ERR_ALIGNMENT;
  if (x.group != SC_DENSE && (!aligned(x.starts, 4) || !aligned(x.counts, 4))) return GEMM_ERR_ALIGNMENT;
  return GEMM_OK;
}

// ---------------------------------------------------------- choice of kernel

enum ScKernel { SC_TILE, SC_PAIR, SC_SLICED };

struct ScPick {
  ScKernel kernel = SC_TILE;
  int bn = 128, slices = 1, stages = 0, part_rows = 32;
  bool four = false;
};

void set_sliced(ScPick* c, int slices) {
  c->slices = slices;
  c->part_rows = slices > 1 ? c->bn : 32;
  c->stages = 8;
  const auto smem = c->four ? mx4_sliced_smem : scaled_sliced_smem;
  while (c->stages > 2 && smem(c->bn, c->stages, c->part_rows) > kSmemMax) --c->stages;
}

// Clusters of 1 .. 8 CTAs that the device holds at once (16 tiles in 8 slices, 128 CTAs,
// took two waves: a cluster lies within one group of SMs).
struct Residency {
  int clusters[9];
  Residency(bool four, int sms) {
    clusters[0] = 0;
    clusters[1] = sms;
    for (int s = 2; s <= 8; ++s) clusters[s] = four ? mx4_sliced_clusters(s) : scaled_sliced_clusters(s);
  }
};

// Those of the 8-bit or of the 4-bit kernel, which is asked for them at the first product that may take it.
const Residency& residency(bool four, int sms) {
  if (four) {
    static const Residency fits(true, sms);
    return fits;
  }
  static const Residency fits(false, sms);
  return fits;
}

// CTA pairs that the device holds at once, of either too.
int resident_pairs(bool four) {
  if (four) {
    static const int pairs = mx4_tile_clusters();
    return pairs;
  }
  static const int pairs = scaled_tile_clusters();
  return pairs;
}

// `rows` rows of A at most in a tile, `tiles` tiles.  K is cut into as many slices as leave
// every cluster resident at once, a CTA an SM (4096 x 4096, one row: 6.2 us in 4 slices,
// 128 CTAs, against 7.9 in 5).  A slice may be empty: its CTA still takes its share of the rows that
// the slices add up (33 x 1024 x 512, four k-blocks: 5.3 us in 8 slices, 6.4 in 2).
ScPick pick_sliced(bool four, int64_t rows, int64_t tiles, int sms) {
  const Residency& fits = residency(four, sms);
  ScPick c;
  c.four = four;
  c.kernel = SC_SLICED;
  c.bn = int(std::min<int64_t>(128, round_up(rows, 32)));
  int s = 8;
  while (s > 1 && fits.clusters[s] < tiles) --s;
  set_sliced(&c, s);
  return c;
}

// Rows of a group up to which the sliced kernel is faster than 128 x 128 tiles (32 experts of 2048 x 2048:
// 32 rows each 30.2 against 33.3 us, 64 rows 35.4 against 33.2).
// 4 bits, the same experts: 16 rows 20.4 and 20.2 us, 32 rows 21.5 and 20.1, 64 rows 24.3 and 20.9.
constexpr int64_t kFewRows = 48, kFewRowsMx4 = 16;

// Which kernel a product takes, by sizes alone (the counts of a grouped call are on
// the device; its rows are estimated from the capacity, which holds up to 127 empty rows a
// group).  GEMM_SCALED_KERNEL=tile|pair|sliced and GEMM_SCALED_SLICES=n override it.
ScPick pick(const Product& x, int sms) {
  const int64_t kb = ceil_div(x.k_bytes(), SC_BK), nb = ceil_div(x.N, 128), mb = ceil_div(x.M, 128);
  ScPick c;
  c.four = x.four;
  if (x.group == SC_ROWS) {
    const int64_t per = std::max<int64_t>(1, x.M / x.groups - 127);
    const int64_t active = std::max<int64_t>(1, std::min(x.groups, x.M / 128));
    if (per <= (x.four ? kFewRowsMx4 : kFewRows))
      c = pick_sliced(x.four, 128, active * nb, sms);
    else  // (256 rows each: 53.6 us on single CTAs, 48.8 on pairs; 8 experts of 4096 x 1024, 150 rows: 14.9 and 18.3.
          // 4 bits, 32 experts of 2048 x 2048: 128 rows 22.4 and 25.3, 160 rows 31.2 and 26.7)
      c.kernel = per < (x.four ? 129 : 256) ? SC_TILE : SC_PAIR;
  } else if (x.group == SC_K) {
    // (16 gradients of 2048 x 2048: 192 rows each, 319 with the padding, 49.8 us on single CTAs, 52.3 on pairs; 384 rows
    // 60.3 and 54.6)
    c.kernel = x.K / x.groups < 512 ? SC_TILE : SC_PAIR;
  } else {
    // 128 x 128 tiles on one CTA each while they fill one wave at most (200 x 6912 x 2048: 10.6
    // us, pairs 12.3), 256 x 256 on pairs beyond (400 x 8192 x 8192: 27 us, 37 on single CTAs).
    // Fewer tiles: K slices, if what they save of the K loop (0.22 us a k-block) pays for adding up
    // the slices' rows (0.07 us a row and CTA).  735 x 6489: 800 rows 14.1 us in 3
    // slices, 19.4 whole; 128 x 6912 x 2048: 11.8 in 2 slices, 10.5 whole.  4 bits: a k-block saves more beside the
    // whole tile's longer start (0.9 us for the same choices: 128 x 4096 x 2048 8.4 in 4 slices, 9.7 whole; 128 x 8192 x 2048 10.1 in
    // 2, 9.9 whole; 256 x 4096 x 8192 14.0 in 2, 15.3 whole).
    // Up to four k-blocks of 4 bits, two and a half waves on single CTAs (1200 x 2048 x 512: 9.2 us, pairs 10.5; 512 x 6912 x 1024 10.5 and
    // 11.2).
    const int64_t whole = x.four && kb <= 4 ? sms * 5 / 2 : sms;
    c.kernel = mb * nb > whole ? SC_PAIR : SC_TILE;
    if (mb * nb <= sms) {
      const ScPick sl = pick_sliced(x.four, x.M, mb * nb, sms);
      const double rows = double(std::min<int64_t>(x.M, 128)), s = sl.slices;
      if (x.M <= 64 || 0.07 * rows / s < (x.four ? 0.9 : 0.22) * double(kb) * (1 - 1 / s)) c = sl;
    }
  }
  if (const char* f = std::getenv("GEMM_SCALED_KERNEL")) {
    if (!std::strcmp(f, "tile")) c.kernel = SC_TILE;
    if (!std::strcmp(f, "pair")) c.kernel = SC_PAIR;
    if (!std::strcmp(f, "sliced") && x.group != SC_K && c.kernel != SC_SLICED)
      c = pick_sliced(x.four, x.group == SC_ROWS ? 128 : x.M, mb * nb, sms);
  }
  if (c.kernel == SC_SLICED) {
    const int s = env_int("GEMM_SCALED_SLICES", 0);
    if (s >= 1 && s <= 8) set_sliced(&c, s);
  }
  return c;
}

// Bytes of a copy of groups x rows rows of K codes, 0 if the TMA can read them as they are
// (16-byte aligned, rows and groups multiples of 16 bytes apart).
size_t repack_bytes(const void* p, int64_t ld, int64_t groups, int64_t group, int64_t rows, int64_t K) {
  if (K == 0 || (aligned(p, 16) && ld % 16 == 0 && (groups <= 1 || group % 16 == 0))) return 0;
  return size_t(groups * rows) * size_t(round_up(K, 16));
}

// Copy such a matrix into `out` (plan workspace) and make the product read it there.
gemm_status_t repack(gemm_plan* plan, const void** p, int64_t* ld, int64_t groups, int64_t* group, int64_t rows, int64_t K,
                     const int32_t* counts, void* out, cudaStream_t s) {
  if (rows * ceil_div(K, 16) > int64_t(0xffffffff)) return GEMM_ERR_UNSUPPORTED;  // (the copy counts in 32 bits)
  RepackArgs a{};
  a.in = static_cast<const uint8_t*>(*p);
  a.ld = *ld;
  a.group = *group;
  a.cols = int(K);
  a.rows = int(rows);
  a.groups = int(groups);
  a.counts = counts;
  a.out = static_cast<uint8_t*>(out);
  a.ld_out = round_up(K, 16);
  a.pdl = plan->pdl;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).input(*p, (groups - 1) * *group + (rows - 1) * *ld + K).bytes(counts, groups * 4)
              .bytes(out, groups * rows * a.ld_out).s;
#endif
  *p = out;
  *ld = a.ld_out;
  *group = rows * a.ld_out;
  return launched(launch_repack(a, s));
}

gemm_status_t run_product(gemm_plan* plan, Product x, cudaStream_t s) {
  gemm_config_info_t info{};
  info.sms = plan->sms;
  info.splitk = 1;
  if (x.nothing()) {
    info.path = GEMM_PATH_NONE;
    plan->last = info;
    return GEMM_OK;
  }
  DeviceGuard guard(plan->device);
  const int64_t b_groups = x.group == SC_ROWS ? x.groups : 1, kbytes = x.k_bytes();
  const size_t a_copy = repack_bytes(x.A, x.lda, 1, 0, x.M, kbytes);
  const size_t b_copy = repack_bytes(x.B, x.ldb, b_groups, x.b_group, x.N, kbytes);
  if (a_copy + b_copy > 0) {
    gemm_status_t st = ensure_tws(plan, a_copy + b_copy, s);
    int64_t none = 0;
    if (st == GEMM_OK && a_copy) st = repack(plan, &x.A, &x.lda, 1, &none, x.M, kbytes, nullptr, plan->tws, s);
    if (st == GEMM_OK && b_copy)
      st = repack(plan, &x.B, &x.ldb, b_groups, &x.b_group, x.N, kbytes, x.group == SC_ROWS ? x.counts : nullptr,
                  static_cast<char*>(plan->tws) + a_copy, s);
    if (st != GEMM_OK) return st;
  }
  const ScPick c = pick(x, plan->sms);
  const bool sliced = c.kernel == SC_SLICED, pair = c.kernel == SC_PAIR;
  const int64_t es = type_bytes(x.d_type);
  const int tile_m = sliced ? c.bn : pair ? 256 : 128, tile_n = sliced ? 128 : pair ? 256 : 128;
  ScParams p{};
  p.M = int(x.M);
  p.N = int(x.N);
  p.group = x.group;
  p.groups = int(x.groups);
  p.starts = x.starts;
  p.counts = x.counts;
  p.cap = int(x.group == SC_K ? x.K : x.M);
  p.m_blocks = int(ceil_div(x.M, tile_m));
  p.n_blocks = int(ceil_div(x.N, tile_n));
  p.k_blocks = int(ceil_div(kbytes, SC_BK));
  p.sa_cols = int(scale_groups(x.K));
  p.sb_cols = p.sa_cols;
  p.sb_group = int(x.four ? std::max<int64_t>(1, ceil_div(x.N, 128)) : scale_tiles(x.N, x.K));  // (4 bits: in row blocks)
  p.out_kind = type_kind(x.d_type);
  p.n_tma = int((x.N * es) / 16 * 16 / es);
  p.d = x.D;
  p.ldd = x.ldd;
  p.d_group = x.group == SC_K ? x.d_group : 0;
  p.alpha = x.alpha;
  p.beta = x.beta;
  p.act = x.epi.act;
  p.slope = x.epi.slope;
  p.bn = c.bn;
  p.stages = c.stages;
  p.part_rows = c.part_rows;
  p.slices = c.slices;
  p.kb_per_slice = int(ceil_div(p.k_blocks, c.slices));
  p.err = plan->err;
  p.timeout_ns = plan->watchdog_ns;
  p.pdl = plan->pdl;
  // tcgen05 instruction descriptor, kind::mxf8f6f4: bits 7-9 A type and 10-12 B type
  // (0 E4M3, 1 E5M2), 17-22 N>>3, 23 scale type (1 = E8M0), 24-28 M>>4; the kernels add the
  // scale ids (4-5 for B, 29-30 for A).  The sliced kernel's MMA takes B's rows as its A, and its N from the tile.
  // 4 bits, kind::mxf4: the same with 1 for E2M1, bit 31 clear (K = 64), the scale ids the kernels' too.
  const uint32_t ta = x.four || x.a_type == GEMM_TYPE_E5M2, tb = x.four || x.b_type == GEMM_TYPE_E5M2;
  const uint32_t mma_m = pair ? 256 : 128, mma_n = sliced ? 0u : uint32_t(tile_n);
  p.idesc = ((sliced ? tb : ta) << 7) | ((sliced ? ta : tb) << 10) | (mma_n >> 3 << 17) | (1u << 23) | (mma_m >> 4 << 24);
  // Groups of tile rows walked column by column: tiles that run at the same time share
  // rows of A and of B in L2.
  // (4 bits, up to eight k-blocks: 8192 x 8192 x 2048 in groups of 4 53.6 us, of 8 54.9; more: 4096 x 4096 x 8192 52.5 and 51.8,
  // 8192 x 8192 x 16384 335 and 320)
  p.raster = sliced ? std::max(1, p.m_blocks) : x.four && p.k_blocks <= 8 ? 4 : 8;
  const int64_t bound = x.group == SC_ROWS  // SC_ROWS: whole tiles and one partial tile for each group at most
                            ? (ceil_div(x.M, tile_m) + std::min<int64_t>(x.groups, ceil_div(x.M, 128))) * p.n_blocks
                            : int64_t(p.m_blocks) * p.n_blocks * (x.group == SC_K ? x.groups : 1);
  if (bound > SC_MAX_TILES) return GEMM_ERR_UNSUPPORTED;
  p.units = int(bound);
  if (x.group == SC_ROWS) p.raster = 4;
  int grid;
  if (pair) {
    const int clusters = resident_pairs(x.four);
    if (clusters <= 0) return GEMM_ERR_UNSUPPORTED;
    grid = int(2 * std::min<int64_t>(bound, clusters));
  } else if (sliced) {
    const int64_t resident = std::max<int64_t>(1, plan->sms / c.slices);
    grid = int(c.slices * (x.group == SC_ROWS ? std::min(bound, resident) : bound));
  } else {
    grid = int(std::min<int64_t>(bound, plan->sms));
  }
  ScMaps m{};
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  const int64_t nb = b_groups;
  bool ok = true;
  // a placeholder where nothing is read or stored through the map
  if (x.K == 0 || p.n_tma == 0 || sliced)
    ok = map3(&m.d, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, plan->err, 32, 32, 1, 32, 1024, 32, 32, sw);
  if (x.K > 0) {
    ok = ok && map3(&m.a, u8, 1, x.A, kbytes, x.M, 1, x.lda, x.lda * x.M, SC_BK, sliced ? 32 : 128, sw);
    ok = ok && map3(&m.b, u8, 1, x.B, kbytes, x.N, nb, x.ldb, nb > 1 ? x.b_group : x.ldb * x.N, SC_BK, 128, sw);
    const CUtensorMapDataType u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
    const CUtensorMapSwizzle plain = CU_TENSOR_MAP_SWIZZLE_NONE;
    if (x.four) {  // tiles along K, row blocks; a box holds a stage's two tiles (B, pairs: of two row blocks)
      const int64_t tk = mx4_scale_tiles(1, x.K), ma = std::max<int64_t>(1, ceil_div(x.M, 128));
      ok = ok && map3(&m.sa, u32, 4, x.SA, 128, tk, ma, 128, 128 * tk, 128, 2, plain);
      ok = ok && map3(&m.sb, u32, 4, x.SB, 128, tk, nb * p.sb_group, 128, 128 * tk, 128, 2, plain, pair ? 2 : 1);
    } else {
      const int64_t ta_n = scale_tiles(x.M, x.K), tb_n = nb * p.sb_group;
      ok = ok && map3(&m.sa, u32, 4, x.SA, 128, ta_n, 1, 128, 128 * ta_n, 128, 1, plain);
      ok = ok && map3(&m.sb, u32, 4, x.SB, 128, tb_n, 1, 128, 128 * tb_n, 128, 1, plain);
    }
  } else {
    m.a = m.b = m.sa = m.sb = m.d;
  }
  if (p.n_tma > 0 && !sliced) {
    const CUtensorMapDataType dt = x.d_type == GEMM_TYPE_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : x.d_type == GEMM_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int64_t nd = x.group == SC_K ? x.groups : 1;
    const int row = x.four ? mx4_tile_box_row(pair, p) : 128;
    ok = ok && map3(&m.d, dt, es, x.D, p.n_tma, x.M, nd, x.ldd, nd > 1 ? x.d_group : x.ldd * x.M, int(row / es), 32,
                    row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : sw);
  }
  if (!ok) return GEMM_ERR_CUDA;
#ifdef DG_DEBUG
  p.dbg = Spans(plan->err).input(x.starts, x.starts ? x.groups * 4 : 0).input(x.counts, x.counts ? x.groups * 4 : 0)
              .out_matrix(x.D, 1, x.group == SC_K ? (x.groups - 1) * x.d_group + (x.M - 1) * x.ldd + x.N
                                                             : (x.M - 1) * x.ldd + x.N, 0, es).s;
#endif
  info.path = sliced ? GEMM_PATH_SCALED_SLICED : GEMM_PATH_SCALED;
  info.tile_m = tile_m;
  info.tile_n = tile_n;
  info.tile_k = x.four ? 2 * SC_BK : SC_BK;
  info.cta_per_tile = pair ? 2 : sliced ? c.slices : 1;
  info.splitk = sliced ? c.slices : 1;
  info.stages = sliced ? c.stages : x.four ? mx4_tile_stages(pair, p) : scaled_tile_stages(pair);
  info.raster_group = p.raster;
  info.grid = grid;
  info.tiles = bound;
  info.units = bound * (sliced ? c.slices : 1);
  info.launches = 1 + int(a_copy > 0) + int(b_copy > 0);
  info.workspace_bytes = int64_t(a_copy + b_copy);
  plan->last = info;
  if (x.four) return launched(sliced ? launch_mx4_sliced(m, p, grid, s) : launch_mx4_tile(pair, m, p, grid, s));
  return launched(sliced ? launch_scaled_sliced(m, p, grid, s) : launch_scaled_tile(pair, m, p, grid, s));
}

gemm_status_t checked_run(gemm_plan_t plan, const Product& x, void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t st = check_product(x);
  if (st != GEMM_OK) return st;
  const CallScope call(plan, "%s %lldx%lldx%lld groups %lld %s %s->%s", x.name, (long long)x.M, (long long)x.N, (long long)x.K,
                       (long long)x.groups, x.four ? "mx4" : type_name(x.a_type), x.four ? "mx4" : type_name(x.b_type), type_name(x.d_type));
  return call.done(run_product(plan, x, static_cast<cudaStream_t>(stream)), &plan->last);
}

// Bytes of the weighted sum's loads and stores, given each matrix's address and bytes between rows.
int access_bytes(int64_t cols, std::initializer_list<std::pair<const void*, int64_t>> rows) {
  int wide = cols % 8 == 0 ? 16 : 4;
  for (const auto& m : rows)
    while (wide && (!aligned(m.first, size_t(wide)) || m.second % wide)) wide = wide == 16 ? 4 : 0;
  return wide;
}

gemm_status_t check_route(int64_t tokens, int64_t experts, const void* logits, int64_t ldl, gemm_type_t type,
                          const gemm_route_t& r) {
  if (tokens < 0 || experts < 1 || !is_float_type(type)) return GEMM_ERR_INVALID_ARG;
  if (r.score != GEMM_SCORE_SOFTMAX && r.score != GEMM_SCORE_SIGMOID) return GEMM_ERR_INVALID_ARG;
  if (r.top_k < 1 || r.groups < 1 || r.top_groups < 1 || r.top_groups > r.groups || (r.group_top != 1 && r.group_top != 2))
    return GEMM_ERR_INVALID_ARG;
  if (experts > ROUTE_MAX_EXPERTS || r.top_k > ROUTE_MAX_K || r.groups > 32 || !size_ok(tokens) ||
      tokens * r.top_k > kMaxDim)
    return GEMM_ERR_UNSUPPORTED;
  if (experts % r.groups || r.top_k > experts / r.groups * r.top_groups) return GEMM_ERR_INVALID_ARG;
  if (ldl < experts) return GEMM_ERR_INVALID_ARG;
  if (tokens > 0 && !logits) return GEMM_ERR_INVALID_ARG;
  return aligned(logits, size_t(type_bytes(type))) ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}

RouteArgs route_args(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ldl, gemm_type_t type,
                     const gemm_route_t& r) {
  RouteArgs a{};
  a.tokens = int(tokens);
  a.experts = int(experts);
  a.logits = logits;
  a.ldl = ldl;
  a.kind = type_kind(type);
  a.sigmoid = r.score == GEMM_SCORE_SIGMOID;
  a.top_k = r.top_k;
  a.groups = r.groups;
  a.top_groups = r.top_groups;
  a.group_top = r.group_top;
  a.renormalize = r.renormalize;
  a.scale = r.scale;
  a.wide = rows_wide(logits, ldl, type_bytes(type));
  a.pdl = plan->pdl;
  return a;
}

gemm_status_t check_balance(int64_t tokens, int64_t experts, const void* logits, int64_t ldl, gemm_type_t type,
                            gemm_score_t score, int32_t top_k, const int32_t* indices) {
  if (top_k < 1) return GEMM_ERR_INVALID_ARG;
  // (the choice may be of any router's: as many experts as choices are not asked for)
  gemm_route_t r{score, int32_t(std::min<int64_t>(top_k, std::max<int64_t>(1, experts))), 1, 1, 1, 0, 1.f};
  const gemm_status_t st = check_route(tokens, experts, logits, ldl, type, r);
  if (st != GEMM_OK) return st;
  if (top_k > ROUTE_MAX_K || tokens * top_k > kMaxDim) return GEMM_ERR_UNSUPPORTED;
  if (tokens > 0 && !indices) return GEMM_ERR_INVALID_ARG;
  return aligned(indices, 4) ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}

BalanceArgs balance_args(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ldl,
                         gemm_type_t type, gemm_score_t score, int32_t top_k, const int32_t* indices) {
  const gemm_route_t r{score, top_k, 1, 1, 1, 0, 1.f};
  BalanceArgs a{};
  static_cast<RouteArgs&>(a) = route_args(plan, tokens, experts, logits, ldl, type, r);
  a.indices = const_cast<int32_t*>(indices);
  return a;
}

gemm_status_t check_combine(int64_t tokens, int64_t top_k, int64_t cols, int64_t rows, const void* Y, int64_t ldy,
                            gemm_type_t y_type, const void* pos, const void* weights, const void* out, int64_t ldo,
                            gemm_type_t o_type) {
  if (tokens < 0 || top_k < 1 || cols < 0 || rows < 0 || !is_float_type(y_type) || !is_float_type(o_type))
    return GEMM_ERR_INVALID_ARG;
  if (!size_ok(tokens) || !size_ok(top_k) || !size_ok(cols) || !size_ok(rows) || tokens * top_k > kMaxDim ||
      cols > int64_t(65535) * 2048 || tokens + rows > kMaxDim)  // (the forward grid's second dimension)
    return GEMM_ERR_UNSUPPORTED;
  if (ldy < std::max<int64_t>(1, cols) || ldo < std::max<int64_t>(1, cols)) return GEMM_ERR_INVALID_ARG;
  if (tokens == 0 || cols == 0) return GEMM_OK;
  if (!pos || !weights || !out || (rows > 0 && !Y)) return GEMM_ERR_INVALID_ARG;
  if (!aligned(pos, 4) || !aligned(weights, 4) || !aligned(Y, size_t(type_bytes(y_type))) ||
      !aligned(out, size_t(type_bytes(o_type))))
    return GEMM_ERR_ALIGNMENT;
  return GEMM_OK;
}

}  // namespace

extern "C" {

int64_t gemm_scale_bytes(int64_t rows, int64_t cols) {
  return size_ok(rows) && size_ok(cols) ? scale_tiles(rows, cols) * 512 : -1;
}

gemm_status_t gemm_check_scaled(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* SA,
                                gemm_type_t a_type, const void* B, int64_t ldb, const void* SB, gemm_type_t b_type,
                                const void* D, int64_t ldd, gemm_type_t d_type, float alpha, float beta,
                                gemm_epilogue_t epilogue) {
  Product x;
  x.M = M, x.N = N, x.K = K;
  x.A = A, x.lda = lda, x.SA = SA, x.a_type = a_type;
  x.B = B, x.ldb = ldb, x.SB = SB, x.b_type = b_type;
  x.D = const_cast<void*>(D), x.ldd = ldd, x.d_type = d_type;
  x.alpha = alpha, x.beta = beta, x.epi = epilogue;
  return check_product(x);
}

gemm_status_t gemm_run_scaled(gemm_plan_t plan, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                              const void* SA, gemm_type_t a_type, const void* B, int64_t ldb, const void* SB,
                              gemm_type_t b_type, void* D, int64_t ldd, gemm_type_t d_type, float alpha, float beta,
                              gemm_epilogue_t epilogue, void* stream) {
  Product x;
  x.M = M, x.N = N, x.K = K;
  x.A = A, x.lda = lda, x.SA = SA, x.a_type = a_type;
  x.B = B, x.ldb = ldb, x.SB = SB, x.b_type = b_type;
  x.D = D, x.ldd = ldd, x.d_type = d_type;
  x.alpha = alpha, x.beta = beta, x.epi = epilogue;
  return checked_run(plan, x, stream);
}

gemm_status_t gemm_run_grouped(gemm_plan_t plan, int64_t groups, int64_t rows, int64_t N, int64_t K,
                               const int32_t* starts, const int32_t* counts, const void* A, int64_t lda,
                               const void* SA, gemm_type_t a_type, const void* B, int64_t ldb, int64_t b_group,
                               const void* SB, gemm_type_t b_type, void* D, int64_t ldd, gemm_type_t d_type,
                               float alpha, float beta, gemm_epilogue_t epilogue, void* stream) {
  Product x;
  x.name = "gemm_run_grouped";
  x.group = SC_ROWS, x.groups = groups, x.M = rows, x.N = N, x.K = K;
  x.starts = starts, x.counts = counts;
  x.A = A, x.lda = lda, x.SA = SA, x.a_type = a_type;
  x.B = B, x.ldb = ldb, x.b_group = b_group, x.SB = SB, x.b_type = b_type;
  x.D = D, x.ldd = ldd, x.d_type = d_type;
  x.alpha = alpha, x.beta = beta, x.epi = epilogue;
  return checked_run(plan, x, stream);
}

gemm_status_t gemm_run_grouped_k(gemm_plan_t plan, int64_t groups, int64_t M, int64_t N, int64_t rows,
                                 const int32_t* starts, const int32_t* counts, const void* A, int64_t lda,
                                 const void* SA, gemm_type_t a_type, const void* B, int64_t ldb, const void* SB,
                                 gemm_type_t b_type, void* D, int64_t ldd, int64_t d_group, gemm_type_t d_type,
                                 float alpha, float beta, gemm_epilogue_t epilogue, void* stream) {
  Product x;
  x.name = "gemm_run_grouped_k";
  x.group = SC_K, x.groups = groups, x.M = M, x.N = N, x.K = rows;
  x.starts = starts, x.counts = counts;
  x.A = A, x.lda = lda, x.SA = SA, x.a_type = a_type;
  x.B = B, x.ldb = ldb, x.SB = SB, x.b_type = b_type;
  x.D = D, x.ldd = ldd, x.d_group = d_group, x.d_type = d_type;
  x.alpha = alpha, x.beta = beta, x.epi = epilogue;
  return checked_run(plan, x, stream);
}

int64_t gemm_mx_scale_bytes(int64_t rows, int64_t cols) {
  return size_ok(rows) && size_ok(cols) ? mx4_scale_tiles(rows, cols) * 512 : -1;
}

gemm_status_t gemm_check_mx(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* SA, const void* B,
                            int64_t ldb, const void* SB, const void* D, int64_t ldd, gemm_type_t d_type, float alpha,
                            float beta, gemm_epilogue_t epilogue) {
  Product x;
  x.four = true;
  x.M = M, x.N = N, x.K = K;
  x.A = A, x.lda = lda, x.SA = SA;
  x.B = B, x.ldb = ldb, x.SB = SB;
  x.D = const_cast<void*>(D), x.ldd = ldd, x.d_type = d_type;
  x.alpha = alpha, x.beta = beta, x.epi = epilogue;
  return check_product(x);
}

gemm_status_t gemm_run_mx(gemm_plan_t plan, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* SA,
                          const void* B, int64_t ldb, const void* SB, void* D, int64_t ldd, gemm_type_t d_type,
                          float alpha, float beta, gemm_epilogue_t epilogue, void* stream) {
  Product x;
  x.name = "gemm_run_mx";
  x.four = true;
  x.M = M, x.N = N, x.K = K;
  x.A = A, x.lda = lda, x.SA = SA;
  x.B = B, x.ldb = ldb, x.SB = SB;
  x.D = D, x.ldd = ldd, x.d_type = d_type;
  x.alpha = alpha, x.beta = beta, x.epi = epilogue;
  return checked_run(plan, x, stream);
}

gemm_status_t gemm_run_grouped_mx(gemm_plan_t plan, int64_t groups, int64_t rows, int64_t N, int64_t K,
                                  const int32_t* starts, const int32_t* counts, const void* A, int64_t lda,
                                  const void* SA, const void* B, int64_t ldb, int64_t b_group, const void* SB, void* D,
                                  int64_t ldd, gemm_type_t d_type, float alpha, float beta, gemm_epilogue_t epilogue,
                                  void* stream) {
  Product x;
  x.name = "gemm_run_grouped_mx";
  x.four = true;
  x.group = SC_ROWS, x.groups = groups, x.M = rows, x.N = N, x.K = K;
  x.starts = starts, x.counts = counts;
  x.A = A, x.lda = lda, x.SA = SA;
  x.B = B, x.ldb = ldb, x.b_group = b_group, x.SB = SB;
  x.D = D, x.ldd = ldd, x.d_type = d_type;
  x.alpha = alpha, x.beta = beta, x.epi = epilogue;
  return checked_run(plan, x, stream);
}

gemm_status_t gemm_quantize(gemm_plan_t plan, int64_t rows, int64_t cols, const void* X, int64_t ldx, gemm_type_t x_type,
                            const int32_t* rowmap, int64_t map_div, int64_t src_rows, gemm_type_t q_type,
                            int32_t block_rows, void* Q, int64_t ldq, void* SQ, void* QT, int64_t ldqt, void* SQT,
                            void* stream) {
  if (!plan || rows < 0 || cols < 0 || src_rows < 0 || !is_float_type(x_type) || !is_code_type(q_type))
    return GEMM_ERR_INVALID_ARG;
  if ((block_rows != 1 && block_rows != 128) || (rowmap && map_div < 1)) return GEMM_ERR_INVALID_ARG;
  // (the tile kernel's grid takes 65535 row blocks)
  if (!size_ok(rows) || !size_ok(cols) || !size_ok(src_rows) || rows > int64_t(65532) * 128 || map_div > kMaxDim)
    return GEMM_ERR_UNSUPPORTED;
  if ((Q == nullptr) != (SQ == nullptr) || (QT == nullptr) != (SQT == nullptr) || (!Q && !QT)) return GEMM_ERR_INVALID_ARG;
  const int64_t one = 1;
  if (ldx < std::max(one, cols) || (Q && ldq < std::max(one, cols)) || (QT && ldqt < std::max(one, rows)))
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM_OK;
  const int64_t xr = rowmap ? src_rows : rows, es = type_bytes(x_type);
  if (!X && xr > 0) return GEMM_ERR_INVALID_ARG;
  if (!aligned(X, size_t(es)) || !aligned(rowmap, 4) || !aligned(Q, 16) || !aligned(SQ, 16) || !aligned(QT, 16) ||
      !aligned(SQT, 16) || (Q && ldq % 16) || (QT && ldqt % 16))
    return GEMM_ERR_ALIGNMENT;
  // no result may share a byte with X, the map or another result
  if (results_meet({region(Q, Q ? rows : 0, cols, ldq, 1), run_of(SQ, gemm_scale_bytes(rows, cols)),
                    region(QT, QT ? cols : 0, rows, ldqt, 1), run_of(SQT, gemm_scale_bytes(cols, rows))},
                   {region(X, xr, cols, ldx, es), run_of(rowmap, rows * 4)}))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_quantize %lldx%lld %s->%s block %dx128%s%s%s", (long long)rows, (long long)cols,
                       type_name(x_type), type_name(q_type),
                       int(block_rows), Q ? " Q" : "", QT ? " QT" : "", rowmap ? " by map" : "");
  DeviceGuard guard(plan->device);
  QuantArgs a{};
  a.x = X;
  a.ldx = ldx;
  a.x_kind = type_kind(x_type);
  a.rows = int(rows);
  a.cols = int(cols);
  a.rows_padded = int(std::min<int64_t>(round_up(rows, 128), kMaxDim));
  a.cols_padded = int(std::min<int64_t>(round_up(cols, 128), kMaxDim));
  a.rowmap = rowmap;
  a.map_div = rowmap ? int(map_div) : 1;
  a.src_rows = int(xr);
  a.block_rows = block_rows;
  a.e5m2 = q_type == GEMM_TYPE_E5M2;
  a.vec = aligned(X, size_t(4 * es)) && ldx % 4 == 0;
  a.q = static_cast<uint8_t*>(Q);
  a.sq = static_cast<uint8_t*>(SQ);
  a.qt = static_cast<uint8_t*>(QT);
  a.sqt = static_cast<uint8_t*>(SQT);
  a.ldq = ldq;
  a.ldqt = ldqt;
  a.q_groups = Q ? int(scale_groups(cols)) : 0;
  a.qt_groups = QT ? int(scale_groups(rows)) : 0;
  a.pdl = plan->pdl;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(X, xr, cols, ldx, es).matrix(Q, Q ? rows : 0, cols, ldq, 1)
              .bytes(SQ, gemm_scale_bytes(rows, cols)).out_matrix(QT, QT ? cols : 0, rows, ldqt, 1)
              .bytes(SQT, gemm_scale_bytes(cols, rows)).bytes(rowmap, rowmap ? rows * 4 : 0).s;
#endif
  return call.done(launched(launch_quantize(a, static_cast<cudaStream_t>(stream))));
}

gemm_status_t gemm_quantize_mx(gemm_plan_t plan, int64_t rows, int64_t cols, const void* X, int64_t ldx,
                               gemm_type_t x_type, const int32_t* rowmap, int64_t map_div, int64_t src_rows, void* Q,
                               int64_t ldq, void* SQ, void* QT, int64_t ldqt, void* SQT, void* stream) {
  if (!plan || rows < 0 || cols < 0 || src_rows < 0 || !is_float_type(x_type)) return GEMM_ERR_INVALID_ARG;
  if (rowmap && map_div < 1) return GEMM_ERR_INVALID_ARG;
  // (indices behind the last tile have to fit 32 bits too)
  if (!size_ok(rows) || !size_ok(cols + 1024) || !size_ok(src_rows) || rows > int64_t(65532) * 128 || map_div > kMaxDim)
    return GEMM_ERR_UNSUPPORTED;
  if ((Q == nullptr) != (SQ == nullptr) || (QT == nullptr) != (SQT == nullptr) || (!Q && !QT)) return GEMM_ERR_INVALID_ARG;
  const int64_t one = 1, cb = ceil_div(cols, 2), rb = ceil_div(rows, 2);
  if (ldx < std::max(one, cols) || (Q && ldq < std::max(one, cb)) || (QT && ldqt < std::max(one, rb)))
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM_OK;
  const int64_t xr = rowmap ? src_rows : rows, es = type_bytes(x_type);
  if (!X && xr > 0) return GEMM_ERR_INVALID_ARG;
  if (!aligned(X, size_t(es)) || !aligned(rowmap, 4) || !aligned(SQ, 16) || !aligned(SQT, 16)) return GEMM_ERR_ALIGNMENT;
  const int64_t sq = mx4_scale_tiles(rows, cols) * 512, sqt = mx4_scale_tiles(cols, rows) * 512;
  // no result may share a byte with X, the map or another result
  if (results_meet({region(Q, Q ? rows : 0, cb, ldq, 1), run_of(SQ, sq), region(QT, QT ? cols : 0, rb, ldqt, 1), run_of(SQT, sqt)},
                   {region(X, xr, cols, ldx, es), run_of(rowmap, rows * 4)}))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_quantize_mx %lldx%lld %s->mx4%s%s%s", (long long)rows, (long long)cols, type_name(x_type),
                       Q ? " Q" : "", QT ? " QT" : "", rowmap ? " by map" : "");
  DeviceGuard guard(plan->device);
  QuantArgs a{};
  a.x = X;
  a.ldx = ldx;
  a.x_kind = type_kind(x_type);
  a.rows = int(rows);
  a.cols = int(cols);
  a.rows_padded = int(std::min<int64_t>(round_up(rows, 128), kMaxDim));
  a.rowmap = rowmap;
  a.map_div = rowmap ? int(map_div) : 1;
  a.src_rows = int(xr);
  a.vec = rows_wide(X, ldx, es);
  a.q = static_cast<uint8_t*>(Q);
  a.sq = static_cast<uint8_t*>(SQ);
  a.qt = static_cast<uint8_t*>(QT);
  a.sqt = static_cast<uint8_t*>(SQT);
  a.ldq = ldq;
  a.ldqt = ldqt;
  a.x_words = aligned(X, 4) && (ldx * es) % 4 == 0;
  a.q_wide = aligned(Q, 4) && ldq % 4 == 0;
  a.qt_wide = rows_wide(QT, ldqt, 1);
  a.q_groups = int(mx4_scale_tiles(1, cols));
  a.qt_groups = int(mx4_scale_tiles(1, rows));
  a.pdl = plan->pdl;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(X, xr, cols, ldx, es).out_matrix(Q, Q && !QT ? rows : 0, cb, ldq, 1).matrix(Q, Q && QT ? rows : 0, cb, ldq, 1)
              .bytes(SQ, SQ ? sq : 0).out_matrix(QT, QT ? cols : 0, rb, ldqt, 1).bytes(SQT, SQT ? sqt : 0)
              .bytes(rowmap, rowmap ? rows * 4 : 0).s;
#endif
  return call.done(launched(launch_quantize_mx4(a, plan->sms, static_cast<cudaStream_t>(stream))));
}

gemm_status_t gemm_dequantize(gemm_plan_t plan, int64_t rows, int64_t cols, const void* Q, int64_t ldq, gemm_type_t q_type,
                              const void* SQ, void* X, int64_t ldx, gemm_type_t x_type, void* stream) {
  const bool four = q_type == GEMM_TYPE_E2M1;
  if (!plan || rows < 0 || cols < 0 || !is_float_type(x_type) || (!four && !is_code_type(q_type))) return GEMM_ERR_INVALID_ARG;
  if (!size_ok(rows + 1024) || !size_ok(cols + 1024) || rows * ceil_div(cols, 512) > kMaxDim * 16)  // (its grid)
    return GEMM_ERR_UNSUPPORTED;
  const int64_t one = 1, cb = four ? ceil_div(cols, 2) : cols;
  if (ldq < std::max(one, cb) || ldx < std::max(one, cols)) return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (!Q || !SQ || !X) return GEMM_ERR_INVALID_ARG;
  const int64_t es = type_bytes(x_type), sq = (four ? mx4_scale_tiles(rows, cols) : scale_tiles(rows, cols)) * 512;
  if (!aligned(SQ, 16) || !aligned(X, size_t(es))) return GEMM_ERR_ALIGNMENT;
  if (results_meet({region(X, rows, cols, ldx, es)}, {region(Q, rows, cb, ldq, 1), run_of(SQ, sq)})) return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_dequantize %lldx%lld %s->%s", (long long)rows, (long long)cols, four ? "mx4" : type_name(q_type),
                       type_name(x_type));
  DeviceGuard guard(plan->device);
  DequantArgs a{};
  a.q = static_cast<const uint8_t*>(Q);
  a.ldq = ldq;
  a.sq = static_cast<const uint8_t*>(SQ);
  a.q_wide = aligned(Q, four ? 4 : 8) && ldq % (four ? 4 : 8) == 0;
  a.code = four ? CODE_E2M1 : q_type == GEMM_TYPE_E5M2 ? CODE_E5M2 : CODE_E4M3;
  a.rows = int(rows);
  a.cols = int(cols);
  a.groups = int(four ? mx4_scale_tiles(1, cols) : scale_groups(cols));
  a.x = X;
  a.ldx = ldx;
  a.x_kind = type_kind(x_type);
  a.wide = rows_wide(X, ldx, es);
  a.pdl = plan->pdl;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(Q, rows, cb, ldq, 1).bytes(SQ, sq).out_matrix(X, rows, cols, ldx, es).s;
#endif
  return call.done(launched(launch_dequantize(a, static_cast<cudaStream_t>(stream))));
}

gemm_status_t gemm_route(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ldl,
                         gemm_type_t l_type, const float* bias, gemm_route_t route, float* weights, int32_t* indices,
                         void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t st = check_route(tokens, experts, logits, ldl, l_type, route);
  if (st != GEMM_OK || tokens == 0) return st;
  if (!weights || !indices) return GEMM_ERR_INVALID_ARG;
  if (!aligned(weights, 4) || !aligned(indices, 4) || !aligned(bias, 4)) return GEMM_ERR_ALIGNMENT;
  const int64_t slots = tokens * route.top_k;
  if (results_meet({run_of(weights, slots * 4), run_of(indices, slots * 4)},
                   {region(logits, tokens, experts, ldl, type_bytes(l_type)), run_of(bias, experts * 4)}))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_route %lldx%lld %s %s top %d groups %d of %d%s%s", (long long)tokens,
                       (long long)experts, type_name(l_type),
                       route.score == GEMM_SCORE_SIGMOID ? "sigmoid" : "softmax", int(route.top_k), int(route.top_groups),
                       int(route.groups), bias ? " bias" : "", route.renormalize ? " renormalized" : "");
  DeviceGuard guard(plan->device);
  RouteArgs a = route_args(plan, tokens, experts, logits, ldl, l_type, route);
  a.bias = bias;
  a.weights = weights;
  a.indices = indices;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(logits, tokens, experts, ldl, type_bytes(l_type)).bytes(bias, bias ? experts * 4 : 0)
              .bytes(weights, tokens * route.top_k * 4).out_matrix(indices, 1, tokens * route.top_k, 0, 4).s;
#endif
  return call.done(launched(launch_route(a, static_cast<cudaStream_t>(stream))));
}

gemm_status_t gemm_route_backward(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ldl,
                                  gemm_type_t l_type, gemm_route_t route, const int32_t* indices, const float* dweights,
                                  void* dlogits, int64_t lddl, void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t st = check_route(tokens, experts, logits, ldl, l_type, route);
  if (st != GEMM_OK) return st;
  if (lddl < experts) return GEMM_ERR_INVALID_ARG;
  if (tokens == 0) return GEMM_OK;
  if (!indices || !dweights || !dlogits) return GEMM_ERR_INVALID_ARG;
  if (!aligned(dweights, 4) || !aligned(indices, 4) || !aligned(dlogits, size_t(type_bytes(l_type))))
    return GEMM_ERR_ALIGNMENT;
  // (a token's logits are read before its gradients are written: these may be the logits' own place)
  const int64_t es = type_bytes(l_type), slots = tokens * route.top_k;
  const bool in_place = dlogits == logits && lddl == ldl;
  if (results_meet({region(dlogits, tokens, experts, lddl, es)},
                   {region(logits, in_place ? 0 : tokens, experts, ldl, es), run_of(indices, slots * 4), run_of(dweights, slots * 4)}))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_route_backward %lldx%lld %s %s top %d%s", (long long)tokens, (long long)experts,
                       type_name(l_type),
                       route.score == GEMM_SCORE_SIGMOID ? "sigmoid" : "softmax", int(route.top_k),
                       route.renormalize ? " renormalized" : "");
  DeviceGuard guard(plan->device);
  RouteArgs a = route_args(plan, tokens, experts, logits, ldl, l_type, route);
  a.indices = const_cast<int32_t*>(indices);
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.lddl = lddl;
  a.wide_out = rows_wide(dlogits, lddl, type_bytes(l_type));
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(logits, tokens, experts, ldl, type_bytes(l_type)).bytes(indices, tokens * route.top_k * 4)
              .bytes(dweights, tokens * route.top_k * 4).out_matrix(dlogits, tokens, experts, lddl, type_bytes(l_type)).s;
#endif
  return call.done(launched(launch_route_backward(a, static_cast<cudaStream_t>(stream))));
}

gemm_status_t gemm_balance(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ldl,
                           gemm_type_t l_type, gemm_score_t score, int32_t top_k, const int32_t* indices, float scale,
                           int32_t* counts, float* shares, float* factor, float* loss, void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t st = check_balance(tokens, experts, logits, ldl, l_type, score, top_k, indices);
  if (st != GEMM_OK) return st;
  if (!counts || !shares || !factor || !loss) return GEMM_ERR_INVALID_ARG;
  if (!aligned(counts, 4) || !aligned(shares, 4) || !aligned(factor, 4) || !aligned(loss, 4)) return GEMM_ERR_ALIGNMENT;
  const int64_t es = type_bytes(l_type);
  if (results_meet({run_of(counts, experts * 4), run_of(shares, experts * 4), run_of(factor, experts * 4), run_of(loss, 4)},
                   {region(logits, tokens, experts, ldl, es), run_of(indices, tokens * top_k * 4)}))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_balance %lldx%lld %s %s top %d", (long long)tokens, (long long)experts, type_name(l_type),
                       score == GEMM_SCORE_SIGMOID ? "sigmoid" : "softmax", int(top_k));
  DeviceGuard guard(plan->device);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int ctas = balance_ctas(tokens, experts, plan->sms);
  const size_t ws = ctas > 1 ? size_t(ctas) * size_t(experts) * 4 : 0;
  if (ctas > 1) {
    gemm_status_t grown = ensure_ws(plan, ws, s);
    if (grown == GEMM_OK) grown = ensure_counters(plan, size_t(experts) + 2, s);
    if (grown != GEMM_OK) return grown;
  }
  BalanceArgs a = balance_args(plan, tokens, experts, logits, ldl, l_type, score, top_k, indices);
  a.scale = scale;
  a.counts = counts;
  a.shares = shares;
  a.factor = factor;
  a.loss = loss;
  a.parts = static_cast<float*>(plan->ws);
  a.counters = plan->counters;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(logits, tokens, experts, ldl, es).bytes(indices, tokens * top_k * 4).bytes(counts, experts * 4)
              .bytes(shares, experts * 4).out_matrix(factor, 1, experts, 0, 4).bytes(loss, 4).bytes(plan->ws, int64_t(ws))
              .bytes(plan->counters, ctas > 1 ? (experts + 2) * 4 : 0).s;
#endif
  return call.done(launched(launch_balance(a, ctas, s)));
}

gemm_status_t gemm_balance_backward(gemm_plan_t plan, int64_t tokens, int64_t experts, const void* logits, int64_t ldl,
                                    gemm_type_t l_type, gemm_score_t score, int32_t top_k, const int32_t* indices,
                                    const float* factor, const float* dloss, int32_t accumulate, void* dlogits, int64_t lddl,
                                    void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t st = check_balance(tokens, experts, logits, ldl, l_type, score, top_k, indices);
  if (st != GEMM_OK) return st;
  if (lddl < experts) return GEMM_ERR_INVALID_ARG;
  if (tokens == 0) return GEMM_OK;
  if (!factor || !dlogits) return GEMM_ERR_INVALID_ARG;
  const int64_t es = type_bytes(l_type);
  if (!aligned(factor, 4) || !aligned(dloss, 4) || !aligned(dlogits, size_t(es))) return GEMM_ERR_ALIGNMENT;
  // (a token's logits are read before its gradients are written: these may be the logits' own place)
  const bool in_place = dlogits == logits && lddl == ldl && !accumulate;
  if (results_meet({region(dlogits, tokens, experts, lddl, es)},
                   {region(logits, in_place ? 0 : tokens, experts, ldl, es), run_of(indices, tokens * top_k * 4),
                    run_of(factor, experts * 4), run_of(dloss, 4)}))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_balance_backward %lldx%lld %s %s top %d%s", (long long)tokens, (long long)experts,
                       type_name(l_type), score == GEMM_SCORE_SIGMOID ? "sigmoid" : "softmax", int(top_k),
                       accumulate ? " accumulated" : "");
  DeviceGuard guard(plan->device);
  BalanceArgs a = balance_args(plan, tokens, experts, logits, ldl, l_type, score, top_k, indices);
  a.factor = const_cast<float*>(factor);
  a.dloss = dloss;
  a.accumulate = accumulate != 0;
  a.dlogits = dlogits;
  a.lddl = lddl;
  a.wide_out = rows_wide(dlogits, lddl, es);
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(logits, tokens, experts, ldl, es).bytes(indices, tokens * top_k * 4).bytes(factor, experts * 4)
              .bytes(dloss, dloss ? 4 : 0).out_matrix(dlogits, tokens, experts, lddl, es).s;
#endif
  return call.done(launched(launch_balance_backward(a, static_cast<cudaStream_t>(stream))));
}

int64_t gemm_route_rows(int64_t tokens, int64_t top_k, int64_t experts) {
  if (!size_ok(tokens) || top_k < 1 || experts < 1 || top_k > kMaxDim || experts > kMaxDim || tokens * top_k > kMaxDim)
    return -1;
  const int64_t slots = tokens * top_k, rows = round_up(slots + 127 * std::min(experts, slots), 128);
  return rows <= kMaxDim ? rows : -1;
}

gemm_status_t gemm_route_map(gemm_plan_t plan, int64_t tokens, int64_t top_k, int64_t experts, const int32_t* indices,
                             int32_t* starts, int32_t* counts, int32_t* pos, int32_t* rowmap, int64_t rows, void* stream) {
  if (!plan || tokens < 0 || top_k < 1 || experts < 1) return GEMM_ERR_INVALID_ARG;
  if (experts > ROUTE_MAX_EXPERTS || !size_ok(rows)) return GEMM_ERR_UNSUPPORTED;
  const int64_t need = gemm_route_rows(tokens, top_k, experts);
  if (need < 0) return GEMM_ERR_UNSUPPORTED;
  if (rows < need || !starts || !counts) return GEMM_ERR_INVALID_ARG;
  if ((tokens > 0 && (!indices || !pos)) || (rows > 0 && !rowmap)) return GEMM_ERR_INVALID_ARG;
  if (!aligned(indices, 4) || !aligned(starts, 4) || !aligned(counts, 4) || !aligned(pos, 4) || !aligned(rowmap, 4))
    return GEMM_ERR_ALIGNMENT;
  const int64_t slots = tokens * top_k;
  if (results_meet({run_of(starts, experts * 4), run_of(counts, experts * 4), run_of(pos, slots * 4), run_of(rowmap, rows * 4)},
                   {run_of(indices, slots * 4)}))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_route_map %lldx%lld experts %lld rows %lld", (long long)tokens, (long long)top_k,
                       (long long)experts, (long long)rows);
  DeviceGuard guard(plan->device);
  const size_t ws = route_map_workspace(slots, experts);
  if (ws > 0) {
    const gemm_status_t st = ensure_ws(plan, ws, static_cast<cudaStream_t>(stream));
    if (st != GEMM_OK) return st;
  }
  RouteMapArgs a{};
  a.indices = indices;
  a.slots = int(slots);
  a.experts = int(experts);
  a.starts = starts;
  a.counts = counts;
  a.pos = pos;
  a.rowmap = rowmap;
  a.rows = int(rows);
  a.wide = aligned(rowmap, 16);
  a.block_counts = static_cast<int*>(plan->ws);
  a.pdl = plan->pdl;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).bytes(indices, tokens * top_k * 4).bytes(starts, experts * 4).bytes(counts, experts * 4)
              .bytes(pos, tokens * top_k * 4).bytes(plan->ws, int64_t(ws)).out_matrix(rowmap, 1, rows, 0, 4).s;
#endif
  return call.done(launched(launch_route_map(a, static_cast<cudaStream_t>(stream))));
}

gemm_status_t gemm_combine(gemm_plan_t plan, int64_t tokens, int64_t top_k, int64_t cols, int64_t rows, const void* Y,
                           int64_t ldy, gemm_type_t y_type, const int32_t* pos, const float* weights, void* out,
                           int64_t ldo, gemm_type_t out_type, void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t st = check_combine(tokens, top_k, cols, rows, Y, ldy, y_type, pos, weights, out, ldo, out_type);
  if (st != GEMM_OK || tokens == 0 || cols == 0) return st;
  const int64_t ye = type_bytes(y_type), oe = type_bytes(out_type);
  const int64_t slots = tokens * top_k;
  if (results_meet({region(out, tokens, cols, ldo, oe)},
                   {region(Y, rows, cols, ldy, ye), run_of(pos, slots * 4), run_of(weights, slots * 4)}))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_combine %lldx%lldx%lld rows %lld %s->%s", (long long)tokens, (long long)top_k,
                       (long long)cols, (long long)rows,
                       type_name(y_type), type_name(out_type));
  DeviceGuard guard(plan->device);
  CombineArgs a{};
  a.tokens = int(tokens);
  a.k = int(top_k);
  a.cols = int(cols);
  a.rows = int(rows);
  a.y = Y;
  a.ldy = ldy;
  a.y_kind = type_kind(y_type);
  a.pos = pos;
  a.weights = weights;
  a.out = out;
  a.ldo = ldo;
  a.o_kind = type_kind(out_type);
  a.wide = access_bytes(cols, {{Y, ldy * ye}, {out, ldo * oe}});
  a.pdl = plan->pdl;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(Y, rows, cols, ldy, ye).bytes(pos, tokens * top_k * 4).bytes(weights, tokens * top_k * 4)
              .out_matrix(out, tokens, cols, ldo, oe).s;
#endif
  return call.done(launched(launch_combine(a, static_cast<cudaStream_t>(stream))));
}

gemm_status_t gemm_combine_backward(gemm_plan_t plan, int64_t tokens, int64_t top_k, int64_t cols, int64_t rows,
                                    const void* dout, int64_t ldo, gemm_type_t out_type, const void* Y, int64_t ldy,
                                    gemm_type_t y_type, const int32_t* pos, const float* weights, const int32_t* rowmap,
                                    void* dY, int64_t lddy, float* dweights, void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t st = check_combine(tokens, top_k, cols, rows, Y, ldy, y_type, pos, weights, dout, ldo, out_type);
  if (st != GEMM_OK) return st;
  if (lddy < std::max<int64_t>(1, cols)) return GEMM_ERR_INVALID_ARG;
  if (tokens == 0 && (rows == 0 || !rowmap)) return GEMM_OK;
  if ((tokens > 0 && !dweights) || (rows > 0 && cols > 0 && !dY)) return GEMM_ERR_INVALID_ARG;
  if (cols == 0 && (!pos || !weights)) return GEMM_ERR_INVALID_ARG;
  const int64_t ye = type_bytes(y_type), oe = type_bytes(out_type);
  if (!aligned(dY, size_t(ye)) || !aligned(dweights, 4) || !aligned(rowmap, 4)) return GEMM_ERR_ALIGNMENT;
  // (a token's weights are read before their gradients are written: these may be the weights' own place)
  const int64_t slots = tokens * top_k;
  if (results_meet({region(dY, rows, cols, lddy, ye), run_of(dweights, slots * 4)},
                   {region(Y, rows, cols, ldy, ye), region(dout, tokens, cols, ldo, oe), run_of(pos, slots * 4),
                    run_of(rowmap, rows * 4)}) ||
      overlaps(region(dY, rows, cols, lddy, ye), run_of(weights, slots * 4)) ||
      (dweights != weights && overlaps(run_of(dweights, slots * 4), run_of(weights, slots * 4))))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_combine_backward %lldx%lldx%lld rows %lld %s->%s%s", (long long)tokens,
                       (long long)top_k, (long long)cols,
                       (long long)rows, type_name(out_type), type_name(y_type), rowmap ? " by map" : "");
  DeviceGuard guard(plan->device);
  CombineArgs a{};
  a.tokens = int(tokens);
  a.k = int(top_k);
  a.cols = int(cols);
  a.rows = int(rows);
  a.y = Y;
  a.ldy = ldy;
  a.y_kind = type_kind(y_type);
  a.pos = pos;
  a.weights = weights;
  a.out = const_cast<void*>(dout);
  a.ldo = ldo;
  a.o_kind = type_kind(out_type);
  a.rowmap = rowmap;
  a.dy = dY;
  a.lddy = lddy;
  a.dweights = dweights;
  a.wide = access_bytes(cols, {{Y, ldy * ye}, {dout, ldo * oe}, {dY, lddy * ye}});
  a.pdl = plan->pdl;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(dout, tokens, cols, ldo, oe).matrix(Y, rows, cols, ldy, ye).bytes(pos, tokens * top_k * 4)
              .bytes(weights, tokens * top_k * 4).bytes(rowmap, rowmap ? rows * 4 : 0).bytes(dweights, tokens * top_k * 4)
              .out_matrix(dY, rows, cols, lddy, ye).s;
#endif
  return call.done(launched(launch_combine_backward(a, static_cast<cudaStream_t>(stream))));
}

}  // extern "C"
