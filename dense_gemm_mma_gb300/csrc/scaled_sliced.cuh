// scaled_sliced.cuh -- block-scaled products with few rows of A, or few tiles:
// single tokens and small batches against a weight matrix, and experts that a few
// rows each go to (formula and scales: scaled.cuh), compiled for 8-bit operands in scaled_sliced.cu and for
// 4-bit ones in mx4_sliced.cu (FOUR: a stage holds 256 values of K, and scale tiles of its own).
//
// What bounds these calls is reading B once.  So B's rows take the 128 lanes of the
// MMA and A's rows its N dimension, as many columns (32 to 128) as the tile has rows of A: no lane
// is spent on rows that do not exist, a ring stage is 16 KB of B and 4 to 16 KB of A, and the ring
// holds enough of B in flight to cover the memory latency.  A tile starts a scale
// tile (a multiple of 128 rows of A): the MMA takes its scales from a multiple of four
// tensor-memory columns, and row 32 i of a scale tile is in column i.  Where there are fewer
// tiles than SMs, the CTAs of a cluster take slices of K: each leaves its fp32 partial
// tile in its own shared memory, and each then sums every slices-th row of the tile over
// all CTAs through distributed shared memory, in slice order, so the result has
// the same bits every time and no workspace or second launch is needed.
//
//  - warp 0: TMA producer; warp 1: MMA issuer (two accumulators,
//    so a tile's MMAs overlap the previous one's epilogue);
//  - warps 2-5: accumulator lanes -> partial tile [rows of A][128 rows of B] in shared
//    memory, then whole rows of it, 512 bytes a warp, to D.  All rows of a tile in one exchange: it
//    takes ~1.5 us whatever its size.  Where a CTA has K to itself nothing is exchanged: each warp turns
//    its 32 columns of D round in 4 KB of its own, 32 rows at a time, and the ring has the room.
//
// Measured: one row, 4096 x 4096: 6.4 us (the 17 MB come from L2 in repeated calls); 48 tokens to 4 of 64
// experts of 2048 x 2048: 34.7 us, 7.2 TB/s of the weights of ~60 experts.  4 bits: 5.7 and 28.3 us (4.9 TB/s with the scales, and the
// launch, ~5 us, in it).
#pragma once

#include <type_traits>

#include "scaled.cuh"

namespace dg {
namespace {

constexpr int kThreads = 192;
constexpr int kEpiWarps = 4;
constexpr int kMaxStages = 8;
constexpr int kMaxSlices = 8;
constexpr int kWeights = 128 * SC_BK;  // bytes of B per stage
constexpr int kRowsA = 32 * SC_BK;     // bytes of a load of A: 32 rows

// scale tiles of B's 128 rows and of the block of A's rows
__host__ __device__ constexpr int scale_bytes(bool four) { return four ? 2048 : 1024; }
__host__ __device__ constexpr int stage_bytes(int bn) { return kWeights + bn * SC_BK; }
// ring (every operand tile is 1024-byte aligned), scales, partial tile, barriers, table
__host__ __device__ constexpr int off_scales(int bn, int stages) { return stages * stage_bytes(bn); }
template <bool FOUR>
__host__ __device__ constexpr int off_part(int bn, int stages) { return off_scales(bn, stages) + stages * scale_bytes(FOUR); }
template <bool FOUR>
__host__ __device__ constexpr int off_bar(int bn, int stages, int part) { return off_part<FOUR>(bn, stages) + part * 128 * 4; }
constexpr int kBarBytes = (2 * kMaxStages + 2 + 2 + 1 + 2) * 8;  // full, empty, tmem_full, tmem_empty, drain, part_full, part_free
template <bool FOUR>
__host__ __device__ constexpr int off_misc(int bn, int stages, int part) { return off_bar<FOUR>(bn, stages, part) + kBarBytes; }
template <bool FOUR>
__host__ __device__ constexpr int off_table(int bn, int stages, int part) { return off_misc<FOUR>(bn, stages, part) + 16; }

// Tensor-memory columns: two accumulators of bn, then four sets of 8 or 16 scale columns
// (B's rows, A's rows).
template <bool FOUR>
__host__ __device__ constexpr uint32_t tmem_cols(int bn) {
  constexpr int scales = FOUR ? 64 : 32;
  return 2 * bn + scales <= 128 ? 128u : 2 * bn + scales <= 256 ? 256u : 512u;
}

// ALL: GELU and SiLU as well.  A kernel of their own: inlined into every variant of the rows'
// loop they fill the instruction cache, and as a call they slowed the other warps' loops (one row,
// 8192 x 8192: 11.6 us, 14.7 with the call).
template <bool ALL, bool FOUR>
__global__ void __launch_bounds__(kThreads)
    scaled_sliced_kernel(const __grid_constant__ ScMaps maps, const __grid_constant__ ScParams p) {
  const int bn = p.bn, S = p.stages, slices = p.slices;
  const uint32_t rank = slices > 1 ? cluster_ctarank() : 0u;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const sbase = smem_raw + (base - raw);
  const int warp = sc_warp();
  const int lane = threadIdx.x & 31;
  const uint32_t full0 = base + off_bar<FOUR>(bn, S, p.part_rows), empty0 = full0 + 8 * kMaxStages;
  const uint32_t tfull0 = empty0 + 8 * kMaxStages, tempty0 = tfull0 + 16, drain_bar = tempty0 + 16;
  const uint32_t part_full = drain_bar + 8, part_free = part_full + 8;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sbase + off_misc<FOUR>(bn, S, p.part_rows));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sbase + off_misc<FOUR>(bn, S, p.part_rows) + 4);
  int* const table = reinterpret_cast<int*>(sbase + off_table<FOUR>(bn, S, p.part_rows));
  const uint32_t cols = tmem_cols<FOUR>(bn);
  constexpr int kScales = scale_bytes(FOUR);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    mbar_init(part_full, kEpiWarps * slices);  // every epilogue warp of the cluster has written its partials
    mbar_init(part_free, kEpiWarps * slices);  // ... has read what it sums of this CTA's
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    prefetch_tmap(&maps.sa);
    prefetch_tmap(&maps.sb);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), cols);
    tmem_relinquish();
  }
  wait_prior_grid();
  if (threadIdx.x == 0) allow_next_grid();
  if (warp == 2 && p.group == SC_ROWS) sc_tile_table(p, bn, nullptr, table);
  tc_fence_before();
  if (slices > 1)
    cluster_sync();  // every CTA's barriers exist before another arrives on them
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = p.group == SC_ROWS ? table[p.groups] : p.units;
  const int unit0 = int(blockIdx.x) / slices;
  const int step = int(gridDim.x) / slices;
  const Watch w{abort_flag, p.err, p.timeout_ns};
  auto unit_of = [&](int u, int* cursor) {
    ScUnit x = sc_unit(p, u, bn, 128, nullptr, table, cursor);
    x.kb0 = int(rank) * p.kb_per_slice;
    x.kb1 = min(p.k_blocks, x.kb0 + p.kb_per_slice);
    return x;
  };
  // 32-row pieces of A in a tile
  auto pieces_of = [&](const ScUnit& x) { return (min(bn, x.row_end - x.row0) + 31) / 32; };

  const uint32_t one = lane == 0;  // the lane that issues

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int stage = 0, issued = 0, cursor = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = unit0; u < units && ok; u += step) {
      const ScUnit x = unit_of(u, &cursor);
      const int pieces = pieces_of(x);
      const int sb_row = x.zb * p.sb_group + (x.n0 / 128) * (FOUR ? 1 : p.sb_cols), sa_row = (x.row0 / 128) * (FOUR ? 1 : p.sa_cols);
      for (int kb = x.kb0; kb < x.kb1; ++kb) {
        const uint32_t eb = empty0 + 8 * stage, fb = full0 + 8 * stage;
        if (!sc_wait<SC_OWN>(eb, phase ^ 1u, w, WAIT_PRODUCER_EMPTY)) {
          ok = false;
          break;
        }
        const bool scales = FOUR || kb == x.kb0 || (kb & 3) == 0;
        mbar_expect_one(fb, uint32_t(kWeights + pieces * kRowsA + (scales ? kScales : 0)), one);
        auto load = [&](uint32_t dst, const CUtensorMap* m, int cx, int cy, int cz, int esize) {
          if (DG_TMA(p.dbg, cx, cy, esize, false)) tma_load_one<false>(dst, m, fb, cx, cy, cz, one);
        };
        const uint32_t st = base + uint32_t(stage * stage_bytes(bn));
        load(st, &maps.b, kb * SC_BK, x.n0, x.zb, 1);
        for (int j = 0; j < pieces; ++j) load(st + kWeights + j * kRowsA, &maps.a, kb * SC_BK, x.row0 + 32 * j, 0, 1);
        if (scales) {
          const uint32_t sf = base + uint32_t(off_scales(bn, S) + stage * kScales);
          if constexpr (FOUR) {  // (two tiles each: past K the box reads zero)
            load(sf, &maps.sb, 0, 2 * kb, sb_row, 4);
            load(sf + 1024, &maps.sa, 0, 2 * kb, sa_row, 4);
          } else {
            load(sf, &maps.sb, 0, sb_row + kb / 4, 0, 4);
            load(sf + 512, &maps.sa, 0, sa_row + kb / 4, 0, 4);
          }
        }
        ++issued;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      // Let the loads already in flight land before the CTA can exit.
      for (int s = 0; s < S; ++s) {
        const int n_s = issued > s ? (issued - s + S - 1) / S : 0;
        if (n_s > 0) sc_wait<SC_OWN>(full0 + 8 * s, (uint32_t)((n_s - 1) & 1), w, 0);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    int stage = 0, it = 0, cursor = 0, tiles = 0;
    uint32_t phase = 0;
    uint32_t set_col = 0;
    ScSets sets;
    bool ok = true;
    for (int u = unit0; u < units && ok; u += step) {
      const ScUnit x = unit_of(u, &cursor);
      if (x.kb0 >= x.kb1) continue;  // no K at all
      const int acc = tiles & 1;
      if (tiles > 1 && !sc_wait<SC_OWN>(tempty0 + 8 * acc, ((tiles - 2) >> 1) & 1, w, WAIT_MMA_TMEM_EMPTY)) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + uint32_t(acc * bn);
      const uint32_t mma_n = uint32_t(pieces_of(x)) * 32;
      for (int kb = x.kb0; kb < x.kb1; ++kb) {
        if (!sc_wait<SC_OWN>(full0 + 8 * stage, phase, w, WAIT_MMA_FULL)) {
          ok = false;
          break;
        }
        if constexpr (FOUR) {
          // The MMAs that read this set last, four k-blocks ago, have completed (S stages ago or more: full barrier `it` says so).
          const int old = it - 4;
          if (old >= 0 && S > 4 && !sc_wait<SC_OWN>(empty0 + 8 * (old % S), uint32_t(old / S) & 1u, w, WAIT_MMA_FULL)) {
            ok = false;
            break;
          }
          set_col = tmem_base + uint32_t(2 * bn) + 16 * uint32_t(it & 3);
          const uint32_t sf = desc_lo(base + uint32_t(off_scales(bn, S) + stage * kScales));
#pragma unroll
          for (int t = 0; t < 4; ++t) tc_copy_scales<false>(set_col + 4 * t, sf + (512 >> 4) * t, one);
        } else if (kb == x.kb0 || (kb & 3) == 0) {
          const int old = sets.last_user();
          if (old >= 0 && old > it - S &&
              !sc_wait<SC_OWN>(empty0 + 8 * (old % S), uint32_t(old / S) & 1u, w, WAIT_MMA_FULL)) {
            ok = false;
            break;
          }
          set_col = tmem_base + uint32_t(2 * bn) + 8 * sets.take(it);
          const uint32_t sf = desc_lo(base + uint32_t(off_scales(bn, S) + stage * kScales));
          tc_copy_scales<false>(set_col, sf, one);
          tc_copy_scales<false>(set_col + 4, sf + (512 >> 4), one);
        }
        const uint32_t lo = desc_lo(base + uint32_t(stage * stage_bytes(bn)));
        if constexpr (FOUR) {
          const uint32_t idesc = p.idesc | (mma_n >> 3 << 17);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_mx4<false>(d_tmem, lo + (32 >> 4) * kk, lo + (kWeights >> 4) + (32 >> 4) * kk, idesc | mx4_ids(kk),
                              set_col + 4 * (kk / 2), set_col + 8 + 4 * (kk / 2), kb > x.kb0 || kk > 0, one);
        } else {
          const uint32_t id = uint32_t(kb & 3);
          const uint32_t idesc = p.idesc | (mma_n >> 3 << 17) | (id << 4) | (id << 29);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_scaled<false>(d_tmem, lo + (32 >> 4) * kk, lo + (kWeights >> 4) + (32 >> 4) * kk, idesc, set_col,
                                 set_col + 4, kb > x.kb0 || kk > 0, one);
        }
        tc_commit_one<false>(empty0 + 8 * stage, one);  // stage free once these MMAs finish
        ++it;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      tc_commit_one<false>(tfull0 + 8 * acc, one);
      ++tiles;
    }
    // Every MMA issued by this warp completes before tensor memory is freed.
    tc_commit_one<false>(drain_bar, one);
    sc_wait<SC_OWN>(drain_bar, 0, w, WAIT_DRAIN);
  } else {
    // ------------------------------------------------------------ epilogue
    const int e = warp - 2;
    const int q = warp & 3;  // tensor-memory lane quarter this warp may read
    const int es = p.out_kind == OUT_F32 ? 4 : 2;
    float* const part = reinterpret_cast<float*>(sbase + off_part<FOUR>(bn, S));
    const uint32_t part_addr = base + uint32_t(off_part<FOUR>(bn, S));
    // four columns of a row go out as one store where rows allow it
    const bool wide = p.ldd % 4 == 0 && (reinterpret_cast<uintptr_t>(p.d) & uintptr_t(4 * es - 1)) == 0;
    int cursor = 0, tiles = 0, done = 0;
    // One arrival per warp on a barrier of every CTA of the cluster.
    auto arrive_all = [&](uint32_t bar) {
      __syncwarp();
      if (lane < slices) mbar_arrive_cluster(mapa_shared(bar, uint32_t(lane)));
      __syncwarp();
    };
    for (int u = unit0; u < units; u += step) {
      const ScUnit x = unit_of(u, &cursor);
      const bool empty = x.kb0 >= x.kb1;
      const int acc = tiles & 1;
      if (!empty) {
        if (!sc_wait<SC_OWN>(tfull0 + 8 * acc, (tiles >> 1) & 1, w, WAIT_EPI_TMEM_FULL)) break;
        tc_fence_after();
        ++tiles;
      }
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(acc * bn);
      const int pieces = pieces_of(x);
      // v[0 .. n) of row `row`, columns from `col` on, to D
      auto store = [&](float (&v)[4], int row, int col) {
        const int n = min(4, p.N - col);
        if (n <= 0) return;
        uint8_t* const dst = static_cast<uint8_t*>(p.d) + (int64_t(row) * p.ldd + col) * es;
        if (!DG_IN(p.dbg, dst, n * es, DBG_SCALED)) return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] *= p.alpha;
          if (p.beta != 0.f && j < n) v[j] = fmaf(p.beta, sc_load1(dst + j * es, p.out_kind), v[j]);
        }
        sc_act<ALL ? ACT_ALL : ACT_SIMPLE>(v, p.act, p.slope);
        if (wide && n == 4 && es == 4)
          *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        else if (wide && n == 4)
          *reinterpret_cast<uint2*>(dst) = make_uint2(sc_pack2(v[0], v[1], p.out_kind), sc_pack2(v[2], v[3], p.out_kind));
        else
          for (int j = 0; j < n; ++j) sc_store1(dst + j * es, v[j], p.out_kind);
      };
      // 32 rows of A of this warp's lanes, as a column of [row][stride] floats
      auto drain = [&](int c, float* at, int stride) {
        uint32_t r[32];
        if (!empty) {
          tmem_ld_32x32b_x32(t_row + 32 * c, r);
          tmem_ld_wait(r);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) at[j * stride] = __uint_as_float(r[j]);
      };
      auto release = [&]() {
        if (empty) return;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty0 + 8 * acc);
      };
      if (slices == 1) {
        float* const own = part + e * 32 * 32;
        for (int c = 0; c < pieces; ++c) {
          __syncwarp();  // the rows before these have been read
          drain(c, own + lane, 32);
          __syncwarp();
          if (c + 1 == pieces) release();
          const int live = min(32, x.row_end - x.row0 - 32 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // four rows at a time, eight lanes each
            const int t = 4 * i + lane / 8;
            const float4 f = *reinterpret_cast<const float4*>(own + t * 32 + 4 * (lane & 7));
            float v[4] = {f.x, f.y, f.z, f.w};
            if (t < live) store(v, x.row0 + 32 * c + t, x.n0 + 32 * q + 4 * (lane & 7));
          }
        }
        continue;
      }
      // the partials of the tile before this one have been read by every CTA
      if (done > 0 && !sc_wait<SC_CLUSTER>(part_free, (done - 1) & 1, w, WAIT_SLICES)) break;
      for (int c = 0; c < pieces; ++c) drain(c, part + c * 32 * 128 + 32 * q + lane, 128);
      release();
      arrive_all(part_full);
      if (!sc_wait<SC_CLUSTER>(part_full, done & 1, w, WAIT_SLICES)) break;
      ++done;
      const int live = min(bn, x.row_end - x.row0);
      const int col = x.n0 + 4 * lane;
      // this warp's rows, several at a time: as many loads in flight whatever the slices
      auto finish_rows = [&](auto rows_c, auto slices_c) {
        constexpr int R = decltype(rows_c)::value, MS = decltype(slices_c)::value;
        for (int t0 = int(rank) + slices * e; t0 < live; t0 += slices * kEpiWarps * R) {
          float4 f[R][MS];
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const int t = t0 + i * slices * kEpiWarps;
            const uint32_t at = part_addr + uint32_t(t * 128 + 4 * lane) * 4u;
#pragma unroll
            for (int s = 0; s < MS; ++s)
              if (s < slices && t < live) f[i][s] = ld_cluster_f4(mapa_shared(at, uint32_t(s)));
          }
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const int t = t0 + i * slices * kEpiWarps;
            if (t >= live) continue;
            float v[4] = {f[i][0].x, f[i][0].y, f[i][0].z, f[i][0].w};
#pragma unroll
            for (int s = 1; s < MS; ++s)
              if (s < slices) v[0] += f[i][s].x, v[1] += f[i][s].y, v[2] += f[i][s].z, v[3] += f[i][s].w;
            store(v, x.row0 + t, col);
          }
        }
      };
      if (slices <= 2)
        finish_rows(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
      else if (slices <= 4)
        finish_rows(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
      else
        finish_rows(std::integral_constant<int, 1>{}, std::integral_constant<int, kMaxSlices>{});
      arrive_all(part_free);
    }
  }

  // The CTAs of a cluster stay until all are done reading each other's partials.
  tc_fence_before();
  if (slices > 1)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem_base, cols);
  }
}

// Shared memory of a CTA.
template <bool FOUR>
int sliced_smem(int bn, int stages, int part_rows) {
  return off_table<FOUR>(bn, stages, part_rows) + (SC_MAX_GROUPS + 1) * 4 + 1024;  // + slack for 1024-B alignment
}

template <bool FOUR>
cudaError_t set_limits() {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit == 0 || (ready.load(std::memory_order_acquire) & bit) == 0) {
    cudaError_t err =
        cudaFuncSetAttribute(scaled_sliced_kernel<false, FOUR>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (err == cudaSuccess)
      err = cudaFuncSetAttribute(scaled_sliced_kernel<true, FOUR>, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (err != cudaSuccess) return err;
    ready.fetch_or(bit, std::memory_order_release);
  }
  return cudaSuccess;
}

// Clusters of that many CTAs that can be resident at once, a CTA an SM.
template <bool FOUR>
int resident_clusters(int slices) {
  if (set_limits<FOUR>() != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(slices));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 160 * 1024;  // one CTA an SM
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(slices);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, scaled_sliced_kernel<true, FOUR>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

template <bool FOUR>
cudaError_t launch(const ScMaps& m, const ScParams& p, int grid, cudaStream_t s) {
  auto kern = p.act >= 3 ? scaled_sliced_kernel<true, FOUR> : scaled_sliced_kernel<false, FOUR>;
  const cudaError_t err = set_limits<FOUR>();
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(sliced_smem<FOUR>(p.bn, p.stages, p.part_rows));
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (p.slices > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = unsigned(p.slices);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (p.pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, m, p);
}

}  // namespace
}  // namespace dg
