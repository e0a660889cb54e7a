// scaled_tile.cuh -- block-scaled products over whole output tiles: the
// persistent, warp-specialised tcgen05 kernel for calls with enough tiles to
// fill the GPU (formula and scales: scaled.cuh), compiled for 8-bit operands in scaled_tile.cu and for 4-bit
// ones in mx4_tile.cu.
//
//  - warp 0: TMA producer.  A ring stage is one k-block: 128 rows of A
//    and of B (a pair: half of the tile's columns per CTA) by 128 bytes of K, and,
//    with the first k-block of a group of four, the scale tiles of that group.
//  - warp 1: MMA issuer.  Copies a group's scale tiles into one of four
//    sets of tensor-memory columns and issues four K = 32 MMAs per k-block.  Both warps run
//    converged and have one lane issue: with the loop inside a one-lane branch its operands
//    went through vector registers, and a k-block took ~450 cycles and 75 more for each MMA to
//    issue, of which the tensor core needs 512 in all.
//  - warps 2-9: epilogue, 32 accumulator lanes (rows) for two of them, through a swizzled
//    shared-memory box and a TMA store; rows of a box that do not all exist (the
//    last rows of a group) are stored by the threads, so rows between groups
//    are never written.
//
// Pair: 256 x 256 tiles on two CTAs (cta_group::2), each staging its 128 rows of A
// and 128 rows of B: 32 KB per 512 MMA cycles and SM where a 128 x 128 tile per CTA
// needs 32 KB per 256.  Two 256-column accumulators would take all 512 columns
// of tensor memory and leave none for the scales, so they overlap by 64: columns
// 0-255 and 192-447, scales from 448.  The epilogue drains the shared columns of
// a tile first and only then lets the next tile's MMAs begin.
//
// FOUR (4-bit operands): a ring stage is the same 128 bytes of K, 256 values, and four K = 64 MMAs; with a scale for
// each 32 values every stage has scale tiles of its own, two for 128 rows, and a set of scale columns (24 of a pair), so that four sets
// need the accumulators to overlap by 128 columns.  A set is written again when the MMAs that read it have completed.
//  - warp 10 copies the scales, six copies a k-block, and signals the MMA warp.  In the MMA warp itself the copies and the
//    wait for their set made a k-block's eleven instructions longer to issue than its MMAs take (8192^3 187 us; 214 with a copy
//    group before every second MMA).
// SIX: a sixth stage where the results are 16-bit and the groups few.  An epilogue warp's box is then 32 columns of 64
// bytes, and the tables of the groups are short: 8192^3 172 -> 159 us, 2304 x 6912 x 8192 54.6 -> 51.1.
// 8192^3 into bf16 157 to 160 us, 6.9 to 7.0 PFLOP/s.  The MMAs of a k-block take 512 cycles; of five stages a k-block took 550 while the
// ring was full and 640 to 1,100 behind it: 168 to 178 us, without the copies (wrong results) 154, without the stores 150, without the
// loads 139.  The MMAs of the next tile begin ~900 cycles after the last of this one (their completion, 500 for 128 columns to be read, the signal).
//
// What bounds it (8 bits): 8192^3 into bf16 330 to 360 us, 3.1 to 3.3 PFLOP/s, at the power limit (287 us, 3.8
// PFLOP/s, with operands whose bits change little).  Short K: the turnover of the tiles, with no unit full.  16 weight
// gradients of 2048 x 2048 over 1,024 rows each (8 k-blocks a tile) read 537 MB of tiles and write 268 MB in 76 us, and take 61 if
// nothing is written; a load takes 4,000 to 5,000 cycles while the tile before is written, of which the ring covers 2,600.
#pragma once

#include <type_traits>

#include "scaled.cuh"

namespace dg {
namespace {

constexpr int kEpiWarps = 8;     // two for each quarter of the accumulator's lanes
constexpr int kCopyWarp = 2 + kEpiWarps;  // FOUR: copies the scales
template <bool FOUR>
__host__ __device__ constexpr int threads() {
  return 64 + 32 * kEpiWarps + (FOUR ? 32 : 0);
}

// Groups whose segments and tile counts the six-stage kernel has room for.
constexpr int kSixGroups = 64;

template <bool PAIR, bool FOUR, bool SIX>
struct Cfg {
  static_assert(!SIX || (PAIR && FOUR), "six stages: pairs, 4-bit operands");
  static constexpr int TILE_M = PAIR ? 256 : 128;
  static constexpr int BN = PAIR ? 256 : 128;
  static constexpr int OPERAND = 128 * SC_BK;         // bytes of A, and of B, per stage and CTA
  static constexpr int TILES = FOUR ? 2 : 1;           // scale tiles along K of a stage
  static constexpr int SCALES = 512 * TILES * (1 + BN / 128);  // scale tiles of a stage: A's rows, all of the tile's columns
  static constexpr int STAGES = SIX ? 6 : 5;
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = OFF_A + STAGES * OPERAND;
  static constexpr int OFF_STG = OFF_B + STAGES * OPERAND;
  static constexpr int ROW = SIX ? 64 : 128;   // bytes to a row of an epilogue warp's box, its swizzle the same
  static constexpr int BOX = 32 * ROW;
  static constexpr int OFF_S = OFF_STG + kEpiWarps * BOX;
  static constexpr int OFF_BAR = OFF_S + STAGES * SCALES;
  // full[S], empty[S], tmem_full[2], tmem_empty[2], drain, set_full[4], copy_drain
  static constexpr int OFF_MISC = OFF_BAR + (2 * STAGES + 10) * 8;
  static constexpr int OFF_SEG = OFF_MISC + 8;
  static constexpr int GROUPS = SIX ? kSixGroups : SC_MAX_GROUPS;
  static constexpr int OFF_TABLE = OFF_SEG + GROUPS * 8;
  // + slack for 1024-byte alignment (SIX: the declaration's)
  static constexpr int SMEM = OFF_TABLE + (GROUPS + 1) * 4 + (SIX ? 0 : 1024);
  static_assert(SMEM <= 232448, "shared memory budget");
  static constexpr int OVERLAP = !PAIR ? 0 : FOUR ? 128 : 64;  // columns that the two accumulators share
  static constexpr int ACC1 = BN - OVERLAP;      // first column of the second accumulator
  static constexpr int SF0 = ACC1 + BN;          // first scale column
  static constexpr int SET = FOUR ? 8 * (1 + BN / 128) : 16;  // columns of a set
  static constexpr int SETS = 4;
  static constexpr int TMEM_COLS = 512;
  static_assert(SF0 + SETS * SET <= TMEM_COLS, "tensor memory budget");
  static_assert(SETS < STAGES, "a set's last MMAs are waited for on a stage that has not been used again");
};

// v <- alpha * v + beta * D for the columns [col, col + 32) of a row, which start at a 16-byte
// boundary: 16 bytes a load where all of them exist (2711 x 3104 x 5376 with beta into bf16: 36.9 us,
// with 2-byte loads 59.5).
template <int ES>
__device__ __forceinline__ void blend(float (&v)[32], const ScParams& p, const uint8_t* row, int col, bool live) {
  constexpr int PER = 16 / ES;
#pragma unroll
  for (int j = 0; j < 32; j += PER) {
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    const int n = live ? p.N - col - j : 0;
    const uint8_t* const src = row + int64_t(col + j) * ES;
    if (n >= PER) {
      if (DG_IN(p.dbg, src, 16, DBG_SCALED)) q = *reinterpret_cast<const uint4*>(src);
    } else if (n > 0 && DG_IN(p.dbg, src, n * ES, DBG_SCALED)) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i < n) {
          if constexpr (ES == 4)
            w[i] = reinterpret_cast<const uint32_t*>(src)[i];
          else
            w[i / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(src)[i]) << (i & 1) * 16;
        }
      q = make_uint4(w[0], w[1], w[2], w[3]);
    }
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (ES == 4) {
        v[j + i] = fmaf(p.beta, __uint_as_float(w[i]), p.alpha * v[j + i]);
      } else {
        const float2 c = sc_unpack2(w[i], p.out_kind);
        v[j + 2 * i] = fmaf(p.beta, c.x, p.alpha * v[j + 2 * i]);
        v[j + 2 * i + 1] = fmaf(p.beta, c.y, p.alpha * v[j + 2 * i + 1]);
      }
    }
  }
}

// The epilogue's arithmetic, compiled for what a call needs: BETA (with every activation), or
// one of ACT_SIMPLE, ACT_GELU and ACT_SILU without it.
template <bool BETA, int A, bool SHORT>
__device__ __forceinline__ void finish(float (&v)[32], const ScParams& p, const uint8_t* row, int col, bool live) {
  if constexpr (BETA) {
    if (p.out_kind == OUT_F32)
      blend<4>(v, p, row, col, live);
    else
      blend<2>(v, p, row, col, live);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= p.alpha;
  }
  sc_act<A, SHORT>(v, p.act, p.slope);
}

template <bool PAIR, bool FOUR, bool SIX>
__global__ void __launch_bounds__(threads<FOUR>(), 1)
    scaled_tile_kernel(const __grid_constant__ ScMaps maps, const __grid_constant__ ScParams p) {
  using C = Cfg<PAIR, FOUR, SIX>;
  constexpr int S = C::STAGES;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const sbase = smem_raw + (base - raw);
  if (SIX && base != raw) {  // (there is no room for another alignment than the declared one)
    if (threadIdx.x == 0) atomicOr(p.err, WAIT_DRAIN);
    return;
  }
  const int warp = sc_warp();
  const int lane = threadIdx.x & 31;
  const uint32_t full0 = base + C::OFF_BAR, empty0 = full0 + 8 * S;
  const uint32_t tfull0 = empty0 + 8 * S, tempty0 = tfull0 + 16, drain_bar = tempty0 + 16;
  const uint32_t sfull0 = drain_bar + 8, copy_drain_bar = sfull0 + 8 * C::SETS;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(sbase + C::OFF_MISC);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sbase + C::OFF_MISC + 4);
  int2* const seg = reinterpret_cast<int2*>(sbase + C::OFF_SEG);
  int* const table = reinterpret_cast<int*>(sbase + C::OFF_TABLE);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, PAIR ? 2 * kEpiWarps : kEpiWarps);  // both CTAs' epilogues
    }
    mbar_init(drain_bar, 1);
    if constexpr (FOUR) {
      for (int b = 0; b < C::SETS; ++b) mbar_init(sfull0 + 8 * b, 1);
      mbar_init(copy_drain_bar, 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    prefetch_tmap(&maps.d);
    prefetch_tmap(&maps.sa);
    prefetch_tmap(&maps.sb);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  wait_prior_grid();
  if (threadIdx.x == 0) allow_next_grid();
  // The groups' segments: a unit's own read from global memory queued behind the operand loads in
  // flight, 2,000 to 5,000 cycles before every tile (K groups of 1,024, 16 x 2048 x 2048: 86 us, with the copy and the release below 78.7).
  if (p.group != SC_DENSE) {
    for (int e = threadIdx.x; e < p.groups; e += threads<FOUR>()) {
      int start, count;
      sc_segment(p, e, &start, &count);
      seg[e] = make_int2(start, count);
    }
  }
  if (p.group == SC_ROWS) {
    __syncthreads();
    if (warp == 2) sc_tile_table(p, C::TILE_M, seg, table);
  }
  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync();  // both CTAs' barriers exist before either signals the other
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = p.group == SC_ROWS ? table[p.groups] : p.units;
  const int unit0 = PAIR ? int(blockIdx.x) / 2 : int(blockIdx.x);
  const int step = PAIR ? int(gridDim.x) / 2 : int(gridDim.x);
  const Watch w{abort_flag, p.err, p.timeout_ns};
  const uint32_t one = lane == 0;  // the lane that issues

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int stage = 0, issued = 0, cursor = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = unit0; u < units && ok; u += step) {
      const ScUnit x = sc_unit(p, u, C::TILE_M, C::BN, seg, table, &cursor);
      const int m0 = x.row0 + int(rank) * 128, n0 = x.n0 + int(rank) * (PAIR ? 128 : 0);
      // FOUR: row blocks, the scale tiles of each a coordinate of their own
      const int sa_row = FOUR ? m0 / 128 : (m0 / 128) * p.sa_cols;
      const int sb_row = FOUR ? x.zb * p.sb_group + x.n0 / 128 : x.zb * p.sb_group + (x.n0 / 128) * p.sb_cols;
      for (int kb = x.kb0; kb < x.kb1; ++kb) {
        const uint32_t eb = empty0 + 8 * stage, fb = full0 + 8 * stage;
        if (!sc_wait<SC_OWN>(eb, phase ^ 1u, w, WAIT_PRODUCER_EMPTY)) {
          ok = false;
          break;
        }
        const bool scales = FOUR || kb == x.kb0 || (kb & 3) == 0;
        const uint32_t fbc = PAIR ? mapa_shared(fb, 0) : fb;
        mbar_expect_one(fb, uint32_t(PAIR ? 2 : 1) * (2 * C::OPERAND + (scales ? C::SCALES : 0)), one & uint32_t(leader));
        auto load = [&](uint32_t dst, const CUtensorMap* m, int cx, int cy, int cz, int esize) {
          if (!DG_TMA(p.dbg, cx, cy, esize, false)) return;  // (its barrier never completes)
          tma_load_one<PAIR>(dst, m, fbc, cx, cy, cz, one);
        };
        load(base + C::OFF_A + stage * C::OPERAND, &maps.a, kb * SC_BK, m0, 0, 1);
        load(base + C::OFF_B + stage * C::OPERAND, &maps.b, kb * SC_BK, n0, x.zb, 1);
        if (scales) {
          // (row blocks past the matrix read another tile or zero: their rows are not stored)
          const uint32_t sf = base + C::OFF_S + stage * C::SCALES;
          if constexpr (FOUR) {  // (two tiles each: past K the box reads zero)
            load(sf, &maps.sa, 0, 2 * kb, sa_row, 4);
            load(sf + 1024, &maps.sb, 0, 2 * kb, sb_row, 4);  // (of all the tile's columns)
          } else {
            load(sf, &maps.sa, 0, sa_row + kb / 4, 0, 4);
#pragma unroll
            for (int j = 0; j < C::BN / 128; ++j) load(sf + 512 * (1 + j), &maps.sb, 0, sb_row + j * p.sb_cols + kb / 4, 0, 4);
          }
        }
        ++issued;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && leader) {
      // Let the loads already in flight land before the CTA can exit.
      for (int s = 0; s < S; ++s) {
        const int n_s = issued > s ? (issued - s + S - 1) / S : 0;
        if (n_s > 0) sc_wait<SC_OWN>(full0 + 8 * s, (uint32_t)((n_s - 1) & 1), w, 0);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (leader) {
      int stage = 0, it = 0, cursor = 0, tiles = 0;
      uint32_t phase = 0;
      uint32_t set_col = 0;
      ScSets sets;
      bool ok = true;
      bool ready = false;  // the next stage's loads have been seen to have landed
      for (int u = unit0; u < units && ok; u += step) {
        const ScUnit x = sc_unit(p, u, C::TILE_M, C::BN, seg, table, &cursor);
        if (x.kb0 >= x.kb1) continue;  // an empty group: the epilogue writes it without an accumulator
        const int acc = tiles & 1;
        // Overlapping accumulators: the previous tile's shared columns have been
        // drained (and with them the whole tile before it).  Separate ones: this
        // accumulator's last tile has.
        if (C::OVERLAP > 0) {
          if (tiles > 0 && !sc_wait<PAIR ? SC_RELAXED : SC_OWN>(tempty0 + 8 * (acc ^ 1), ((tiles - 1) >> 1) & 1, w, WAIT_MMA_TMEM_EMPTY)) break;
        } else {
          if (tiles > 1 && !sc_wait<PAIR ? SC_RELAXED : SC_OWN>(tempty0 + 8 * acc, ((tiles - 2) >> 1) & 1, w, WAIT_MMA_TMEM_EMPTY)) break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + uint32_t(acc ? C::ACC1 : 0);
        for (int kb = x.kb0; kb < x.kb1; ++kb) {
          if (!__all_sync(0xffffffffu, ready) && !sc_wait<SC_OWN>(full0 + 8 * stage, phase, w, WAIT_MMA_FULL)) {
            ok = false;
            break;
          }
          const int next_stage = stage + 1 == S ? 0 : stage + 1;
          const uint32_t next_phase = phase ^ uint32_t(stage + 1 == S);
          ready = mbar_try_wait(full0 + 8 * next_stage, next_phase);
          if constexpr (FOUR) {
            const int set = it % C::SETS;
            if (!sc_wait<SC_OWN>(sfull0 + 8 * set, uint32_t(it / C::SETS) & 1u, w, WAIT_MMA_FULL)) {
              ok = false;
              break;
            }
            tc_fence_after();
            set_col = tmem_base + C::SF0 + C::SET * uint32_t(set);
          } else if (kb == x.kb0 || (kb & 3) == 0) {
            const int old = sets.last_user();
            if (old >= 0 && old > it - S &&
                !sc_wait<SC_OWN>(empty0 + 8 * (old % S), uint32_t(old / S) & 1u, w, WAIT_MMA_FULL)) {
              ok = false;
              break;
            }
            set_col = tmem_base + C::SF0 + 16 * sets.take(it);
            const uint32_t sf = desc_lo(base + C::OFF_S + stage * C::SCALES);
#pragma unroll
            for (int j = 0; j < 1 + C::BN / 128; ++j) tc_copy_scales<PAIR>(set_col + 4 * j, sf + (512 >> 4) * j, one);
          }
          const uint32_t alo = desc_lo(base + C::OFF_A + stage * C::OPERAND);
          const uint32_t blo = desc_lo(base + C::OFF_B + stage * C::OPERAND);
          if constexpr (FOUR) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_mx4<PAIR>(d_tmem, alo + (32 >> 4) * kk, blo + (32 >> 4) * kk, p.idesc | mx4_ids(kk), set_col + 4 * (kk / 2),
                               set_col + 8 + 4 * (C::BN / 128) * (kk / 2), kb > x.kb0 || kk > 0, one);
          } else {
            const uint32_t id = uint32_t(kb & 3);
            const uint32_t idesc = p.idesc | (id << 4) | (id << 29);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_scaled<PAIR>(d_tmem, alo + (32 >> 4) * kk, blo + (32 >> 4) * kk, idesc, set_col, set_col + 4,
                                  kb > x.kb0 || kk > 0, one);
          }
          tc_commit_one<PAIR>(empty0 + 8 * stage, one);  // stage free (in both CTAs of a pair) once these MMAs finish
          ++it;
          stage = next_stage;
          phase = next_phase;
        }
        if (!ok) break;
        tc_commit_one<PAIR>(tfull0 + 8 * acc, one);
        ++tiles;
      }
      // Every MMA issued by this warp completes before tensor memory is freed.
      tc_commit_leader<PAIR>(drain_bar, one);
      sc_wait<SC_OWN>(drain_bar, 0, w, WAIT_DRAIN);
    }
  } else if (FOUR && warp == kCopyWarp) {
    // ---------------------------------------------------- copy of the scales
    if (leader) {
      int stage = 0, it = 0, cursor = 0, old_stage = 0;
      uint32_t phase = 0, old_phase = 0;
      bool ok = true;
      for (int u = unit0; u < units && ok; u += step) {
        const ScUnit x = sc_unit(p, u, C::TILE_M, C::BN, seg, table, &cursor);
        for (int kb = x.kb0; kb < x.kb1; ++kb, ++it) {
          // The stage has landed, and the MMAs that read this set last, SETS k-blocks ago, have completed.
          if (!sc_wait<SC_OWN>(full0 + 8 * stage, phase, w, WAIT_MMA_FULL) ||
              (it >= C::SETS && !sc_wait<SC_OWN>(empty0 + 8 * old_stage, old_phase, w, WAIT_MMA_FULL))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t set_col = tmem_base + C::SF0 + C::SET * uint32_t(it % C::SETS);
          const uint32_t sf = desc_lo(base + C::OFF_S + stage * C::SCALES);
          // columns: A's two tiles, then B's first tile of each 128 rows, then their second ones
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            tc_copy_scales<PAIR>(set_col + 4 * t, sf + (512 >> 4) * t, one);
#pragma unroll
            for (int j = 0; j < C::BN / 128; ++j)
              tc_copy_scales<PAIR>(set_col + 8 + 4 * (t * (C::BN / 128) + j), sf + (512 >> 4) * (2 * (1 + j) + t), one);
          }
          tc_commit_leader<PAIR>(sfull0 + 8 * (it % C::SETS), one);
          if (it >= C::SETS && ++old_stage == S) {
            old_stage = 0;
            old_phase ^= 1u;
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Every copy completes before tensor memory is freed.
      tc_commit_leader<PAIR>(copy_drain_bar, one);
      sc_wait<SC_OWN>(copy_drain_bar, 0, w, WAIT_DRAIN);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int e = warp - 2;
    const int q = warp & 3;       // tensor-memory lane quarter this warp may read
    const int half = e >> 2;      // which of the quarter's warps: chunks half, half + 2, ...
    constexpr int kHalves = kEpiWarps / 4;
    const uint32_t stg0 = base + C::OFF_STG + e * C::BOX;
    uint8_t* const stg_p0 = sbase + C::OFF_STG + e * C::BOX;
    const int es = !SIX && p.out_kind == OUT_F32 ? 4 : 2;
    const int cw = C::ROW / es;  // columns of a box
    const int chunks = C::BN / cw;
    const int shared_chunks = C::OVERLAP / cw;
    constexpr int kSteps = C::BN / 32 / kHalves;  // 32-column steps of a warp
    static_assert(kSteps % 2 == 0, "steps go in pairs");
    const int per = cw / 32;  // steps to a chunk
    // 128-byte swizzle: 16-byte piece j of row r lives at j ^ (r % 8); 64-byte: at j ^ (r / 2 % 4)
    const int sw = SIX ? lane >> 1 & 3 : lane & 7;
    int cursor = 0, tiles = 0;
    auto tiles_loop = [&](auto beta_c, auto act_c) {
      constexpr bool BETA = decltype(beta_c)::value;
      constexpr int A = decltype(act_c)::value;
      for (int u = unit0; u < units; u += step) {
        const ScUnit x = sc_unit(p, u, C::TILE_M, C::BN, seg, table, &cursor);
        const bool empty = x.kb0 >= x.kb1;
        const int acc = tiles & 1;
        if (!empty) {
          if (!sc_wait<SC_OWN>(tfull0 + 8 * acc, (tiles >> 1) & 1, w, WAIT_EPI_TMEM_FULL)) break;
          tc_fence_after();
          ++tiles;
        }
        // This warp's reads that the next MMAs wait for are complete.  To the leader of a pair without
        // ordering memory: there is none to order, and it took 1,100 to 3,300 cycles.
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (PAIR)
              mbar_arrive_cluster_relaxed(mapa_shared(tempty0 + 8 * acc, 0));
            else
              mbar_arrive(tempty0 + 8 * acc);
          }
          __syncwarp();
        };
        const int y0 = x.row0 + int(rank) * 128 + 32 * q;
        const int live = min(32, x.row_end - y0);  // rows of the box that exist
        if (live <= 0) {
          if (!empty) release();
          continue;
        }
        const bool mine = lane < live;
        // past the last row of a product the TMA clips; past a group's it must not write
        const bool by_tma = p.group != SC_ROWS || live == 32;
        const uint32_t t_row =
            tmem_base + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(acc ? C::ACC1 : 0);
        uint8_t* const d_row = static_cast<uint8_t*>(p.d) + (int64_t(x.zd) * p.d_group + int64_t(y0 + lane) * p.ldd) * es;
        // the shared columns first: the last ones of accumulator 0, the first ones of accumulator 1
        const int first = acc == 0 ? chunks - shared_chunks : 0;
        // Steps of 32 columns, two to a chunk of 16-bit results (SIX: one): step s is columns 32 * (s % per) of
        // this warp's chunk s / per.  After step last_shared it has read what the next MMAs wait for (-1: it
        // has none of it).
        auto chunk_of = [&](int s) { return (half + s / per * kHalves + first) & (chunks - 1); };
        const int last_shared = shared_chunks == 0 ? kSteps - 1 : (shared_chunks - half + kHalves - 1) / kHalves * per - 1;
        if (!empty && last_shared < 0) release();
        // Where the arithmetic is short each step is loaded while the one before is converted (a
        // prompt through 32 experts 215 -> 208 us, weight gradients of 16 experts 78.6 -> 76.2).  Those steps are unrolled,
        // so that no copy of registers that a load still writes is needed on the way; GELU or SiLU four times over no longer
        // fits the instruction cache (2711 x 3104 x 5376, GELU: 44 us, 56 unrolled; 8192 x 8192 x 1024, SiLU: 71 and 84).
        // Nor do their short forms gain (SIX, 8192 x 8192 x 512: SiLU 57 us, 61 unrolled; GELU 76 and 100).
        uint32_t ra[32], rb[32];
        auto load = [&](uint32_t (&r)[32], int s) { tmem_ld_32x32b_x32(t_row + chunk_of(s) * cw + 32 * (s % per), r); };
        auto loaded = [&](uint32_t (&r)[32], int s) {
          tmem_ld_wait(r);
          if (s == last_shared) release();
        };
        auto process = [&](const uint32_t (&r)[32], int s, bool opens, bool closes) {
          const int h = s % per;
          const int x0 = x.n0 + chunk_of(s) * cw;
          if (x0 >= p.N) return;
          uint8_t* const row_p = stg_p0 + lane * C::ROW;
          float v[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
          finish<BETA, A, SIX>(v, p, d_row, x0 + 32 * h, mine);
          if (opens) {
            if (lane == 0) bulk_wait_read<0>();  // the store that last used this box has read it
            __syncwarp();
          }
          if (!SIX && es == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4*>(row_p + ((j ^ sw) << 4)) =
                  make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(row_p + (((4 * h + j) ^ sw) << 4)) = make_uint4(
                  sc_pack2(v[8 * j], v[8 * j + 1], p.out_kind), sc_pack2(v[8 * j + 2], v[8 * j + 3], p.out_kind),
                  sc_pack2(v[8 * j + 4], v[8 * j + 5], p.out_kind), sc_pack2(v[8 * j + 6], v[8 * j + 7], p.out_kind));
          }
          if (!closes) return;
          if (mine) {
            // by the threads: rows of a box that is not whole, in 16-byte pieces up to
            // n_tma, and the columns past the last whole piece of a row
            if (!by_tma) {
              const int piece = 16 / es;
#pragma unroll 1
              for (int j = 0; j < C::ROW / 16 && x0 + (j + 1) * piece <= p.n_tma; ++j) {
                uint8_t* const dst = d_row + int64_t(x0 + j * piece) * es;
                if (DG_IN(p.dbg, dst, 16, DBG_SCALED))
                  *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(row_p + ((j ^ sw) << 4));
              }
            }
            for (int col = max(x0, p.n_tma); col < min(x0 + cw, p.N); ++col) {
              const int b = (col - x0) * es;
              const uint8_t* const src = row_p + (((b >> 4) ^ sw) << 4) + (b & 15);
              uint8_t* const dst = d_row + int64_t(col) * es;
              if (!DG_IN(p.dbg, dst, es, DBG_SCALED)) continue;
              if (es == 4)
                *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
              else
                *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (by_tma && x0 < p.n_tma && DG_TMA(p.dbg, x0, y0, es, true)) tma_store_3d(&maps.d, stg0, x0, y0, x.zd);
            bulk_commit();  // one group per chunk (possibly empty) keeps the buffer accounting exact
          }
          __syncwarp();  // whole again before the next tcgen05.ld
        };
        if (BETA || A != ACT_SIMPLE || empty) {
          // (the next MMAs wait for two steps' columns: both are read before the first one's arithmetic, of which there is one copy)
#pragma unroll 1
          for (int s = 0; s < kSteps; s += 2) {
            if (!empty) {
              load(ra, s);
              load(rb, s + 1);
              loaded(ra, s);
              loaded(rb, s + 1);
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) ra[k] = rb[k] = 0u;
            }
#pragma unroll 1
            for (int t = s; t < s + 2; ++t) {
              process(ra, t, t % per == 0, t % per == per - 1);
#pragma unroll
              for (int k = 0; k < 32; ++k) ra[k] = rb[k];
            }
          }
          continue;
        }
        load(ra, 0);
        load(rb, 1);
#pragma unroll
        for (int s = 0; s < kSteps; s += 2) {
          loaded(ra, s);
          loaded(rb, s + 1);
          process(ra, s, true, SIX || es == 4);
          if (s + 2 < kSteps) load(ra, s + 2);
          process(rb, s + 1, SIX || es == 4, true);
          if (s + 2 < kSteps) load(rb, s + 3);
        }
      }
    };
    if (p.beta != 0.f)
      tiles_loop(std::true_type{}, std::integral_constant<int, ACT_ALL>{});
    else if (p.act == 4)
      tiles_loop(std::false_type{}, std::integral_constant<int, ACT_SILU>{});
    else if (p.act == 3)
      tiles_loop(std::false_type{}, std::integral_constant<int, ACT_GELU>{});
    else
      tiles_loop(std::false_type{}, std::integral_constant<int, ACT_SIMPLE>{});
    // The stores must have read the staging buffers before the CTA exits; the
    // grid's completion covers their writes to global memory.
    if (lane == 0) bulk_wait_read<0>();
  }

  // A pair's CTAs stay until both are done: the leader's MMAs read the peer's
  // shared memory and write its tensor memory.
  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else
      tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <bool PAIR, bool FOUR, bool SIX = false>
cudaError_t launch(const ScMaps& m, const ScParams& p, int grid, cudaStream_t s) {
  constexpr int smem = Cfg<PAIR, FOUR, SIX>::SMEM;
  auto kern = scaled_tile_kernel<PAIR, FOUR, SIX>;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit == 0 || (ready.load(std::memory_order_acquire) & bit) == 0) {
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads<FOUR>());
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (PAIR) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
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

// Pairs that can be resident at once.
template <bool FOUR, bool SIX = false>
int resident_pairs() {
  auto kern = scaled_tile_kernel<true, FOUR, SIX>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<true, FOUR, SIX>::SMEM) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(threads<FOUR>());
  cfg.dynamicSmemBytes = Cfg<true, FOUR, SIX>::SMEM;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

}  // namespace
}  // namespace dg
