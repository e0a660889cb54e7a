// scaled.cuh -- what the two 8-bit block-scaled product kernels share.
//
// D[m, n] = act(alpha * sum_k a[m,k] b[n,k] 2^(ea[m,k/128] + eb[n,k/128]) + beta * D[m, n])
//
// a and b are E4M3 or E5M2, K contiguous; ea and eb are power-of-two scales, one
// E8M0 byte for each row and block of 128 along K.  The tensor core applies them:
// tcgen05.mma.kind::mxf8f6f4 multiplies each 32 products of a row pair by two E8M0
// scales before they enter the fp32 accumulator in tensor memory, so a block of 128
// is four MMAs (K = 32) that name the same scale byte, and no partial sum ever leaves
// the accumulator to be scaled.  A power-of-two scale costs nothing in precision: it
// moves the block's exponents and leaves its fractions alone.
//
// The scales come as 512-byte tiles (128 rows x 4 blocks; include/gemm.h), which is
// the image tcgen05.cp lays into tensor memory: one copy per 128 rows serves four
// k-blocks, whose MMAs pick byte (k-block mod 4) of each 32-bit word.
#pragma once

#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace dg {

__device__ __forceinline__ uint32_t sc_pack2(float a, float b, int kind) {
  if (kind == OUT_BF16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float sc_load1(const void* p, int kind) {
  if (kind == OUT_F32) return *static_cast<const float*>(p);
  if (kind == OUT_BF16) return __bfloat162float(*static_cast<const __nv_bfloat16*>(p));
  return __half2float(*static_cast<const __half*>(p));
}

// Two neighbouring 16-bit values of a word.
__device__ __forceinline__ float2 sc_unpack2(uint32_t w, int kind) {
  if (kind == OUT_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}

__device__ __forceinline__ void sc_store1(void* p, float v, int kind) {
  if (kind == OUT_F32)
    *static_cast<float*>(p) = v;
  else if (kind == OUT_BF16)
    *static_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(v);
  else
    *static_cast<__half*>(p) = __float2half_rn(v);
}

// Index of the warp, known to be the same in all its lanes.
__device__ __forceinline__ int sc_warp() { return __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0); }

// One output tile of a call.
struct ScUnit {
  int row0, row_end;  // first row of A (and D) of the tile; end of the rows that exist
  int n0;             // first column
  int zb, zd;         // group whose B / D this is
  int kb0, kb1;       // k-blocks
};

// A group's rows (or K values) as the kernels take them: a start that is no
// multiple of 128 or lies outside [0, cap) means an empty group, a count that
// reaches past cap is cut there, so that no device value leads out of a buffer.
__device__ __forceinline__ void sc_segment(const ScParams& p, int e, int* start, int* count) {
  *start = *count = 0;
  if (!DG_IN(p.dbg, p.starts + e, 4, DBG_SCALED) || !DG_IN(p.dbg, p.counts + e, 4, DBG_SCALED)) return;
  const int s = __ldg(p.starts + e), c = __ldg(p.counts + e);
  const bool ok = s >= 0 && s < p.cap && (s & 127) == 0 && c > 0;
  *start = ok ? s : 0;
  *count = ok ? min(c, p.cap - s) : 0;
}

// From the copy in shared memory, if the kernel has one.
__device__ __forceinline__ void sc_segment_of(const ScParams& p, const int2* seg, int e, int* start, int* count) {
  if (seg) {
    const int2 s = seg[e];
    *start = s.x;
    *count = s.y;
  } else {
    sc_segment(p, e, start, count);
  }
}

// Tile rows of a group.
__device__ __forceinline__ int sc_tile_rows(int count, int tile_rows) {
  return int((uint32_t(count) + uint32_t(tile_rows) - 1) / uint32_t(tile_rows));
}

// SC_ROWS: table[e] = tiles of the groups before e, table[groups] = all tiles; SC_MAX_TILES where there
// would be more (one group has no more, so that only groups that share rows, which a caller's starts
// should not make, get there; tiles past it are left out, and no sum wraps).
// Executed by one warp.  seg: the groups' segments in shared memory, or null.
__device__ __forceinline__ void sc_tile_table(const ScParams& p, int tile_rows, const int2* seg, int* table) {
  const int lane = threadIdx.x & 31;
  int carry = 0;
  for (int e0 = 0; e0 < p.groups; e0 += 32) {
    const int e = e0 + lane;
    int sum = 0;
    if (e < p.groups) {
      int start, count;
      sc_segment_of(p, seg, e, &start, &count);
      sum = sc_tile_rows(count, tile_rows) * p.n_blocks;
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum = min(sum, SC_MAX_TILES - o) + o;
    }
    sum = min(sum, SC_MAX_TILES - carry) + carry;
    if (e < p.groups) table[e + 1] = sum;
    carry = __shfl_sync(0xffffffffu, sum, 31);
  }
  if (lane == 0) table[0] = 0;
}

// Unit u -> tile.  `cursor` (SC_ROWS) is the group of the caller's last unit:
// units are visited in ascending order, so the search for u's group goes on there.
__device__ __forceinline__ ScUnit sc_unit(const ScParams& p, int u, int tile_rows, int tile_cols, const int2* seg,
                                          const int* table, int* cursor) {
  ScUnit x;
  int mb, nb;
  x.zb = x.zd = 0;
  x.kb0 = 0;
  x.kb1 = p.k_blocks;
  if (p.group == SC_ROWS) {
    int e = *cursor;
    while (e + 1 < p.groups && u >= table[e + 1]) ++e;
    *cursor = e;
    int start, count;
    sc_segment_of(p, seg, e, &start, &count);
    tile_coords(u - table[e], sc_tile_rows(count, tile_rows), p.n_blocks, p.raster, &mb, &nb);
    x.row0 = start + mb * tile_rows;
    x.row_end = start + count;
    x.zb = e;
  } else {
    int t = u;
    if (p.group == SC_K) {
      const int per = p.m_blocks * p.n_blocks;
      const int e = u / per;
      t = u - e * per;
      int start, count;
      sc_segment_of(p, seg, e, &start, &count);
      x.kb0 = start / SC_BK;
      x.kb1 = start / SC_BK + sc_tile_rows(count, SC_BK);  // (a start is a multiple of 128)
      x.zd = e;
    }
    tile_coords(t, p.m_blocks, p.n_blocks, p.raster, &mb, &nb);
    x.row0 = mb * tile_rows;
    x.row_end = p.M;
  }
  x.n0 = nb * tile_cols;
  return x;
}

// The MMA warp's cursor through the sets of scale columns in tensor memory.  Set
// g mod 4 holds the scales of the g-th copied group of k-blocks (`it` counts this
// CTA's k-blocks from 0).  The MMAs of group g - 4 must have completed before their
// set is written again.  Full barrier `it` already says that k-blocks up to it -
// stages have: only short groups (a K range that starts or ends inside a group of
// four) leave anything to wait for, on the empty barrier of that group's last stage.
struct ScSets {
  int s1 = -1000000, s2 = -1000000, s3 = -1000000;  // first k-blocks of the last three groups
  uint32_t next = 0;
  // Last k-block that used the set about to be written (group g - 4: group g - 3 starts after it).
  __device__ __forceinline__ int last_user() const { return s3 - 1; }
  __device__ __forceinline__ uint32_t take(int it) {
    s3 = s2;
    s2 = s1;
    s1 = it;
    return (next++) & 3u;
  }
};

// A whole warp's bounded wait: true in every lane, or false in every lane, which then
// leave their loop (the limit ran out, or another role of the CTA gave up).  SC_CLUSTER:
// threads of other CTAs arrive on the barrier, and the wait orders memory after what they wrote;
// SC_RELAXED: they do, and it orders nothing.  The loop is spelled out here: a call on the slow
// path would make every value of the caller's loop leave the uniform registers.
enum : int { SC_OWN, SC_CLUSTER, SC_RELAXED };
template <int FROM>
__device__ __forceinline__ bool sc_wait(uint32_t bar, uint32_t parity, const Watch& w, int code) {
  uint64_t t0 = 0;
  while (true) {
    const bool done = FROM == SC_CLUSTER   ? mbar_try_wait_cluster(bar, parity)
                      : FROM == SC_RELAXED ? mbar_try_wait_cluster_relaxed(bar, parity)
                                           : mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    const uint64_t t = global_timer_ns();
    if (t0 == 0) t0 = t;
    const bool late = t - t0 > w.limit_ns;
    if (__any_sync(0xffffffffu, late)) {
      *w.abort = 1;
      if ((threadIdx.x & 31) == 0) atomicOr(w.err, code);
      return false;
    }
    if (__any_sync(0xffffffffu, *w.abort != 0)) return false;
  }
}

// Which activations a compiled epilogue holds: what a call does not need costs it the instruction
// cache, so that the tile kernel's loops are compiled apart.
enum : int { ACT_SIMPLE = 0, ACT_GELU = 1, ACT_SILU = 2, ACT_ALL = 3 };  // identity, LeakyReLU and ReLU in every one

// x / (1 + exp(-x)) with the fast division (2 units in the last place; 0 where exp(-x) is past 2^126, of
// which the quotient is below 2^-119): the exact one is a call for some operands, and with it in
// the loop a 2711 x 3104 x 5376 product with SiLU took 64.7 us; now 35.2, without an activation 31.8.
__device__ __forceinline__ float sc_silu(float x) { return __fdividef(x, 1.f + expf(-x)); }

// v <- act(v), every run-time choice outside the unrolled loops.
template <int A, int N>
__device__ __forceinline__ void sc_act(float (&v)[N], int act, float slope) {
  if (act == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? v[i] * slope : v[i];
  } else if (act == 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
  }
  if constexpr ((A & ACT_GELU) != 0) {
    if (act == 3) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = apply_act(v[i], 3, 0.f);
    }
  }
  if constexpr ((A & ACT_SILU) != 0) {
    if (act == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = sc_silu(v[i]);
    }
  }
}

}  // namespace dg
