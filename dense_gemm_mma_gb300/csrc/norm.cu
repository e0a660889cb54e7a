// norm.cu -- root-mean-square norm of a residual stream, and its gradients:
//
//   h = x + r      rho = 1 / sqrt(mean(h^2) + eps)      y = h rho gain
//   g = dy gain    xhat = h rho     dx = rho (g - xhat mean(g xhat)) + dh     dgain = sum over rows of dy xhat
//
// y leaves in the input's type and / or as 8-bit codes with one power-of-two scale for each block of 128 (the
// quantiser's rule, quantize.cu), so that a product's operand needs no pass of its own.  What bounds it is
// memory: x, r, dy and dh are read once, h, y (or codes) and dx written once.
//
// A row stays in registers between its sum of squares and its scaling.  A warp takes 512 columns
// (four blocks of scales, one word of them) at a time, a lane twice eight neighbouring ones: half a warp holds a
// block, whose largest magnitude is four exchanges away.  The row's sum meets in shared memory, one barrier a row.
// Sums, rho and the normalised values are fp32; y and the codes come from the unrounded sum h, one rounding each
// (the kept h is rounded on its own way out), and the gradients from the kept h, which is what the
// caller still has.  The gain's gradient is summed row after row in registers, then over the CTAs in the order
// of their indices by a second launch: the same bits every time, no atomics.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "codes.cuh"
#include "kernels.h"

namespace dg {
namespace {

template <typename T>
__host__ __device__ constexpr int kind_of() {
  return sizeof(T) == 4 ? OUT_F32 : std::is_same<T, __half>::value ? OUT_F16 : OUT_BF16;
}

template <typename T>
__device__ __forceinline__ float to_f(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
}

// Eight neighbouring values of a row as they are loaded; what is not there is zero.
template <typename T>
struct Eight {
  static constexpr int WORDS = int(sizeof(T)) * 2;
  uint32_t w[WORDS];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (std::is_same<T, __half>::value) {
      const uint16_t h = uint16_t(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
      return __half2float(*reinterpret_cast<const __half*>(&h));
    } else {
      return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
  __device__ __forceinline__ void put(int i, T v) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(v);
    } else {
      const uint32_t b = *reinterpret_cast<const uint16_t*>(&v);
      w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | b << 16 : (w[i / 2] & 0xffff0000u) | b;
    }
  }
  // All eight by 16-byte loads.
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
};

// `left` columns from p to the end of the row (none: nothing is read).  a.wide: p is on a 16-byte boundary, so that eight
// columns are loaded whole; the last few of a row one by one.
template <typename T, typename A>
__device__ __forceinline__ void load8(const A& a, Eight<T>& o, const T* p, int left, int site) {
  o.clear();
  if (a.wide && left >= 8) {
    if (DG_IN(a.dbg, p, 8 * int(sizeof(T)), site)) o.load(p);
  } else if (left > 0 && DG_IN(a.dbg, p, min(left, 8) * int(sizeof(T)), site)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) o.put(i, p[i]);
  }
}

template <typename T, typename A>
__device__ __forceinline__ void store8(const A& a, T* p, const float (&v)[8], int left, int site) {
  if (a.wide && left >= 8) {
    Eight<T> o;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o.w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
          const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
          o.w[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          o.w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
    }
    if (!DG_IN(a.dbg, p, 8 * int(sizeof(T)), site)) return;
#pragma unroll
    for (int i = 0; i < Eight<T>::WORDS / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(o.w[4 * i], o.w[4 * i + 1], o.w[4 * i + 2], o.w[4 * i + 3]);
  } else if (left > 0 && DG_IN(a.dbg, p, min(left, 8) * int(sizeof(T)), site)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = from_f<T>(v[i]);
  }
}

// Eight values of the gain (none: ones), which is of the input's type or fp32.
template <typename T, typename A>
__device__ __forceinline__ void load_gain(const A& a, float (&g)[8], int col, int left) {
  if (a.gain == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.f;
  } else if (a.g_kind == kind_of<T>()) {
    Eight<T> o;
    load8(a, o, static_cast<const T*>(a.gain) + col, left, DBG_NORM);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = o.at(i);
  } else {
    Eight<float> o;
    load8(a, o, static_cast<const float*>(a.gain) + col, left, DBG_NORM);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = o.at(i);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// The sum over a row's warps, [first, first + warps) of the CTA's; every thread of the CTA calls it.  (All lanes get
// lane 0's order of additions, whatever their own would be.)
__device__ __forceinline__ float row_sum(float v, float* sums, int first, int warps) {
  if (warps == 1) return warp_sum(v);
  const int lane = threadIdx.x & 31;
  v = warp_sum(v);
  if (lane == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? sums[first + lane] : 0.f;
  // (16 warps at most)
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return __shfl_sync(kAll, v, 0);
}

// Codes of eight values and the scale byte of the block of 128 that they share with the other lanes of half a warp.
template <bool E5M2>
__device__ __forceinline__ uint2 block_codes(const float (&y)[8], uint32_t* byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7fffffffu);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(kAll, m, d));
  const bool careful = __any_sync(kAll, m >= kInf);
  if (careful) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_bits(y[i]));
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(kAll, m, d));
  }
  *byte = scale_byte<E5M2>(m);
  const float inv = inverse_scale(*byte);
  if (careful)
    return make_uint2(codes4<E5M2, true>(y[0], y[1], y[2], y[3], inv), codes4<E5M2, true>(y[4], y[5], y[6], y[7], inv));
  return make_uint2(codes4<E5M2, false>(y[0], y[1], y[2], y[3], inv), codes4<E5M2, false>(y[4], y[5], y[6], y[7], inv));
}

// Eight of a part's sums; parts are on 16-byte boundaries.
__device__ __forceinline__ void store_part(const NormBackArgs& a, float* p, const float (&v)[8]) {
  if (!DG_IN(a.dbg, p, 32, DBG_NORM)) return;
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A row's values as they are loaded, a lane's part of it: x and r, or dy, h and dh.
template <typename TA, typename TB, int G, bool THREE>
struct RowOf {
  Eight<TA> a[2 * G];
  Eight<TB> b[2 * G], c[THREE ? 2 * G : 1];
};

// First column of a lane's i-th eight.
__device__ __forceinline__ int column_of(int i, int mine, int warps) {
  return (mine + i / 2 * warps) * 512 + (i & 1) * 256 + int(threadIdx.x & 31) * 8;
}

// A CTA takes a.per rows at a time, a.warps warps to a row, G groups of 512 columns to a warp; with one group the
// next rows' loads are under way while it works on one (more leave no registers for that).
template <typename TX, typename TH, int G>
__global__ void __launch_bounds__(512, G == 1 && sizeof(TX) == 2 && sizeof(TH) == 2 ? 2 : 1) norm_kernel(const NormArgs a) {
  __shared__ float sums[2][16];
  wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = warp / a.warps, mine = warp - slot * a.warps;
  const bool scaled = a.y || a.q;
  const int rows = a.q ? a.rows_padded : a.rows, step = int(gridDim.x) * a.per;
  auto load = [&](RowOf<TX, TH, G, false>& v, int64_t row) {
    const bool live = row < a.rows;
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
      const int col = column_of(i, mine, a.warps), left = live ? a.cols - col : 0;
      load8(a, v.a[i], static_cast<const TX*>(a.x) + row * a.ldx + col, left, DBG_NORM);
      if (a.r)
        load8(a, v.b[i], static_cast<const TH*>(a.r) + row * a.ldr + col, left, DBG_NORM);
      else
        v.b[i].clear();
    }
  };
  RowOf<TX, TH, G, false> next;
  if constexpr (G == 1) load(next, int64_t(blockIdx.x) * a.per + slot);
  float gain[G < 4 ? 2 * G : 1][8];
  if constexpr (G < 4) {  // (four groups of it leave no registers for the rest)
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
      const int col = column_of(i, mine, a.warps);
      load_gain<TX>(a, gain[i], col, scaled ? a.cols - col : 0);
    }
  }
  int turn = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * a.per; row0 < rows; row0 += step, turn ^= 1) {
    const int64_t row = row0 + slot;  // past the matrix: only scale bytes, zero
    const bool live = row < a.rows;
    if constexpr (G > 1) load(next, row);
    float v[2 * G][8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * G; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = next.a[i].at(j) + next.b[i].at(j);
        sum = fmaf(v[i][j], v[i][j], sum);
      }
    if constexpr (G == 1) {
      if (row0 + step < rows) load(next, row + step);
    }
    sum = row_sum(sum, sums[turn], slot * a.warps, a.warps);
    const float rho = __frsqrt_rn(__fdiv_rn(sum, float(a.cols)) + a.eps);
    if (live && a.rstd && mine == 0 && lane == 0 && DG_IN(a.dbg, a.rstd + row, 4, DBG_NORM)) a.rstd[row] = rho;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
      const int col = column_of(i, mine, a.warps), group = col >> 9;
      const int left = live ? a.cols - col : 0;
      if (a.h) store8(a, static_cast<TH*>(a.h) + row * a.ldh + col, v[i], left, DBG_NORM);
      if (!scaled) continue;
      if constexpr (G == 4) load_gain<TX>(a, gain[0], col, left);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rho * gain[G < 4 ? i : 0][j];
      if (a.y) store8(a, static_cast<TX*>(a.y) + row * a.ldy + col, v[i], left, DBG_NORM);
      if (a.q) {
        // (what is not there is zero, unless rho is infinite)
        if (left < 8) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j >= left) v[i][j] = 0.f;
        }
        uint32_t byte;
        const uint2 c = a.e5m2 ? block_codes<true>(v[i], &byte) : block_codes<false>(v[i], &byte);
        uint8_t* const dst = a.q + row * a.ldq + col;
        if (left >= 8) {
          if (DG_IN(a.dbg, dst, 8, DBG_NORM)) *reinterpret_cast<uint2*>(dst) = c;
        } else if (left > 0 && DG_IN(a.dbg, dst, left, DBG_NORM)) {
          for (int j = 0; j < left; ++j) dst[j] = uint8_t((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
        }
        // bytes of blocks 2 (i & 1) and 2 (i & 1) + 1 of the group, in lanes 0 and 16
        const uint32_t other = __shfl_down_sync(kAll, byte, 16);
        word = (i & 1 ? word : 0u) | (byte | other << 8) << (16 * (i & 1));
        if ((i & 1) && lane == 0 && group < a.q_groups && row < a.rows_padded) {
          uint8_t* const s = a.sq + scale_at(row, int64_t(group) * 4, a.q_groups);
          if (DG_IN(a.dbg, s, 4, DBG_NORM)) *reinterpret_cast<uint32_t*>(s) = word;
        }
      }
    }
  }
}

// Rows of up to kBackCols columns: a lane's sixteen stay in registers, the next row's loads under way.
constexpr int kBackCols = 16 * 512;

template <typename TX, typename TH>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormBackArgs a) {
  __shared__ float sums[2][16];
  wait_prior_grid();
  const int warp = threadIdx.x >> 5;
  const int slot = warp / a.warps, mine = warp - slot * a.warps;
  const int step = int(gridDim.x) * a.per;
  auto load = [&](RowOf<TX, TH, 1, true>& v, float* rho, int64_t row) {
    const bool live = row < a.rows;
    *rho = live && DG_IN(a.dbg, a.rstd + row, 4, DBG_NORM) ? __ldg(a.rstd + row) : 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = column_of(i, mine, a.warps), left = live ? a.cols - col : 0;
      load8(a, v.a[i], static_cast<const TX*>(a.dy) + row * a.lddy + col, left, DBG_NORM);
      load8(a, v.b[i], static_cast<const TH*>(a.h) + row * a.ldh + col, left, DBG_NORM);
      if (a.dh)
        load8(a, v.c[i], static_cast<const TH*>(a.dh) + row * a.lddh + col, left, DBG_NORM);
      else
        v.c[i].clear();
    }
  };
  RowOf<TX, TH, 1, true> now, next;
  float rho_next;
  load(next, &rho_next, int64_t(blockIdx.x) * a.per + slot);
  float gain[2][8], acc[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int col = column_of(i, mine, a.warps);
    load_gain<TX>(a, gain[i], col, a.cols - col);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  }
  int turn = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * a.per; row0 < a.rows; row0 += step, turn ^= 1) {
    const int64_t row = row0 + slot;
    const bool live = row < a.rows;
    now = next;
    const float rho = rho_next;
    if (row0 + step < a.rows) load(next, &rho_next, row + step);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xhat = now.b[i].at(j) * rho, d = now.a[i].at(j);
        acc[i][j] = fmaf(d, xhat, acc[i][j]);
        sum = fmaf(d * gain[i][j], xhat, sum);
      }
    sum = row_sum(sum, sums[turn], slot * a.warps, a.warps);
    const float mean = __fdiv_rn(sum, float(a.cols));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = column_of(i, mine, a.warps);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = fmaf(rho, fmaf(-now.b[i].at(j) * rho, mean, now.a[i].at(j) * gain[i][j]), now.c[i].at(j));
      store8(a, static_cast<TH*>(a.dx) + row * a.lddx + col, v, live ? a.cols - col : 0, DBG_NORM);
    }
  }
  if (!a.parts) return;
  float* const part = a.parts + (int64_t(blockIdx.x) * a.per + slot) * a.part_cols;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int col = column_of(i, mine, a.warps);
    if (col < a.part_cols) store_part(a, part + col, acc[i]);
  }
}

// Longer rows: read twice, the second time from a cache; the gain's gradient is summed in shared memory, each column
// by the one thread that has it.  A CTA a row, a.warps = 16.
template <typename TX, typename TH>
__global__ void __launch_bounds__(512) norm_backward_long_kernel(const NormBackArgs a) {
  extern __shared__ float4 acc_room[];
  __shared__ float sums[2][16];
  wait_prior_grid();
  float* const acc = reinterpret_cast<float*>(acc_room);
  const int first = int(threadIdx.x) * 8, stride = 512 * 8;
  for (int col = first; col < a.part_cols; col += stride)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[col + j] = 0.f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const float rho = DG_IN(a.dbg, a.rstd + row, 4, DBG_NORM) ? __ldg(a.rstd + row) : 0.f;
    const TX* const dy = static_cast<const TX*>(a.dy) + row * a.lddy;
    const TH* const h = static_cast<const TH*>(a.h) + row * a.ldh;
    Eight<TX> d8;
    Eight<TH> h8, p8;
    float gain[8], sum = 0.f;
    for (int col = first; col < a.cols; col += stride) {
      load8(a, d8, dy + col, a.cols - col, DBG_NORM);
      load8(a, h8, h + col, a.cols - col, DBG_NORM);
      load_gain<TX>(a, gain, col, a.cols - col);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xhat = h8.at(j) * rho, d = d8.at(j);
        acc[col + j] = fmaf(d, xhat, acc[col + j]);
        sum = fmaf(d * gain[j], xhat, sum);
      }
    }
    sum = row_sum(sum, sums[turn], 0, 16);
    const float mean = __fdiv_rn(sum, float(a.cols));
    for (int col = first; col < a.cols; col += stride) {
      load8(a, d8, dy + col, a.cols - col, DBG_NORM);
      load8(a, h8, h + col, a.cols - col, DBG_NORM);
      load_gain<TX>(a, gain, col, a.cols - col);
      if (a.dh)
        load8(a, p8, static_cast<const TH*>(a.dh) + row * a.lddh + col, a.cols - col, DBG_NORM);
      else
        p8.clear();
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaf(rho, fmaf(-h8.at(j) * rho, mean, d8.at(j) * gain[j]), p8.at(j));
      store8(a, static_cast<TH*>(a.dx) + row * a.lddx + col, v, a.cols - col, DBG_NORM);
    }
  }
  if (!a.parts) return;
  float* const part = a.parts + int64_t(blockIdx.x) * a.part_cols;
  for (int col = first; col < a.part_cols; col += stride) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = acc[col + j];
    store_part(a, part + col, v);
  }
}

// dgain[c] = sum over the parts: eight columns a CTA, every 128th part to a thread of a column; the threads' sums are
// added in a fixed order.  (32 columns a CTA, every 32nd part: 1 us more for 456 parts of 2050.)
__global__ void __launch_bounds__(1024) norm_gain_kernel(const NormBackArgs a, int parts) {
  __shared__ float sums[32][8];
  wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = int(blockIdx.x) * 8 + (lane & 7);
  float s = 0.f;
  if (col < a.cols) {
#pragma unroll 4
    for (int p = warp * 4 + (lane >> 3); p < parts; p += 128) {
      const float* const at = a.parts + int64_t(p) * a.part_cols + col;
      s += DG_IN(a.dbg, at, 4, DBG_NORM) ? __ldcg(at) : 0.f;
    }
  }
  s += __shfl_xor_sync(kAll, s, 8);
  s += __shfl_xor_sync(kAll, s, 16);
  if (lane < 8) sums[warp][lane] = s;
  __syncthreads();
  if (threadIdx.x >= 8 || col >= a.cols) return;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < 32; ++w) s += sums[w][threadIdx.x];
  if (DG_IN(a.dbg, a.dgain + col, 4, DBG_NORM)) a.dgain[col] = s;
}

// Warps to a row and groups to a warp, for `cols` columns; rows to a CTA, so that it has four warps at least.
struct Shape {
  int g, warps, per;
};
Shape shape_of(int cols, int most_warps, int64_t rows) {
  const int groups = (cols + 511) / 512;
  Shape s;
  s.g = groups <= most_warps ? 1 : groups <= 2 * most_warps ? 2 : 4;
  s.warps = (groups + s.g - 1) / s.g;
  s.per = int(std::max<int64_t>(1, std::min<int64_t>(4 / s.warps, rows)));
  return s;
}

// CTAs of the forward kernel that an SM holds at once, looked up once for each number of warps.
template <typename TX, typename TH, int G>
int norm_ctas(int threads) {
  static std::atomic<int> known[17];
  std::atomic<int>& k = known[threads / 32];
  int n = k.load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_kernel<TX, TH, G>, threads, 0) != cudaSuccess) {
    cudaGetLastError();
    n = 1;
  }
  n = std::max(1, n);
  k.store(n, std::memory_order_relaxed);
  return n;
}

template <typename F>
cudaError_t by_types(int x_kind, int h_kind, F f) {
  if (x_kind == OUT_F32) return f(float{}, float{});
  if (x_kind == OUT_BF16) return h_kind == OUT_F32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
  return h_kind == OUT_F32 ? f(__half{}, float{}) : f(__half{}, __half{});
}

template <typename F>
cudaError_t by_groups(int g, F f) {
  if (g == 1) return f(std::integral_constant<int, 1>{});
  if (g == 2) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 4>{});
}

}  // namespace

cudaError_t launch_norm(NormArgs a, int sms, cudaStream_t s) {
  const int64_t rows = a.q ? a.rows_padded : a.rows;
  const Shape sh = shape_of(a.cols, 16, rows);
  a.warps = sh.warps;
  a.per = sh.per;
  return by_types(a.x_kind, a.h_kind, [&](auto x, auto h) {
    return by_groups(sh.g, [&](auto g) {
      const int64_t fit =
          int64_t(sms) * norm_ctas<decltype(x), decltype(h), decltype(g)::value>(32 * sh.warps * sh.per);
      return launch_k(norm_kernel<decltype(x), decltype(h), decltype(g)::value>, dim3(unsigned(std::min((rows + sh.per - 1) / sh.per, fit))), dim3(unsigned(32 * sh.warps * sh.per)),
                      0, s, a.pdl, a);
    });
  });
}

// Rows' partial sums of the gain's gradient that the launch below makes, and its CTAs.  (16 warps an SM: 128 registers a thread.)
static int norm_parts(int64_t rows, int cols, int sms, int* grid) {
  const Shape sh = shape_of(cols, 16, rows);
  *grid = int(std::min<int64_t>((rows + sh.per - 1) / sh.per, int64_t(sms) * std::max(1, 16 / (sh.warps * sh.per))));
  return *grid * sh.per;
}

size_t norm_backward_workspace(int64_t rows, int64_t cols, int sms) {
  int grid;
  return size_t(norm_parts(rows, int(cols), sms, &grid)) * size_t((cols + 7) / 8 * 8) * 4;
}

namespace {

// The shared memory of the sums has to be asked for, once on each device.
template <typename TX, typename TH>
cudaError_t launch_long(const NormBackArgs& a, int grid, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit == 0 || (ready.load(std::memory_order_acquire) & bit) == 0) {
    const cudaError_t err =
        cudaFuncSetAttribute(norm_backward_long_kernel<TX, TH>, cudaFuncAttributeMaxDynamicSharedMemorySize, NORM_MAX_COLS * 4);
    if (err != cudaSuccess) return err;
    ready.fetch_or(bit, std::memory_order_release);
  }
  return launch_k(norm_backward_long_kernel<TX, TH>, dim3(unsigned(grid)), dim3(512), size_t(a.part_cols) * 4, s, a.pdl, a);
}

}  // namespace

cudaError_t launch_norm_backward(NormBackArgs a, int sms, cudaStream_t s) {
  int grid = 0;
  const int parts = norm_parts(a.rows, a.cols, sms, &grid);
  const Shape sh = shape_of(a.cols, 16, a.rows);
  a.warps = sh.warps;
  a.per = sh.per;
  a.part_cols = (a.cols + 7) / 8 * 8;
  if (!a.dgain) a.parts = nullptr;
  if (a.rows > 0) {
    const cudaError_t err = by_types(a.x_kind, a.h_kind, [&](auto x, auto h) {
      using TX = decltype(x);
      using TH = decltype(h);
      if (a.cols > kBackCols) return launch_long<TX, TH>(a, grid, s);
      return launch_k(norm_backward_kernel<TX, TH>, dim3(unsigned(grid)), dim3(unsigned(32 * sh.warps * sh.per)), 0, s, a.pdl, a);
    });
    if (err != cudaSuccess || !a.dgain) return err;
  }
  return launch_k(norm_gain_kernel, dim3(unsigned((a.cols + 7) / 8)), dim3(1024), 0, s, a.pdl, a, parts);
}

}  // namespace dg
