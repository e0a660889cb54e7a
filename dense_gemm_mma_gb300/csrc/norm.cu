// norm.cu -- root-mean-square norm of a residual stream, and its gradients:
//
//   h = x + r      rho = 1 / sqrt(mean(h^2) + eps)      y = h rho gain
//   g = dy gain    xhat = h rho     dx = rho (g - xhat mean(g xhat)) + dh     dgain = sum over rows of dy xhat
//
// y leaves in the input's type and / or as 8-bit codes with one power-of-two scale for each block of 128 (the
// quantiser's rule, quantize.cu), so that a product's operand needs no pass of its own.  What bounds it is
// memory: x, r, dy and dh are read once, h, y (or codes) and dx written once.
//
// A row stays in registers between its sum of squares and its scaling.  A warp takes 256 columns
// (two blocks of scales) at a time, a lane eight neighbouring ones: half a warp holds a
// block, whose largest magnitude is four exchanges away.  The row's sum meets in shared memory, one barrier a row.
// Sums, rho and the normalised values are fp32; y and the codes come from the unrounded sum h, one rounding each
// (the kept h is rounded on its own way out), and the gradients from the kept h, which is what the
// caller still has.  The gain's gradient is summed row after row in registers, then over the CTAs in the order
// of their indices by a second launch: the same bits every time, no atomics.
// Measured, bf16: 1 x 4096 2.1 us; 8192 x 4096 with the residual 44 us (6.1 TB/s), into codes 43 (5.5); 6912 x 2050 21.5 us, its
// gradients 27.1 with the gain's, 24.7 without; 4096 x 10240 gradients 79.7 us (4.2), x 16384 124 (4.3), fp32 199 (5.4).
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

// `left` columns from p to the end of the row (none: nothing is read).  a.wide: what p's alignment allows, 16 bytes (eight
// columns are loaded whole), 4 (words, as the last columns of a row always are then) or 0 (value by value).  Words go
// straight to their registers: a value that has to be put together is waited for at once, which made the
// loads for the next row no loads ahead (6912 x 2050, gradients: 36.6 us for 113 MB, 8192 x 2048 26.9 for 134).
template <typename T, typename A>
__device__ __forceinline__ void load8(const A& a, Eight<T>& o, const T* p, int left, int site) {
  o.clear();
  if (a.wide == 16 && left >= 8) {
    if (DG_IN(a.dbg, p, 8 * int(sizeof(T)), site)) o.load(p);
  } else if (left > 0 && DG_IN(a.dbg, p, min(left, 8) * int(sizeof(T)), site)) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) o.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else if (a.wide) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (2 * i + 1 < left)
          o.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else if (2 * i < left)
          o.w[i] = reinterpret_cast<const uint16_t*>(p)[2 * i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) o.put(i, p[i]);
    }
  }
}

template <typename T, typename A>
__device__ __forceinline__ void store8(const A& a, T* p, const float (&v)[8], int left, int site) {
  if (left <= 0 || !DG_IN(a.dbg, p, min(left, 8) * int(sizeof(T)), site)) return;
  if constexpr (sizeof(T) == 4) {
    if (a.wide == 16 && left >= 8) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = v[i];
    }
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    if (a.wide == 16 && left >= 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (a.wide && 2 * i + 1 < left) {
          reinterpret_cast<uint32_t*>(p)[i] = w[i];
        } else {
          if (2 * i < left) reinterpret_cast<uint16_t*>(p)[2 * i] = uint16_t(w[i]);
          if (2 * i + 1 < left) reinterpret_cast<uint16_t*>(p)[2 * i + 1] = uint16_t(w[i] >> 16);
        }
      }
    }
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
template <typename TA, typename TB, int NE, bool THREE>
struct RowOf {
  Eight<TA> a[NE];
  Eight<TB> b[NE], c[THREE ? NE : 1];
};

// First column of a lane's i-th eight: two neighbouring 256s of a warp are a word of scales.
template <int NE>
__device__ __forceinline__ int column_of(int i, int mine, int warps) {
  const int piece = NE == 1 ? mine : (mine + i / 2 * warps) * 2 + (i & 1);
  return piece * 256 + int(threadIdx.x & 31) * 8;
}

// A CTA takes a.per rows at a time, a.warps warps to a row, NE times 256 columns to a warp; up to two the
// next rows' loads are under way while it works on one (more leave no registers for that).
template <typename TX, typename TH, int NE>
__global__ void __launch_bounds__(512, NE <= 2 && sizeof(TX) == 2 && sizeof(TH) == 2 ? 2 : 1) norm_kernel(const NormArgs a) {
  __shared__ float sums[2][16];
  wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = warp / a.warps, mine = warp - slot * a.warps;
  const bool scaled = a.y || a.q;
  const int rows = a.q ? a.rows_padded : a.rows, step = int(gridDim.x) * a.per;
  auto load = [&](RowOf<TX, TH, NE, false>& v, int64_t row) {
    const bool live = row < a.rows;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int col = column_of<NE>(i, mine, a.warps), left = live ? a.cols - col : 0;
      load8(a, v.a[i], static_cast<const TX*>(a.x) + row * a.ldx + col, left, DBG_NORM);
      if (a.r)
        load8(a, v.b[i], static_cast<const TH*>(a.r) + row * a.ldr + col, left, DBG_NORM);
      else
        v.b[i].clear();
    }
  };
  RowOf<TX, TH, NE, false> next;
  if constexpr (NE <= 2) load(next, int64_t(blockIdx.x) * a.per + slot);
  float gain[NE < 8 ? NE : 1][8];
  if constexpr (NE < 8) {  // (eight of them leave no registers for the rest)
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int col = column_of<NE>(i, mine, a.warps);
      load_gain<TX>(a, gain[i], col, scaled ? a.cols - col : 0);
    }
  }
  int turn = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * a.per; row0 < rows; row0 += step, turn ^= 1) {
    const int64_t row = row0 + slot;  // past the matrix: only scale bytes, zero
    const bool live = row < a.rows;
    if constexpr (NE > 2) load(next, row);
    float v[NE][8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = next.a[i].at(j) + next.b[i].at(j);
        sum = fmaf(v[i][j], v[i][j], sum);
      }
    if constexpr (NE <= 2) {
      if (row0 + step < rows) load(next, row + step);
    }
    sum = row_sum(sum, sums[turn], slot * a.warps, a.warps);
    const float rho = __frsqrt_rn(__fdiv_rn(sum, float(a.cols)) + a.eps);
    if (live && a.rstd && mine == 0 && lane == 0 && DG_IN(a.dbg, a.rstd + row, 4, DBG_NORM)) a.rstd[row] = rho;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int col = column_of<NE>(i, mine, a.warps);
      const int left = live ? a.cols - col : 0;
      if (a.h) store8(a, static_cast<TH*>(a.h) + row * a.ldh + col, v[i], left, DBG_NORM);
      if (!scaled) continue;
      if constexpr (NE == 8) load_gain<TX>(a, gain[0], col, left);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rho * gain[NE < 8 ? i : 0][j];
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
        // the bytes of both blocks, in lane 0
        const uint32_t two = byte | __shfl_down_sync(kAll, byte, 16) << 8;
        word = i & 1 ? word | two << 16 : two;
        if (lane == 0 && (NE == 1 || (i & 1)) && (col >> 9) < a.q_groups && row < a.rows_padded) {
          uint8_t* const s = a.sq + scale_at(row, NE == 1 ? col >> 7 : col >> 9 << 2, a.q_groups);
          if constexpr (NE == 1) {
            if (DG_IN(a.dbg, s, 2, DBG_NORM)) *reinterpret_cast<uint16_t*>(s) = uint16_t(word);
          } else {
            if (DG_IN(a.dbg, s, 4, DBG_NORM)) *reinterpret_cast<uint32_t*>(s) = word;
          }
        }
      }
    }
  }
}

// Rows of up to kBackCols columns: a lane's eight or sixteen stay in registers, the next row's loads under way.
constexpr int kBackCols = 16 * 512;

template <typename TX, typename TH, int NE>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormBackArgs a) {
  __shared__ float sums[2][16];
  wait_prior_grid();
  const int warp = threadIdx.x >> 5;
  const int slot = warp / a.warps, mine = warp - slot * a.warps;
  const int step = int(gridDim.x) * a.per;
  auto load = [&](RowOf<TX, TH, NE, true>& v, float* rho, int64_t row) {
    const bool live = row < a.rows;
    *rho = live && DG_IN(a.dbg, a.rstd + row, 4, DBG_NORM) ? __ldg(a.rstd + row) : 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int col = column_of<NE>(i, mine, a.warps), left = live ? a.cols - col : 0;
      load8(a, v.a[i], static_cast<const TX*>(a.dy) + row * a.lddy + col, left, DBG_NORM);
      load8(a, v.b[i], static_cast<const TH*>(a.h) + row * a.ldh + col, left, DBG_NORM);
      if (a.dh)
        load8(a, v.c[i], static_cast<const TH*>(a.dh) + row * a.lddh + col, left, DBG_NORM);
      else
        v.c[i].clear();
    }
  };
  RowOf<TX, TH, NE, true> now, next;
  float rho_next;
  load(next, &rho_next, int64_t(blockIdx.x) * a.per + slot);
  float gain[NE][8], acc[NE][8];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int col = column_of<NE>(i, mine, a.warps);
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
    for (int i = 0; i < NE; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xhat = now.b[i].at(j) * rho, d = now.a[i].at(j);
        acc[i][j] = fmaf(d, xhat, acc[i][j]);
        sum = fmaf(d * gain[i][j], xhat, sum);
      }
    sum = row_sum(sum, sums[turn], slot * a.warps, a.warps);
    const float mean = __fdiv_rn(sum, float(a.cols));
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int col = column_of<NE>(i, mine, a.warps);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = fmaf(rho, fmaf(-now.b[i].at(j) * rho, mean, now.a[i].at(j) * gain[i][j]), now.c[i].at(j));
      store8(a, static_cast<TH*>(a.dx) + row * a.lddx + col, v, live ? a.cols - col : 0, DBG_NORM);
    }
  }
  if (!a.parts) return;
  // the CTA's rows together, in the order of their slots (several only where four warps have a row each or two rows)
  __shared__ float room[4 * 2 * 256];
  for (int k = 1; k < a.per; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      float* const at = room + column_of<NE>(i, mine, a.warps);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (slot == k) at[j] = acc[i][j];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const float* const at = room + column_of<NE>(i, mine, a.warps);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (slot == 0) acc[i][j] += at[j];
    }
  }
  if (slot > 0) return;
  float* const part = a.parts + int64_t(blockIdx.x) * a.part_cols;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int col = column_of<NE>(i, mine, a.warps);
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
    for (int p0 = warp * 4 + (lane >> 3); p0 < parts; p0 += 4 * 128) {  // (four loads together, whatever is left)
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = p0 + j * 128;
        const float* const at = a.parts + int64_t(p) * a.part_cols + col;
        v[j] = p < parts && DG_IN(a.dbg, at, 4, DBG_NORM) ? __ldcg(at) : 0.f;
      }
      s += (v[0] + v[1]) + (v[2] + v[3]);
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

// Warps to a row, each with `ne` times 256 columns (codes: whole words of scales, 512 columns), and rows to a CTA, so that it
// has four warps at least.  256 columns a warp up to 16 warps, which is latency's best (1 x 4096: 2.1 us, with 512 a warp 2.4;
// 8192 x 4096 bf16 44.4 and 47.9), except where more warps cost more than they hide: codes of many rows
// (8192 x 4096: 50.3, with 512 a warp 48.8) and the gradients of 16-bit rows (8192 x 4096: 60.1 and 49.3; 32-bit 87.6 and 101).
enum Form : int { FORM_PLAIN, FORM_CODES, FORM_BACK16, FORM_BACK32 };
struct Shape {
  int ne, warps, per;
};
Shape shape_of(int cols, Form form, int64_t rows) {
  const int pieces = form == FORM_CODES ? (cols + 511) / 512 * 2 : (cols + 255) / 256;
  const int most = form == FORM_BACK16 || (form == FORM_CODES && rows > 1024) ? 4 : 16;
  Shape s;
  s.ne = pieces <= most ? 1 : pieces <= 32 ? 2 : pieces <= 64 ? 4 : 8;
  s.warps = (pieces + s.ne - 1) / s.ne;
  s.per = int(std::max<int64_t>(1, std::min<int64_t>(4 / s.warps, rows)));
  return s;
}

Shape back_shape(int x_kind, int64_t cols, int64_t rows) {
  return shape_of(int(cols), x_kind == OUT_F32 ? FORM_BACK32 : FORM_BACK16, rows);
}

// CTAs of a kernel that an SM holds at once; `known`: the kernel's, by warps, looked up once each.
template <typename K>
int resident(K kern, int threads, size_t smem, std::atomic<int>* known) {
  std::atomic<int>& k = known[threads / 32];
  int n = k.load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) != cudaSuccess) {
    cudaGetLastError();
    n = 1;
  }
  n = std::max(1, n);
  k.store(n, std::memory_order_relaxed);
  return n;
}

template <typename TX, typename TH, int NE>
int norm_ctas(int threads) {
  static std::atomic<int> known[17];
  return resident(norm_kernel<TX, TH, NE>, threads, 0, known);
}

template <typename TX, typename TH, int NE>
int norm_backward_ctas(int threads) {
  static std::atomic<int> known[17];
  return resident(norm_backward_kernel<TX, TH, NE>, threads, 0, known);
}

template <typename F>
cudaError_t by_types(int x_kind, int h_kind, F f) {
  if (x_kind == OUT_F32) return f(float{}, float{});
  if (x_kind == OUT_BF16) return h_kind == OUT_F32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
  return h_kind == OUT_F32 ? f(__half{}, float{}) : f(__half{}, __half{});
}

template <typename F>
cudaError_t by_eights(int ne, F f) {
  if (ne == 1) return f(std::integral_constant<int, 1>{});
  if (ne == 2) return f(std::integral_constant<int, 2>{});
  if (ne == 4) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 8>{});
}

}  // namespace

cudaError_t launch_norm(NormArgs a, int sms, cudaStream_t s) {
  const int64_t rows = a.q ? a.rows_padded : a.rows;
  const Shape sh = shape_of(a.cols, a.q ? FORM_CODES : FORM_PLAIN, rows);
  a.warps = sh.warps;
  a.per = sh.per;
  return by_types(a.x_kind, a.h_kind, [&](auto x, auto h) {
    return by_eights(sh.ne, [&](auto g) {
      const int64_t fit =
          int64_t(sms) * norm_ctas<decltype(x), decltype(h), decltype(g)::value>(32 * sh.warps * sh.per);
      return launch_k(norm_kernel<decltype(x), decltype(h), decltype(g)::value>, dim3(unsigned(std::min((rows + sh.per - 1) / sh.per, fit))), dim3(unsigned(32 * sh.warps * sh.per)),
                      0, s, a.pdl, a);
    });
  });
}

namespace {

// The shared memory of the sums has to be asked for, once on each device.
template <typename TX, typename TH>
cudaError_t allow_long() {
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
  return cudaSuccess;
}

// CTAs of the long rows' kernel that an SM holds at once: registers allow two or three, the rows' sums one to six.  As many as the
// sums allow, waves of which the last was half empty and up to three times the parts: 4096 x 10240 bf16 97.6 us, so 79.7; x 16384 fp32 248
// and 199.  (Asked at every call: it goes by the columns.)
template <typename TX, typename TH>
int norm_long_ctas(size_t smem) {
  int n = 0;
  if (allow_long<TX, TH>() != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, norm_backward_long_kernel<TX, TH>, 512, smem) != cudaSuccess)
    cudaGetLastError();
  return std::max(1, n);
}

}  // namespace

int norm_backward_grid(int x_kind, int h_kind, int64_t rows, int64_t cols, int sms) {
  const Shape sh = back_shape(x_kind, cols, rows);
  int fit = 1;
  by_types(x_kind, h_kind, [&](auto x, auto h) {
    using TX = decltype(x);
    using TH = decltype(h);
    const int threads = 32 * sh.warps * sh.per;
    fit = cols > kBackCols ? norm_long_ctas<TX, TH>(size_t(norm_part_cols(cols)) * 4)
          : sh.ne == 1     ? norm_backward_ctas<TX, TH, 1>(threads)
                           : norm_backward_ctas<TX, TH, 2>(threads);
    return cudaSuccess;
  });
  return int(std::min<int64_t>((rows + sh.per - 1) / sh.per, int64_t(sms) * fit));
}

namespace {

template <typename TX, typename TH>
cudaError_t launch_long(const NormBackArgs& a, int grid, cudaStream_t s) {
  const cudaError_t err = allow_long<TX, TH>();
  if (err != cudaSuccess) return err;
  return launch_k(norm_backward_long_kernel<TX, TH>, dim3(unsigned(grid)), dim3(512), size_t(a.part_cols) * 4, s, a.pdl, a);
}

}  // namespace

cudaError_t launch_norm_backward(NormBackArgs a, int grid, cudaStream_t s) {
  const Shape sh = back_shape(a.x_kind, a.cols, a.rows);
  a.warps = sh.warps;
  a.per = sh.per;
  a.part_cols = norm_part_cols(a.cols);
  if (!a.dgain) a.parts = nullptr;
  if (a.rows > 0) {
    const cudaError_t err = by_types(a.x_kind, a.h_kind, [&](auto x, auto h) {
      using TX = decltype(x);
      using TH = decltype(h);
      if (a.cols > kBackCols) return launch_long<TX, TH>(a, grid, s);
      return launch_k(sh.ne == 1 ? norm_backward_kernel<TX, TH, 1> : norm_backward_kernel<TX, TH, 2>, dim3(unsigned(grid)), dim3(unsigned(32 * sh.warps * sh.per)), 0, s, a.pdl, a);
    });
    if (err != cudaSuccess || !a.dgain) return err;
  }
  return launch_k(norm_gain_kernel, dim3(unsigned((a.cols + 7) / 8)), dim3(1024), 0, s, a.pdl, a, grid);
}

}  // namespace dg
