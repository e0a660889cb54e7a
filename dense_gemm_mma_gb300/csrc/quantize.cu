// quantize.cu -- a matrix to 8 bits with one power-of-two scale for each block of
// 128 values, as it stands and transposed; and the copy of codes whose rows the TMA
// cannot address.
//
// For a block with largest finite magnitude m, the scale is 2^e with the least e that
// keeps m * 2^-e within the type's largest value (448 = 1.75 * 2^8 for E4M3, 57344 =
// 1.75 * 2^15 for E5M2), at least 2^-127.  With m = f * 2^E, 1 <= f < 2, that is
// e = E - 8 + (f > 1.75) (E - 15 ... for E5M2): integer arithmetic on m's bits, no
// logarithm.  Multiplying by 2^-e is exact, so a code is one rounding (to nearest, ties to even)
// away from its value.  Infinities and NaN take no part in m and become NaN.
//
// What bounds it is memory: each value is read once, and written once per
// orientation.  Maxima are taken on the magnitudes' bits (ordered like the numbers),
// one warp reduction per row and block.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kernels.h"

namespace dg {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }

// Four consecutive values of a row, the first n of which exist (the rest are 0).
template <typename T>
__device__ __forceinline__ void load4(float (&v)[4], const T* p, int n, bool vec) {
  if (vec && n >= 4) {
    if constexpr (sizeof(T) == 4) {
      const float4 q = *reinterpret_cast<const float4*>(p);
      v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      alignas(8) T h[4];
      *reinterpret_cast<uint2*>(h) = q;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = to_f(h[i]);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < n ? to_f(p[i]) : 0.f;
}

// |v|'s bits, 0 for infinities and NaN.
__device__ __forceinline__ uint32_t magnitude(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}

// Scale byte (e + 127) of a block whose largest magnitude has the bits m.
template <bool E5M2>
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  const int b = int(m >> 23) - (E5M2 ? 15 : 8) + int((m & 0x7fffffu) > 0x600000u);
  return uint32_t(max(b, 0));
}

__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Codes of v * inv; what is not finite becomes NaN (the conversion would saturate infinities).
template <bool E5M2>
__device__ __forceinline__ uint32_t codes2(float a, float b, float inv) {
  const float nan = __uint_as_float(0x7fc00000u);
  a = fabsf(a) < __uint_as_float(0x7f800000u) ? a * inv : nan;
  b = fabsf(b) < __uint_as_float(0x7f800000u) ? b * inv : nan;
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, E5M2 ? __NV_E5M2 : __NV_E4M3);
}

// Byte of row r, block c in the packed scales of a matrix with `groups` groups of four blocks.
__device__ __forceinline__ int64_t scale_at(int64_t r, int64_t c, int64_t groups) {
  return ((r >> 7) * groups + (c >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (c & 3);
}

__device__ __forceinline__ int source_row(const QuantArgs& a, int r) {
  if (r >= a.rows) return -1;
  if (!a.rowmap) return r;
  const int s = __ldg(a.rowmap + r);
  if (s < 0) return -1;
  const int row = s / a.map_div;
  return row < a.src_rows ? row : -1;
}

// One orientation, a scale for each row's block: a warp takes kRows rows of 512
// columns (one word of scale bytes each), all its loads in flight together.
constexpr int kRows = 2;

template <typename T, bool E5M2>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantArgs a) {
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int groups = a.q_groups;
  const int r0 = int(warp / groups) * kRows;
  const int g = int(warp % groups);
  if (r0 >= a.rows_padded) return;
  const T* const x = static_cast<const T*>(a.x);
  float v[kRows][4][4];
  int src[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) src[i] = source_row(a, r0 + i);
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int col = g * 512 + b * 128 + 4 * lane;
      const T* const p = x + int64_t(src[i]) * a.ldx + col;
      const int n = src[i] >= 0 ? min(4, a.cols - col) : 0;
      load4(v[i][b], p, n > 0 && DG_IN(a.dbg, p, n * int(sizeof(T)), DBG_QUANTIZE) ? n : 0, a.vec);
    }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    uint32_t word = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      float(&w)[4] = v[i][b];
      const uint32_t m = __reduce_max_sync(
          kAll, max(max(magnitude(w[0]), magnitude(w[1])), max(magnitude(w[2]), magnitude(w[3]))));
      const uint32_t byte = scale_byte<E5M2>(m);
      word |= byte << (8 * b);
      const int col = g * 512 + b * 128 + 4 * lane;
      const int n = src[i] >= 0 ? min(4, a.cols - col) : 0;
      if (n <= 0) continue;
      const float inv = inverse_scale(byte);
      const uint32_t c = codes2<E5M2>(w[0], w[1], inv) | codes2<E5M2>(w[2], w[3], inv) << 16;
      uint8_t* const dst = a.q + int64_t(r0 + i) * a.ldq + col;
      if (!DG_IN(a.dbg, dst, n, DBG_QUANTIZE)) continue;
      if (n == 4)
        *reinterpret_cast<uint32_t*>(dst) = c;
      else
        for (int t = 0; t < n; ++t) dst[t] = uint8_t(c >> (8 * t));
    }
    uint8_t* const s = a.sq + scale_at(r0 + i, int64_t(g) * 4, groups);
    if (lane == 0 && DG_IN(a.dbg, s, 4, DBG_QUANTIZE)) *reinterpret_cast<uint32_t*>(s) = word;
  }
}

// Both orientations (or 128 x 128 scales): a CTA takes one 128 x 128 tile, 16 rows a
// warp and 4 columns a lane, held in registers.  Row maxima are warp reductions;
// column maxima meet in shared memory.  A thread's 16 rows of a column are 16 consecutive
// bytes of the transposed matrix: they are turned round in a swizzled shared-memory tile
// and leave as 128-byte rows.
template <typename T, bool E5M2>
__global__ void __launch_bounds__(256) quantize_tile_kernel(const QuantArgs a) {
  __shared__ uint32_t col_max[8][128];
  __shared__ uint4 turn[128 * 8];  // [column][16-byte piece of rows ^ (column / 4 % 8)]
  wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cb = blockIdx.x, rb = blockIdx.y;  // past the matrix: only scale bytes, zero
  const int row0 = rb * 128 + warp * 16, col = cb * 128 + 4 * lane;
  const T* const x = static_cast<const T*>(a.x);
  float v[16][4];
  uint32_t live = 0;  // rows that are read
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int src = source_row(a, row0 + i);
    const int n = src >= 0 ? min(4, a.cols - col) : 0;
    const T* const p = x + int64_t(src) * a.ldx + col;
    load4(v[i], p, n > 0 && DG_IN(a.dbg, p, n * int(sizeof(T)), DBG_QUANTIZE) ? n : 0, a.vec);
    live |= uint32_t(src >= 0) << i;
  }
  uint32_t cm[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) cm[j] = max(cm[j], magnitude(v[i][j]));
  *reinterpret_cast<uint4*>(&col_max[warp][4 * lane]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const uint4 o = *reinterpret_cast<const uint4*>(&col_max[w][4 * lane]);
    cm[0] = max(cm[0], o.x), cm[1] = max(cm[1], o.y), cm[2] = max(cm[2], o.z), cm[3] = max(cm[3], o.w);
  }
  uint32_t tile = 0;  // scale byte of the whole tile
  if (a.block_rows > 1) tile = scale_byte<E5M2>(__reduce_max_sync(kAll, max(max(cm[0], cm[1]), max(cm[2], cm[3]))));
  if (a.q) {
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint32_t byte = tile;
      if (a.block_rows == 1)
        byte = scale_byte<E5M2>(__reduce_max_sync(
            kAll, max(max(magnitude(v[i][0]), magnitude(v[i][1])), max(magnitude(v[i][2]), magnitude(v[i][3])))));
      if (lane == i) mine = byte;
      const int n = (live >> i) & 1 ? min(4, a.cols - col) : 0;
      if (n <= 0) continue;
      const float inv = inverse_scale(byte);
      const uint32_t c = codes2<E5M2>(v[i][0], v[i][1], inv) | codes2<E5M2>(v[i][2], v[i][3], inv) << 16;
      uint8_t* const dst = a.q + int64_t(row0 + i) * a.ldq + col;
      if (!DG_IN(a.dbg, dst, n, DBG_QUANTIZE)) continue;
      if (n == 4)
        *reinterpret_cast<uint32_t*>(dst) = c;
      else
        for (int t = 0; t < n; ++t) dst[t] = uint8_t(c >> (8 * t));
    }
    if (lane < 16 && row0 < a.rows_padded) {
      uint8_t* const s = a.sq + scale_at(row0 + lane, cb, a.q_groups);
      if (DG_IN(a.dbg, s, 1, DBG_QUANTIZE)) *s = uint8_t(row0 + lane < a.rows || a.block_rows == 1 ? mine : 0u);
    }
  }
  if (a.qt) {
    uint32_t bytes[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) bytes[j] = a.block_rows == 1 ? scale_byte<E5M2>(cm[j]) : tile;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float inv = inverse_scale(bytes[j]);
      uint32_t w[4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        w[h] = codes2<E5M2>(v[4 * h][j], v[4 * h + 1][j], inv) | codes2<E5M2>(v[4 * h + 2][j], v[4 * h + 3][j], inv) << 16;
      turn[(4 * lane + j) * 8 + (warp ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (warp == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (col + j < a.cols_padded) {
          uint8_t* const s = a.sqt + scale_at(col + j, rb, a.qt_groups);
          if (DG_IN(a.dbg, s, 1, DBG_QUANTIZE)) *s = uint8_t(col + j < a.cols || a.block_rows == 1 ? bytes[j] : 0u);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int pass = 0; pass < 4; ++pass) {
      const int c = pass * 32 + int(threadIdx.x >> 3), piece = threadIdx.x & 7;
      const int r = rb * 128 + piece * 16;
      if (cb * 128 + c >= a.cols || r >= a.rows) continue;
      const uint4 w = turn[c * 8 + (piece ^ ((c >> 2) & 7))];
      uint8_t* const dst = a.qt + int64_t(cb * 128 + c) * a.ldqt + r;
      const int n = min(16, a.rows - r);
      if (!DG_IN(a.dbg, dst, n, DBG_QUANTIZE)) continue;
      if (n == 16) {
        *reinterpret_cast<uint4*>(dst) = w;
      } else {
        const uint32_t part[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int t = 0; t < 16; ++t)
          if (t < n) dst[t] = uint8_t(part[t / 4] >> (8 * (t & 3)));
      }
    }
  }
}

template <typename T, bool E5M2>
cudaError_t launch(const QuantArgs& a, cudaStream_t s) {
  if (!a.qt && a.block_rows == 1) {
    const int64_t warps = int64_t(a.rows_padded / kRows) * a.q_groups;
    return launch_k(quantize_rows_kernel<T, E5M2>, dim3(unsigned((warps + 7) / 8)), dim3(256), 0, s, a.pdl, a);
  }
  // blocks past the matrix write the zero bytes that pad the scales to whole words
  const int col_blocks = a.q ? a.q_groups * 4 : (a.cols + 127) / 128;
  const int row_blocks = a.qt ? a.qt_groups * 4 : (a.rows + 127) / 128;
  return launch_k(quantize_tile_kernel<T, E5M2>, dim3(unsigned(col_blocks), unsigned(row_blocks)), dim3(256), 0, s,
                  a.pdl, a);
}

template <typename T>
cudaError_t launch_type(const QuantArgs& a, cudaStream_t s) {
  return a.e5m2 ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

// One thread 16 bytes of a row, loaded in pieces that the rows' alignment allows (T).
template <typename T>
__global__ void __launch_bounds__(256) repack_kernel(const RepackArgs a) {
  wait_prior_grid();
  const int r = int(blockIdx.x), z = int(blockIdx.z);
  const int col = int(blockIdx.y * blockDim.x + threadIdx.x) * 16;
  if (col >= a.cols || (a.counts && __ldg(a.counts + z) <= 0)) return;
  const uint8_t* const src = a.in + z * a.group + r * a.ld + col;
  uint8_t* const dst = a.out + (int64_t(z) * a.rows + r) * a.ld_out + col;
  const int n = min(16, a.cols - col);
  if (!DG_IN(a.dbg, src, n, DBG_QUANTIZE) || !DG_IN(a.dbg, dst, 16, DBG_QUANTIZE)) return;
  alignas(16) uint8_t b[16] = {};
  if (n == 16) {
#pragma unroll
    for (int i = 0; i < int(16 / sizeof(T)); ++i) reinterpret_cast<T*>(b)[i] = __ldg(reinterpret_cast<const T*>(src) + i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) b[i] = __ldg(src + i);
  }
  *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(b);
}

template <typename T>
cudaError_t launch_repack_type(const RepackArgs& a, cudaStream_t s) {
  const int pieces = (a.cols + 15) / 16;
  const int threads = pieces >= 256 ? 256 : (pieces + 31) / 32 * 32;
  return launch_k(repack_kernel<T>, dim3(unsigned(a.rows), unsigned((pieces + threads - 1) / threads), unsigned(a.groups)),
                  dim3(unsigned(threads)), 0, s, a.pdl, a);
}

}  // namespace

cudaError_t launch_repack(const RepackArgs& a, cudaStream_t s) {
  const uint64_t low = reinterpret_cast<uint64_t>(a.in) | uint64_t(a.ld) | uint64_t(a.groups > 1 ? a.group : 0);
  if (low % 8 == 0) return launch_repack_type<uint64_t>(a, s);
  if (low % 4 == 0) return launch_repack_type<uint32_t>(a, s);
  return launch_repack_type<uint8_t>(a, s);
}

cudaError_t launch_quantize(const QuantArgs& a, cudaStream_t s) {
  switch (a.x_kind) {
    case OUT_F32: return launch_type<float>(a, s);
    case OUT_BF16: return launch_type<__nv_bfloat16>(a, s);
    default: return launch_type<__half>(a, s);
  }
}

}  // namespace dg
