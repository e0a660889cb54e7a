// quantize_mx4.cu -- a matrix to 4 bits (E2M1) with one power-of-two scale for each block of 32 values along a
// row, as it stands and transposed; and the values of block-scaled matrices of 4 and 8 bits.
//
// For a block with largest magnitude m = f * 2^E, 1 <= f < 2, the scale is 2^e with the least e, -127 at least, that
// keeps m * 2^-e within 6 = 1.5 * 2^2: e = E - 2 + (f > 1.5), by integer arithmetic on m's bits.
// Multiplying by 2^-e is exact, so a code is one rounding (to nearest, ties to the even code) away from its value.
// E2M1 has neither infinities nor NaN: a block that holds any has the scale byte 255, which is NaN, and codes of 0.
//
// A CTA takes 128 x 128 values, which is one scale tile (128 rows x 4 blocks) in either orientation.  A half warp
// holds 128 columns of a row, a lane eight neighbouring columns of four neighbouring rows: a row's block is four
// lanes (two exchanges), a column's block 32 rows of four warps (through shared memory).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <type_traits>

#include "codes.cuh"
#include "kernels.h"

namespace dg {
namespace {

constexpr int kWarps = 16;   // 8 rows each
constexpr int kLaneRows = 4;  // rows of a lane

template <typename T>
__device__ __forceinline__ float to_f(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else return __bfloat162float(v);
}

// Scale byte (e + 127) of a block whose largest magnitude has the bits m (infinities and NaN: kInf and more).
__device__ __forceinline__ uint32_t mx4_byte(uint32_t m) {
  if (m >= kInf) return 255u;
  return uint32_t(max(int(m >> 23) - 2 + int((m & 0x7fffffu) > 0x400000u), 0));
}

// 2^-e; 0 for a block without a number, whose codes are 0.
__device__ __forceinline__ float mx4_inverse(uint32_t byte) { return byte == 255u ? 0.f : inverse_scale(byte); }

// The codes of two values times inv, the first one's in the low four bits.  (NaN would become the largest code: a
// block that holds any has inv = 0, and NaN * 0 is NaN.)
__device__ __forceinline__ uint32_t mx4_codes2(float a, float b, float inv) {
  return __nv_cvt_float2_to_fp4x2(make_float2(a * inv, b * inv), __NV_E2M1, cudaRoundNearest);
}

// Eight neighbouring values, as fp32.
template <typename T, bool VEC>
__device__ __forceinline__ void load_row(const QuantArgs& a, int src, int col, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  if (src < 0 || col >= a.cols) return;
  const T* const p = static_cast<const T*>(a.x) + int64_t(src) * a.ldx + col;
  if (VEC && col + 8 <= a.cols) {
    if (!DG_IN(a.dbg, p, 8 * int(sizeof(T)), DBG_QUANTIZE)) return;
    alignas(16) T t[8];
#pragma unroll
    for (int i = 0; i < int(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(t)[i] = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_f(t[j]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (col + j < a.cols && DG_IN(a.dbg, p + j, int(sizeof(T)), DBG_QUANTIZE)) v[j] = to_f(p[j]);
}

template <typename T, bool VEC, bool TURN>
__global__ void __launch_bounds__(32 * kWarps) quantize_mx4_kernel(const QuantArgs a) {
  __shared__ uint32_t row_bytes[128];          // the scale tile of Q, word by row
  __shared__ uint32_t col_max[TURN ? kWarps : 1][128];
  __shared__ uint8_t col_byte[TURN ? 4 : 1][128];  // [block of 32 rows][column]
  __shared__ uint16_t turn[TURN ? 128 * 32 : 1];   // [column][4 rows ^ swizzle]
  wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cb = blockIdx.x, rb = blockIdx.y;
  const int row0 = warp * 8 + (lane >> 4) * kLaneRows;  // of the tile
  const int piece = lane & 15, col = cb * 128 + piece * 8;
  float v[kLaneRows][8];
  uint32_t live = 0;
#pragma unroll
  for (int i = 0; i < kLaneRows; ++i) {
    const int src = source_row(a, rb * 128 + row0 + i);
    live |= uint32_t(src >= 0) << i;
    load_row<T, VEC>(a, src, col, v[i]);
  }
  if constexpr (TURN) {
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0;
#pragma unroll
      for (int i = 0; i < kLaneRows; ++i) m[j] = max(m[j], __float_as_uint(v[i][j]) & 0x7fffffffu);
      m[j] = max(m[j], __shfl_xor_sync(kAll, m[j], 16));
    }
    if (lane < 16) {
      *reinterpret_cast<uint4*>(&col_max[warp][piece * 8]) = make_uint4(m[0], m[1], m[2], m[3]);
      *reinterpret_cast<uint4*>(&col_max[warp][piece * 8 + 4]) = make_uint4(m[4], m[5], m[6], m[7]);
    }
  }
  if (a.q) {
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7fffffffu);
      m = max(m, __shfl_xor_sync(kAll, m, 1));
      m = max(m, __shfl_xor_sync(kAll, m, 2));
      const uint32_t byte = mx4_byte(m);
      const float inv = mx4_inverse(byte);
      uint32_t c = 0;
      if (byte != 255u)
        c = mx4_codes2(v[i][0], v[i][1], inv) | mx4_codes2(v[i][2], v[i][3], inv) << 8 | mx4_codes2(v[i][4], v[i][5], inv) << 16 |
            mx4_codes2(v[i][6], v[i][7], inv) << 24;
      // the word of four blocks, in lanes 0 and 16
      uint32_t word = byte | __shfl_down_sync(kAll, byte, 4) << 8;
      word |= __shfl_down_sync(kAll, word, 8) << 16;
      if (piece == 0) row_bytes[row0 + i] = word;
      if ((live >> i) & 1u) {
        const int n = min(4, (a.cols - col + 1) / 2);  // bytes of the row that exist
        uint8_t* const dst = a.q + int64_t(rb * 128 + row0 + i) * a.ldq + col / 2;
        if (n == 4) {
          if (DG_IN(a.dbg, dst, 4, DBG_QUANTIZE)) *reinterpret_cast<uint32_t*>(dst) = c;
        } else if (n > 0 && DG_IN(a.dbg, dst, n, DBG_QUANTIZE)) {
          for (int j = 0; j < n; ++j) dst[j] = uint8_t(c >> (8 * j));
        }
      }
    }
  }
  __syncthreads();
  if (a.q && threadIdx.x < 32) {  // line `lane` of the tile: rows lane, lane + 32, lane + 64, lane + 96
    uint8_t* const s = a.sq + (int64_t(rb) * a.q_groups + cb) * 512 + lane * 16;
    if (DG_IN(a.dbg, s, 16, DBG_QUANTIZE))
      *reinterpret_cast<uint4*>(s) = make_uint4(row_bytes[lane], row_bytes[lane + 32], row_bytes[lane + 64], row_bytes[lane + 96]);
  }
  if constexpr (TURN) {
    {  // one thread a column and block of 32 rows
      const int c = threadIdx.x & 127, b = threadIdx.x >> 7;
      const uint32_t m = max(max(col_max[4 * b][c], col_max[4 * b + 1][c]), max(col_max[4 * b + 2][c], col_max[4 * b + 3][c]));
      col_byte[b][c] = uint8_t(mx4_byte(m));
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t byte = col_byte[warp / 4][piece * 8 + j];
      const float inv = mx4_inverse(byte);
      uint32_t c = 0;
      if (byte != 255u) c = mx4_codes2(v[0][j], v[1][j], inv) | mx4_codes2(v[2][j], v[3][j], inv) << 8;
      turn[(piece * 8 + j) * 32 + ((warp * 2 + (lane >> 4)) ^ (piece * 2))] = uint16_t(c);
    }
    __syncthreads();
    {  // 16 bytes of a column: 32 rows
      const int c = threadIdx.x >> 2, part = threadIdx.x & 3, x = (c >> 3) * 2;
      const int out_row = cb * 128 + c, r = rb * 128 + part * 32;
      if (out_row < a.cols && r < a.rows) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const uint32_t*>(&turn[c * 32 + ((part * 8 + 2 * k) ^ x)]);
        uint8_t* const dst = a.qt + int64_t(out_row) * a.ldqt + r / 2;
        const int n = min(16, (a.rows - r + 1) / 2);
        if (DG_IN(a.dbg, dst, n, DBG_QUANTIZE)) {
          if (n == 16) {
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (k < n) dst[k] = uint8_t(w[k / 4] >> (8 * (k & 3)));
          }
        }
      }
    }
    if (threadIdx.x < 32) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = lane + 32 * k;
        w[k] = uint32_t(col_byte[0][c]) | uint32_t(col_byte[1][c]) << 8 | uint32_t(col_byte[2][c]) << 16 | uint32_t(col_byte[3][c]) << 24;
      }
      uint8_t* const s = a.sqt + (int64_t(cb) * a.qt_groups + rb) * 512 + lane * 16;
      if (DG_IN(a.dbg, s, 16, DBG_QUANTIZE)) *reinterpret_cast<uint4*>(s) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <typename T, bool VEC>
cudaError_t launch_mx4(const QuantArgs& a, cudaStream_t s) {
  const dim3 grid(unsigned((a.cols + 127) / 128), unsigned((a.rows + 127) / 128));
  if (a.qt) return launch_k(quantize_mx4_kernel<T, VEC, true>, grid, dim3(32 * kWarps), 0, s, a.pdl, a);
  return launch_k(quantize_mx4_kernel<T, VEC, false>, grid, dim3(32 * kWarps), 0, s, a.pdl, a);
}

template <typename T>
cudaError_t launch_mx4_type(const QuantArgs& a, cudaStream_t s) {
  return a.vec ? launch_mx4<T, true>(a, s) : launch_mx4<T, false>(a, s);
}

// ------------------------------------------------------------------ values

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23);
}

// A thread takes kPieces pieces of eight values, a warp's width of pieces apart; T: the result's type.
constexpr int kPieces = 4;

template <typename T, int CODE>
__global__ void __launch_bounds__(256) dequantize_kernel(const DequantArgs a, uint32_t pieces) {
  constexpr int BLOCK = CODE == CODE_E2M1 ? 32 : 128, BYTES = CODE == CODE_E2M1 ? 4 : 8;
  wait_prior_grid();
  uint32_t w[kPieces][2], byte[kPieces];
  int row[kPieces], col[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const uint64_t item = (uint64_t(blockIdx.x) * kPieces + i) * 256 + threadIdx.x;
    const uint64_t r = item / pieces;
    row[i] = r < uint64_t(a.rows) ? int(r) : -1;
    col[i] = int(item - r * pieces) * 8;
    w[i][0] = w[i][1] = byte[i] = 0u;
    if (row[i] < 0) continue;
    const uint8_t* const q = a.q + int64_t(row[i]) * a.ldq + int64_t(col[i]) * BYTES / 8;
    const int n = CODE == CODE_E2M1 ? min(4, (a.cols - col[i] + 1) / 2) : min(8, a.cols - col[i]);
    if (DG_IN(a.dbg, q, n, DBG_QUANTIZE)) {
      if (n == BYTES) {
        if constexpr (BYTES == 4) {
          w[i][0] = *reinterpret_cast<const uint32_t*>(q);
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(q);
          w[i][0] = u.x, w[i][1] = u.y;
        }
      } else {
        for (int j = 0; j < n; ++j) w[i][j / 4] |= uint32_t(q[j]) << (8 * (j & 3));
      }
    }
    const uint8_t* const s = a.sq + scale_at(row[i], col[i] / BLOCK, a.groups);
    if (DG_IN(a.dbg, s, 1, DBG_QUANTIZE)) byte[i] = *s;
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    if (row[i] < 0) continue;
    const float by = scale_value(byte[i]);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      __half2_raw h;
      if constexpr (CODE == CODE_E2M1) {
        h = __nv_cvt_fp4x2_to_halfraw2(__nv_fp4x2_storage_t(w[i][0] >> (4 * j)), __NV_E2M1);
      } else {
        h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w[i][j / 4] >> (8 * (j & 3))), CODE == CODE_E5M2 ? __NV_E5M2 : __NV_E4M3);
      }
      const float2 f = __half22float2(__half2(h));
      v[j] = f.x * by, v[j + 1] = f.y * by;
    }
    T* const dst = static_cast<T*>(a.x) + int64_t(row[i]) * a.ldx + col[i];
    const int n = min(8, a.cols - col[i]);
    alignas(16) T t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (sizeof(T) == 4) t[j] = v[j];
      else if constexpr (std::is_same<T, __half>::value) t[j] = __float2half_rn(v[j]);
      else t[j] = __float2bfloat16_rn(v[j]);
    }
    if (!DG_IN(a.dbg, dst, n * int(sizeof(T)), DBG_QUANTIZE)) continue;
    if (n == 8 && a.wide) {
#pragma unroll
      for (int k = 0; k < int(sizeof(T)) / 2; ++k) reinterpret_cast<uint4*>(dst)[k] = reinterpret_cast<const uint4*>(t)[k];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) dst[j] = t[j];
    }
  }
}

template <typename T>
cudaError_t launch_values(const DequantArgs& a, cudaStream_t s) {
  const uint32_t pieces = uint32_t((a.cols + 7) / 8);
  const uint64_t items = uint64_t(a.rows) * pieces;
  const dim3 grid(unsigned((items + 256 * kPieces - 1) / (256 * kPieces)));
  switch (a.code) {
    case CODE_E4M3: return launch_k(dequantize_kernel<T, CODE_E4M3>, grid, dim3(256), 0, s, a.pdl, a, pieces);
    case CODE_E5M2: return launch_k(dequantize_kernel<T, CODE_E5M2>, grid, dim3(256), 0, s, a.pdl, a, pieces);
    default: return launch_k(dequantize_kernel<T, CODE_E2M1>, grid, dim3(256), 0, s, a.pdl, a, pieces);
  }
}

}  // namespace

cudaError_t launch_quantize_mx4(const QuantArgs& a, cudaStream_t s) {
  switch (a.x_kind) {
    case OUT_F32: return launch_mx4_type<float>(a, s);
    case OUT_BF16: return launch_mx4_type<__nv_bfloat16>(a, s);
    default: return launch_mx4_type<__half>(a, s);
  }
}

cudaError_t launch_dequantize(const DequantArgs& a, cudaStream_t s) {
  switch (a.x_kind) {
    case OUT_F32: return launch_values<float>(a, s);
    case OUT_BF16: return launch_values<__nv_bfloat16>(a, s);
    default: return launch_values<__half>(a, s);
  }
}

}  // namespace dg
