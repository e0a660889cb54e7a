// quantize_mx4.cu -- a matrix to 4 bits (E2M1) with one power-of-two scale for each block of 32 values along a
// row, as it stands and transposed; and the values of block-scaled matrices of 4 and 8 bits.
//
// For a block with largest magnitude m = f * 2^E, 1 <= f < 2, the scale is 2^e with the least e, -127 at least, that
// keeps m * 2^-e within 6 = 1.5 * 2^2: e = E - 2 + (f > 1.5), by integer arithmetic on m's bits.
// Multiplying by 2^-e is exact, so a code is one rounding (to nearest, ties to the even code) away from its value.
// E2M1 has neither infinities nor NaN: a block that holds any has the scale byte 255, which is NaN, and codes of 0.
//
// One orientation: warps take rows, no barrier.  Both: a CTA takes 128 x 128 values, which is one scale tile (128 rows x
// 4 blocks) in either orientation; half a warp holds 128 columns of a row, a lane eight neighbouring columns of four
// neighbouring rows.  A row's block is four lanes (two exchanges), a column's block 32 rows of four warps (through shared memory).
// What bounds it is issuing instructions: 8192 x 4096 bf16 19 us one way (85 MB, 4.4 TB/s), 28 both (103 MB), where a thread spends ~22
// instructions a value; back to bf16 14.6 us (85 MB, 5.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "codes.cuh"
#include "kernels.h"

namespace dg {
namespace {

constexpr int kWarps = 16;   // 8 rows each
constexpr int kLaneRows = 4;  // rows of a lane

// Scale byte (e + 127) of a block whose largest magnitude has the bits m (infinities and NaN: kInf and more).
__device__ __forceinline__ uint32_t mx4_byte(uint32_t m) {
  if (m >= kInf) return 255u;
  return uint32_t(max(int(m >> 23) - 2 + int((m & 0x7fffffu) > 0x400000u), 0));
}

// 2^-e; 0 for a block without a number, whose codes are 0.
__device__ __forceinline__ float mx4_inverse(uint32_t byte) { return byte == 255u ? 0.f : inverse_scale(byte); }

// The codes of eight values, the first one's in the low four bits.  (cvt rounds to nearest, ties to the even code, and
// takes its second value for the low half.)
__device__ __forceinline__ uint32_t mx4_codes8(float a, float b, float c, float d, float e, float f, float g, float h) {
  uint32_t out;
  asm("{\n\t.reg .b8 p, q, r, s;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\t"
      "mov.b32 %0, {p, q, r, s};\n\t}"
      : "=r"(out)
      : "f"(a), "f"(b), "f"(c), "f"(d), "f"(e), "f"(f), "f"(g), "f"(h));
  return out;
}

// The values of eight codes, two to a word of fp16.
__device__ __forceinline__ void mx4_values8(uint32_t codes, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 p, q, r, s;\n\t"
      "mov.b32 {p, q, r, s}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, q;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, r;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, s;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(codes));
}

// Eight neighbouring values as they are loaded: 16-bit types two to a word, whose magnitudes' bits are ordered like
// the numbers, so that maxima are taken on words.
template <typename T>
struct Row8 {
  static constexpr int WORDS = int(sizeof(T)) * 2;
  uint32_t w[WORDS];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (std::is_same<T, __half>::value) {
      const uint16_t h = uint16_t(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
      return __half2float(*reinterpret_cast<const __half*>(&h));
    } else {
      return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
  }
  __device__ __forceinline__ void load(const QuantArgs& a, int src, int col, bool vec) {
#pragma unroll
    for (int j = 0; j < WORDS; ++j) w[j] = 0u;
    if (src < 0 || col >= a.cols) return;
    const T* const p = static_cast<const T*>(a.x) + int64_t(src) * a.ldx + col;
    if (vec && col + 8 <= a.cols) {
      if (!DG_IN(a.dbg, p, 8 * int(sizeof(T)), DBG_QUANTIZE)) return;
#pragma unroll
      for (int i = 0; i < WORDS / 4; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
      return;
    }
    const int n = min(8, a.cols - col);
    if (!DG_IN(a.dbg, p, n * int(sizeof(T)), DBG_QUANTIZE)) return;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) w[j] = reinterpret_cast<const uint32_t*>(p)[j];
    } else if (a.x_words) {  // words, and the last value of an odd number
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (2 * j + 1 < n)
          w[j] = reinterpret_cast<const uint32_t*>(p)[j];
        else if (2 * j < n)
          w[j] = reinterpret_cast<const uint16_t*>(p)[2 * j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) w[j / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[j]) << (16 * (j & 1));
    }
  }
};

// A word's magnitudes, and the larger ones of two words' (16-bit types two each; NaN wins: its bits are the largest).
template <typename T>
__device__ __forceinline__ uint32_t magnitude(uint32_t x) {
  return x & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu);
}
template <typename T>
__device__ __forceinline__ uint32_t most(uint32_t x, uint32_t y) {
  if constexpr (sizeof(T) == 4) return max(x, y);
  else return __vmaxu2(x, y);
}

// Scale byte of a magnitude's bits in the input's type.
template <typename T>
__device__ __forceinline__ uint32_t byte_of(uint32_t bits) {
  if constexpr (sizeof(T) == 4) return mx4_byte(bits);
  else if constexpr (std::is_same<T, __half>::value) {
    const uint16_t h = uint16_t(bits);
    return mx4_byte(__float_as_uint(__half2float(*reinterpret_cast<const __half*>(&h))));
  } else {
    return mx4_byte(bits << 16);
  }
}

// Scale byte of a row's block of 32: the magnitudes of four lanes' eight values.
template <typename T>
__device__ __forceinline__ uint32_t row_byte(const Row8<T>& v) {
  uint32_t m = magnitude<T>(v.w[0]);
#pragma unroll
  for (int j = 1; j < Row8<T>::WORDS; ++j) m = most<T>(m, magnitude<T>(v.w[j]));
  m = most<T>(m, __shfl_xor_sync(kAll, m, 1));
  m = most<T>(m, __shfl_xor_sync(kAll, m, 2));
  if constexpr (sizeof(T) == 2) m = max(m >> 16, m & 0xffffu);
  return byte_of<T>(m);
}

// A word's two bf16 values times those of another word.  By a power of two that is exact, but for results below bf16's
// least normal number, which are codes of 0 either way; and bf16 has fp32's exponents, so that every 2^-e is one.
__device__ __forceinline__ uint32_t times2(uint32_t w, uint32_t by) {
  const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&by));
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Codes of a row's eight values; a block without a number has codes of 0.
template <typename T>
__device__ __forceinline__ uint32_t row_codes(uint32_t byte, const Row8<T>& v) {
  const float inv = mx4_inverse(byte);
  uint32_t codes;
  if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const uint32_t by = __byte_perm(__float_as_uint(inv), 0u, 0x3232);
    const uint32_t a = times2(v.w[0], by), b = times2(v.w[1], by), c = times2(v.w[2], by), d = times2(v.w[3], by);
    codes = mx4_codes8(low(a), high(a), low(b), high(b), low(c), high(c), low(d), high(d));
  } else {
    codes = mx4_codes8(v.at(0) * inv, v.at(1) * inv, v.at(2) * inv, v.at(3) * inv, v.at(4) * inv, v.at(5) * inv, v.at(6) * inv,
                       v.at(7) * inv);
  }
  return byte == 255u ? 0u : codes;
}

// `n` bytes of a word, or all four: as a word where rows allow it.
__device__ __forceinline__ void store_codes(const QuantArgs& a, uint8_t* dst, uint32_t c, int n) {
  if (n >= 4 && a.q_wide) {
    if (DG_IN(a.dbg, dst, 4, DBG_QUANTIZE)) *reinterpret_cast<uint32_t*>(dst) = c;
  } else if (n > 0 && DG_IN(a.dbg, dst, min(n, 4), DBG_QUANTIZE)) {
    for (int j = 0; j < min(n, 4); ++j) dst[j] = uint8_t(c >> (8 * j));
  }
}

// One orientation: a warp takes kRowRows rows of 512 columns, all its loads in flight together; a word of four
// scale bytes is half a warp's.
constexpr int kRowRows = 2;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_mx4_rows_kernel(const QuantArgs a, uint32_t chunks) {
  wait_prior_grid();
  const int lane = threadIdx.x & 31, piece = lane & 15;
  const uint32_t warp = uint32_t((uint64_t(blockIdx.x) * 256 + threadIdx.x) >> 5);
  const int r0 = int(warp / chunks) * kRowRows, c0 = int(warp % chunks) * 512 + 8 * lane;
  if (r0 >= a.rows_padded) return;
  Row8<T> v[kRowRows][2];
  int src[kRowRows];
  source_rows(a, r0, src);
#pragma unroll
  for (int i = 0; i < kRowRows; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) v[i][h].load(a, src[i], c0 + 256 * h, VEC);
#pragma unroll
  for (int i = 0; i < kRowRows; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = c0 + 256 * h;
      const Row8<T>& x = v[i][h];
      const uint32_t byte = row_byte<T>(x);
      const uint32_t c = row_codes(byte, x);
      uint32_t word = byte | __shfl_down_sync(kAll, byte, 4) << 8;
      word |= __shfl_down_sync(kAll, word, 8) << 16;
      if (src[i] >= 0) store_codes(a, a.q + int64_t(r0 + i) * a.ldq + col / 2, c, (a.cols - col + 1) / 2);
      if (piece == 0 && col / 128 < a.q_groups) {
        uint8_t* const s = a.sq + scale_at(r0 + i, col / 32, a.q_groups);
        if (DG_IN(a.dbg, s, 4, DBG_QUANTIZE)) *reinterpret_cast<uint32_t*>(s) = word;
      }
    }
}

// 16 bytes from global to shared memory, complete for the thread that asked after copies_wait().
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Rows of X that this lane's rows of a tile come from: half a warp's kLaneRows of the warp's eight from r0 on.  (Without a map there is
// nothing to exchange.)
__device__ __forceinline__ void lane_rows(const QuantArgs& a, int r0, int (&src)[kLaneRows]) {
  const bool lower = (threadIdx.x & 31) < 16;
  if (a.rowmap) {
    int all[2 * kLaneRows];
    source_rows(a, r0, all);
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) src[i] = lower ? all[i] : all[i + kLaneRows];
  } else {
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) {
      const int r = r0 + (lower ? i : i + kLaneRows);
      src[i] = r < a.rows ? r : -1;
    }
  }
}

// Both orientations, or the transposed one.  AHEAD (16-bit types by 16 bytes): a CTA takes one tile after another, and the next tile's
// values are copied to shared memory, where each thread reads its own again, while it works on one.
template <typename T, bool VEC, bool AHEAD>
__global__ void __launch_bounds__(32 * kWarps, 2) quantize_mx4_kernel(const QuantArgs a) {
  constexpr int COLS = 8 / (sizeof(T) == 4 ? 1 : 2);  // words of maxima of a lane's eight columns
  static_assert(!AHEAD || (VEC && sizeof(T) == 2), "copies of eight values are 16 bytes");
  __shared__ uint32_t row_bytes[128];          // the scale tile of Q, word by row
  alignas(16) __shared__ uint32_t col_max[kWarps][16 * COLS];
  __shared__ uint8_t col_byte[4][128];         // [block of 32 rows][column]
  __shared__ uint16_t turn[128 * 32];          // [column][4 rows ^ swizzle]
  __shared__ uint4 ahead[AHEAD ? kLaneRows * 32 * kWarps : 1];  // [row of a lane][thread]
  wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row0 = warp * 8 + (lane >> 4) * kLaneRows;  // of the tile
  const int piece = lane & 15;
  const int col_blocks = (a.cols + 127) / 128, row_blocks = (a.rows + 127) / 128;
  int cb = blockIdx.x, rb = blockIdx.y, step_c = 0, step_r = 0;
  if constexpr (AHEAD) {  // (one row of CTAs, no more than there are tiles)
    rb = int(blockIdx.x / unsigned(col_blocks)), cb = int(blockIdx.x % unsigned(col_blocks));
    step_r = int(gridDim.x / unsigned(col_blocks)), step_c = int(gridDim.x % unsigned(col_blocks));
  }
  // The tile's rows of this lane that exist, whose values are on their way (of whole eights; the others are loaded when it
  // is the tile's turn).
  auto fetch = [&](int c, int r) {
    int src[kLaneRows];
    lane_rows(a, r * 128 + warp * 8, src);
    uint32_t rows = 0;
    const int at = c * 128 + piece * 8;
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) {
      rows |= uint32_t(src[i] >= 0) << i;
      const T* const p = static_cast<const T*>(a.x) + int64_t(src[i]) * a.ldx + at;
      if (src[i] >= 0 && at + 8 <= a.cols && DG_IN(a.dbg, p, 16, DBG_QUANTIZE)) copy16(&ahead[i * 32 * kWarps + threadIdx.x], p);
    }
    return rows;
  };
  uint32_t live = 0;
  if constexpr (AHEAD) live = fetch(cb, rb);
  do {
    const int col = cb * 128 + piece * 8;
    Row8<T> v[kLaneRows];
    if constexpr (AHEAD) {
      copies_wait();
#pragma unroll
      for (int i = 0; i < kLaneRows; ++i) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (((live >> i) & 1u) && col + 8 <= a.cols) w = ahead[i * 32 * kWarps + threadIdx.x];
        v[i].w[0] = w.x, v[i].w[1] = w.y, v[i].w[2] = w.z, v[i].w[3] = w.w;
      }
    }
    if (!AHEAD || __any_sync(kAll, col < a.cols && col + 8 > a.cols)) {
      int src[kLaneRows];
      lane_rows(a, rb * 128 + warp * 8, src);
      if (!AHEAD) live = 0;
#pragma unroll
      for (int i = 0; i < kLaneRows; ++i) {
        if (!AHEAD) live |= uint32_t(src[i] >= 0) << i;
        if (!AHEAD || col + 8 > a.cols) v[i].load(a, src[i], col, VEC && !AHEAD);
      }
    }
    {
      uint32_t m[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) {
        m[j] = magnitude<T>(v[0].w[j]);
#pragma unroll
        for (int i = 1; i < kLaneRows; ++i) m[j] = most<T>(m[j], magnitude<T>(v[i].w[j]));
        m[j] = most<T>(m[j], __shfl_xor_sync(kAll, m[j], 16));
      }
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < COLS; j += 4)
          *reinterpret_cast<uint4*>(&col_max[warp][piece * COLS + j]) = make_uint4(m[j], m[j + 1], m[j + 2], m[j + 3]);
      }
    }
    if (a.q) {
#pragma unroll
      for (int i = 0; i < kLaneRows; ++i) {
        const uint32_t byte = row_byte<T>(v[i]);
        const uint32_t c = row_codes(byte, v[i]);
        if ((piece & 3) == 0) reinterpret_cast<uint8_t*>(row_bytes + row0 + i)[piece >> 2] = uint8_t(byte);
        if ((live >> i) & 1u) store_codes(a, a.q + int64_t(rb * 128 + row0 + i) * a.ldq + col / 2, c, (a.cols - col + 1) / 2);
      }
    }
    __syncthreads();
    int next_c = cb + step_c, next_r = rb + step_r;
    if constexpr (AHEAD) {
      if (next_c >= col_blocks) next_c -= col_blocks, ++next_r;
      if (next_r < row_blocks) live = fetch(next_c, next_r);
    }
    if (a.q && threadIdx.x < 32) {  // line `lane` of the tile: rows lane, lane + 32, lane + 64, lane + 96
      uint8_t* const s = a.sq + (int64_t(rb) * a.q_groups + cb) * 512 + lane * 16;
      if (DG_IN(a.dbg, s, 16, DBG_QUANTIZE))
        *reinterpret_cast<uint4*>(s) = make_uint4(row_bytes[lane], row_bytes[lane + 32], row_bytes[lane + 64], row_bytes[lane + 96]);
    }
    if (threadIdx.x < 64 * COLS) {  // one thread a word of columns and block of 32 rows
      const int c = threadIdx.x % (16 * COLS), b = threadIdx.x / (16 * COLS);
      const uint32_t m = most<T>(most<T>(col_max[4 * b][c], col_max[4 * b + 1][c]), most<T>(col_max[4 * b + 2][c], col_max[4 * b + 3][c]));
      if constexpr (sizeof(T) == 4)
        col_byte[b][c] = uint8_t(byte_of<T>(m));
      else
        *reinterpret_cast<uint16_t*>(&col_byte[b][2 * c]) = uint16_t(byte_of<T>(m & 0xffffu) | byte_of<T>(m >> 16) << 8);
    }
    __syncthreads();
    {
      const uint2 bytes = *reinterpret_cast<const uint2*>(&col_byte[warp / 4][piece * 8]);
      uint16_t* const to = turn + piece * 8 * 32 + ((warp * 2 + (lane >> 4)) ^ (piece * 2));
#pragma unroll
      for (int j = 0; j < 8; j += 2) {  // two columns at a time
        const uint32_t b0 = ((j < 4 ? bytes.x : bytes.y) >> (8 * (j & 3))) & 0xffu, b1 = ((j < 4 ? bytes.x : bytes.y) >> (8 * (j & 3) + 8)) & 0xffu;
        const float i0 = mx4_inverse(b0), i1 = mx4_inverse(b1);
        uint32_t c;
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          const uint32_t by = __byte_perm(__float_as_uint(i0), __float_as_uint(i1), 0x7632);
          const uint32_t p = times2(v[0].w[j / 2], by), q = times2(v[1].w[j / 2], by), r = times2(v[2].w[j / 2], by),
                         s = times2(v[3].w[j / 2], by);
          c = mx4_codes8(low(p), low(q), low(r), low(s), high(p), high(q), high(r), high(s));
        } else {
          c = mx4_codes8(v[0].at(j) * i0, v[1].at(j) * i0, v[2].at(j) * i0, v[3].at(j) * i0, v[0].at(j + 1) * i1,
                         v[1].at(j + 1) * i1, v[2].at(j + 1) * i1, v[3].at(j + 1) * i1);
        }
        to[j * 32] = uint16_t(b0 == 255u ? 0u : c);
        to[(j + 1) * 32] = uint16_t(b1 == 255u ? 0u : c >> 16);
      }
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
          if (n == 16 && a.qt_wide) {
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
    cb = next_c, rb = next_r;
  } while (AHEAD && rb < row_blocks);
}

template <typename T, bool VEC>
cudaError_t launch_mx4(const QuantArgs& a, int sms, cudaStream_t s) {
  if (!a.qt) {
    const uint32_t chunks = uint32_t((a.cols + 511) / 512);
    const int64_t warps = int64_t(a.rows_padded / kRowRows) * chunks;
    return launch_k(quantize_mx4_rows_kernel<T, VEC>, dim3(unsigned((warps + 7) / 8)), dim3(256), 0, s, a.pdl, a, chunks);
  }
  const dim3 tiles(unsigned((a.cols + 127) / 128), unsigned((a.rows + 127) / 128));
  // Tiles one after another once there are more than run at the same time (8192 x 4096 bf16, both orientations: 29.3 us, each tile a CTA of its
  // own 30.9; transposed alone 20.1 and 24.6; 1024 x 4096 5.2 and 4.9; fp32, without the copies ahead, 37.6 and 34.6).
  if constexpr (VEC && sizeof(T) == 2) {
    if (int64_t(tiles.x) * tiles.y > 2 * sms) return launch_k(quantize_mx4_kernel<T, true, true>, dim3(unsigned(2 * sms)), dim3(32 * kWarps), 0, s, a.pdl, a);
  }
  return launch_k(quantize_mx4_kernel<T, VEC, false>, tiles, dim3(32 * kWarps), 0, s, a.pdl, a);
}

template <typename T>
cudaError_t launch_mx4_type(const QuantArgs& a, int sms, cudaStream_t s) {
  return a.vec ? launch_mx4<T, true>(a, sms, s) : launch_mx4<T, false>(a, sms, s);
}

// ------------------------------------------------------------------ values

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23);
}

// Eight values from their codes (one word of 4-bit ones, two of 8-bit ones) and their scale.
template <int CODE>
__device__ __forceinline__ void code_values(uint32_t w0, uint32_t w1, float by, float (&v)[8]) {
  uint32_t pairs[4];  // fp16, which holds every code's value
  if constexpr (CODE == CODE_E2M1) {
    mx4_values8(w0, pairs);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t((j < 2 ? w0 : w1) >> (16 * (j & 1))),
                                                       CODE == CODE_E5M2 ? __NV_E5M2 : __NV_E4M3);
      pairs[j] = uint32_t(h.x) | uint32_t(h.y) << 16;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&pairs[j]));
    v[2 * j] = f.x * by, v[2 * j + 1] = f.y * by;
  }
}

// A warp takes kValueRows rows of 512 columns, a lane twice eight neighbouring ones: rows' addresses are worked out once, and
// the second eight's codes, scale and result are a constant further on.  T: the result's type.  (Pieces of eight wherever
// they fell, each with its own addresses: 8192 x 4096 to bf16 from 4 bits 17.2 us.)
constexpr int kValueRows = 2;

template <typename T, int CODE>
__global__ void __launch_bounds__(256) dequantize_kernel(const DequantArgs a, uint32_t chunks) {
  constexpr int BLOCK = CODE == CODE_E2M1 ? 32 : 128, BYTES = CODE == CODE_E2M1 ? 4 : 8;
  constexpr int NEXT_SCALE = CODE == CODE_E2M1 ? 1024 : 2;  // bytes from a block's scale to that of the block 256 columns on
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const uint64_t warp = uint64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const uint64_t pair = warp >> 32 ? warp / chunks : uint64_t(uint32_t(warp) / chunks);
  const int r0 = int(pair) * kValueRows, c0 = int(warp - pair * chunks) * 512 + 8 * lane;
  if (pair * kValueRows >= uint64_t(a.rows)) return;
  uint32_t w[kValueRows][2][2], byte[kValueRows][2];
#pragma unroll
  for (int i = 0; i < kValueRows; ++i) {
    const uint8_t* const q = a.q + int64_t(r0 + i) * a.ldq + int64_t(c0) * BYTES / 8;
    const uint8_t* const s = a.sq + scale_at(r0 + i, c0 / BLOCK, a.groups);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[i][h][0] = w[i][h][1] = byte[i][h] = 0u;
      const int left = r0 + i < a.rows ? a.cols - c0 - 256 * h : 0;
      const uint8_t* const p = q + 256 * h * BYTES / 8;
      if (left >= 8 && a.q_wide) {
        if (DG_IN(a.dbg, p, BYTES, DBG_QUANTIZE)) {
          if constexpr (BYTES == 8) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[i][h][0] = u.x, w[i][h][1] = u.y;
          } else {
            w[i][h][0] = *reinterpret_cast<const uint32_t*>(p);
          }
        }
      } else if (left > 0) {
        const int n = min(BYTES, CODE == CODE_E2M1 ? (left + 1) / 2 : left);
        if (DG_IN(a.dbg, p, n, DBG_QUANTIZE)) {
#pragma unroll
          for (int j = 0; j < BYTES; ++j)
            if (j < n) w[i][h][j / 4] |= uint32_t(p[j]) << (8 * (j & 3));
        }
      }
      if (left > 0 && DG_IN(a.dbg, s + NEXT_SCALE * h, 1, DBG_QUANTIZE)) byte[i][h] = s[NEXT_SCALE * h];
    }
  }
#pragma unroll
  for (int i = 0; i < kValueRows; ++i) {
    T* const x = static_cast<T*>(a.x) + int64_t(r0 + i) * a.ldx + c0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int left = r0 + i < a.rows ? a.cols - c0 - 256 * h : 0;
      if (left <= 0) continue;
      T* const dst = x + 256 * h;
      float v[8];
      code_values<CODE>(w[i][h][0], w[i][h][1], scale_value(byte[i][h]), v);
      alignas(16) T t[8];
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        if constexpr (sizeof(T) == 4)
          t[j] = v[j], t[j + 1] = v[j + 1];
        else if constexpr (std::is_same<T, __half>::value)
          *reinterpret_cast<__half2*>(t + j) = __floats2half2_rn(v[j], v[j + 1]);
        else
          *reinterpret_cast<__nv_bfloat162*>(t + j) = __floats2bfloat162_rn(v[j], v[j + 1]);
      }
      if (!DG_IN(a.dbg, dst, min(8, left) * int(sizeof(T)), DBG_QUANTIZE)) continue;
      if (left >= 8 && a.wide) {
#pragma unroll
        for (int k = 0; k < int(sizeof(T)) / 2; ++k) reinterpret_cast<uint4*>(dst)[k] = reinterpret_cast<const uint4*>(t)[k];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) dst[j] = t[j];
      }
    }
  }
}

template <typename T>
cudaError_t launch_values(const DequantArgs& a, cudaStream_t s) {
  const uint32_t chunks = uint32_t((a.cols + 511) / 512);
  const uint64_t warps = uint64_t((a.rows + kValueRows - 1) / kValueRows) * chunks;
  const dim3 grid(unsigned((warps + 7) / 8));
  switch (a.code) {
    case CODE_E4M3: return launch_k(dequantize_kernel<T, CODE_E4M3>, grid, dim3(256), 0, s, a.pdl, a, chunks);
    case CODE_E5M2: return launch_k(dequantize_kernel<T, CODE_E5M2>, grid, dim3(256), 0, s, a.pdl, a, chunks);
    default: return launch_k(dequantize_kernel<T, CODE_E2M1>, grid, dim3(256), 0, s, a.pdl, a, chunks);
  }
}

}  // namespace

cudaError_t launch_quantize_mx4(const QuantArgs& a, int sms, cudaStream_t s) {
  switch (a.x_kind) {
    case OUT_F32: return launch_mx4_type<float>(a, sms, s);
    case OUT_BF16: return launch_mx4_type<__nv_bfloat16>(a, sms, s);
    default: return launch_mx4_type<__half>(a, sms, s);
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
