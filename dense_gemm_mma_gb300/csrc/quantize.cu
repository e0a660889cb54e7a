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
// Each value is read once, and written once per orientation; what bounds it is latency and issue more than memory.
// Maxima are taken on the magnitudes' bits (ordered like the numbers),
// one warp reduction per row and block.  8192 x 4096 bf16: one orientation 19.5 us (5.2 TB/s), both 29.7
// us (4.5 TB/s; the columns' scales need the whole tile before the first transposed code).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "kernels.h"

namespace dg {
namespace {

constexpr uint32_t kAll = 0xffffffffu;

// Four consecutive values of a row as they are loaded.
template <typename T>
struct Four;
template <>
struct Four<float> {
  uint4 w;
  __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const float* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void put(int i, float v) { (&w.x)[i] = __float_as_uint(v); }
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w); }
};
// 16-bit types: a magnitude's bits are ordered like the number, two to a register.
template <typename T>
struct Four {
  uint2 w;
  __device__ __forceinline__ void clear() { w = make_uint2(0, 0); }
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void put(int i, T v) {
    const uint32_t b = *reinterpret_cast<const uint16_t*>(&v);
    uint32_t& r = i < 2 ? w.x : w.y;
    r = i & 1 ? (r & 0xffffu) | b << 16 : (r & 0xffff0000u) | b;
  }
  __device__ __forceinline__ float at(int i) const {
    const uint32_t r = i < 2 ? w.x : w.y;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(i & 1 ? r & 0xffff0000u : r << 16);
    const uint16_t h = uint16_t(i & 1 ? r >> 16 : r);
    return __half2float(*reinterpret_cast<const __half*>(&h));
  }
};

// Largest magnitudes: of a row's four values, and column by column of several rows; as
// fp32 bits at the end.  Infinities and NaN come out as bits of at least kInf.
constexpr uint32_t kInf = 0x7f800000u;

template <typename T>
struct Peak {  // 16-bit types: columns 0-1 and 2-3 of a lane
  using Pair = typename std::conditional<std::is_same<T, __nv_bfloat16>::value, __nv_bfloat162, __half2>::type;
  uint32_t a = 0, b = 0;
  // (NaN wins and stays: its bits are past kInf)
  static __device__ __forceinline__ uint32_t most(uint32_t x, uint32_t y) {
    const Pair m = __hmax2_nan(*reinterpret_cast<const Pair*>(&x), *reinterpret_cast<const Pair*>(&y));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  __device__ __forceinline__ void take(const Four<T>& f) {
    a = most(a, f.w.x & 0x7fff7fffu);
    b = most(b, f.w.y & 0x7fff7fffu);
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t h) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return h << 16;
    const uint16_t u = uint16_t(h);
    return __float_as_uint(__half2float(*reinterpret_cast<const __half*>(&u)));
  }
  __device__ __forceinline__ uint32_t column(int j) const {
    const uint32_t r = j < 2 ? a : b;
    return bits(j & 1 ? r >> 16 : r & 0xffffu);
  }
  __device__ __forceinline__ uint32_t row() const {
    const uint32_t m = most(a, b);
    return bits(max(m >> 16, m & 0xffffu));
  }
};
template <>
struct Peak<float> {
  uint32_t m[4] = {0, 0, 0, 0};
  __device__ __forceinline__ void take(const Four<float>& f) {
    m[0] = max(m[0], f.w.x & 0x7fffffffu), m[1] = max(m[1], f.w.y & 0x7fffffffu);
    m[2] = max(m[2], f.w.z & 0x7fffffffu), m[3] = max(m[3], f.w.w & 0x7fffffffu);
  }
  __device__ __forceinline__ uint32_t column(int j) const { return m[j]; }
  __device__ __forceinline__ uint32_t row() const { return max(max(m[0], m[1]), max(m[2], m[3])); }
};

// |v|'s bits, 0 for infinities and NaN.
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < kInf ? b : 0u;
}

// Scale byte (e + 127) of a block whose largest magnitude has the bits m.
template <bool E5M2>
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  const int b = int(m >> 23) - (E5M2 ? 15 : 8) + int((m & 0x7fffffu) > 0x600000u);
  return uint32_t(max(b, 0));
}

__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Codes of two values times inv.  NaN converts to NaN; infinities would saturate, so that
// where a tile holds any (CAREFUL) they are made NaN first.
template <bool E5M2, bool CAREFUL>
__device__ __forceinline__ uint32_t codes2(float a, float b, float inv) {
  if constexpr (CAREFUL) {
    const float nan = __uint_as_float(0x7fc00000u);
    if (!(fabsf(a) < __uint_as_float(kInf))) a = nan;
    if (!(fabsf(b) < __uint_as_float(kInf))) b = nan;
  }
  return __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, E5M2 ? __NV_E5M2 : __NV_E4M3);
}

template <bool E5M2, bool CAREFUL>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  return codes2<E5M2, CAREFUL>(a, b, inv) | codes2<E5M2, CAREFUL>(c, d, inv) << 16;
}

// Byte of row r, block c in the packed scales of a matrix with `groups` groups of four blocks.
__device__ __forceinline__ int64_t scale_at(int64_t r, int64_t c, int64_t groups) {
  return ((r >> 7) * groups + (c >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (c & 3);
}

// Row of X that row r of the result comes from, -1 for none.
__device__ __forceinline__ int source_row(const QuantArgs& a, int r) {
  if (r >= a.rows) return -1;
  if (!a.rowmap) return r;
  if (!DG_IN(a.dbg, a.rowmap + r, 4, DBG_QUANTIZE)) return -1;
  int src = __ldg(a.rowmap + r);
  if (src >= 0) src /= a.map_div;
  return src < a.src_rows ? src : -1;
}

// The same of rows r0 .. r0 + N, each looked up by one lane; by a whole warp.  (Every lane looking all of
// them up: 4096 tokens to 4 of 32 experts, 2048 bf16, both ways: 43.3 us, so 34.6.)
template <int N>
__device__ __forceinline__ void source_rows(const QuantArgs& a, int r0, int (&src)[N]) {
  const int lane = threadIdx.x & 31;
  const int mine = lane < N ? source_row(a, r0 + lane) : -1;
#pragma unroll
  for (int i = 0; i < N; ++i) src[i] = __shfl_sync(kAll, mine, i);
}

// n rows' groups of four columns, from `col` on: whole groups as one load each (VEC: rows
// allow it) without a branch between them, so that all are in flight together; then the
// columns of a group that reaches past the matrix, one by one.
template <typename T, bool VEC, int N>
__device__ __forceinline__ void load_rows(Four<T> (&f)[N], const QuantArgs& a, const int (&src)[N], int col) {
  const T* const x = static_cast<const T*>(a.x) + col;
  const int n = min(4, a.cols - col);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f[i].clear();
    const T* const p = x + int64_t(src[i]) * a.ldx;
    if (VEC && n == 4 && src[i] >= 0 && DG_IN(a.dbg, p, 4 * int(sizeof(T)), DBG_QUANTIZE)) f[i].load(p);
  }
  if (n > 0 && (!VEC || n < 4)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const T* const p = x + int64_t(src[i]) * a.ldx;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (src[i] >= 0 && j < n && DG_IN(a.dbg, p + j, int(sizeof(T)), DBG_QUANTIZE)) f[i].put(j, p[j]);
    }
  }
}

__device__ __forceinline__ void store4(const QuantArgs& a, uint8_t* dst, uint32_t c, int n) {
  if (n <= 0 || !DG_IN(a.dbg, dst, n < 4 ? n : 4, DBG_QUANTIZE)) return;
  if (n >= 4)
    *reinterpret_cast<uint32_t*>(dst) = c;
  else
    for (int t = 0; t < n; ++t) dst[t] = uint8_t(c >> (8 * t));
}

// One orientation, a scale for each row's block: a warp takes kRows rows of 512
// columns (one word of scale bytes each), all its loads in flight together.
constexpr int kRows = 2;

template <typename T, bool E5M2, bool VEC>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantArgs a) {
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const uint32_t warp = uint32_t((uint64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5);
  const uint32_t groups = uint32_t(a.q_groups);
  const int r0 = int(warp / groups) * kRows;
  const int g = int(warp % groups);
  if (r0 >= a.rows_padded) return;
  Four<T> f[4][kRows];
  int src[kRows];
  source_rows(a, r0, src);
#pragma unroll
  for (int b = 0; b < 4; ++b) load_rows<T, VEC>(f[b], a, src, g * 512 + b * 128 + 4 * lane);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    uint32_t word = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const Four<T>& v = f[b][i];
      Peak<T> peak;
      peak.take(v);
      uint32_t m = __reduce_max_sync(kAll, peak.row());
      const bool careful = m >= kInf;
      if (careful)
        m = __reduce_max_sync(kAll, max(max(finite_bits(v.at(0)), finite_bits(v.at(1))),
                                        max(finite_bits(v.at(2)), finite_bits(v.at(3)))));
      const uint32_t byte = scale_byte<E5M2>(m);
      word |= byte << (8 * b);
      const int col = g * 512 + b * 128 + 4 * lane;
      const float inv = inverse_scale(byte);
      const uint32_t c = careful ? codes4<E5M2, true>(v.at(0), v.at(1), v.at(2), v.at(3), inv)
                                 : codes4<E5M2, false>(v.at(0), v.at(1), v.at(2), v.at(3), inv);
      if (src[i] >= 0) store4(a, a.q + int64_t(r0 + i) * a.ldq + col, c, a.cols - col);
    }
    uint8_t* const s = a.sq + scale_at(r0 + i, int64_t(g) * 4, groups);
    if (lane == 0 && DG_IN(a.dbg, s, 4, DBG_QUANTIZE)) *reinterpret_cast<uint32_t*>(s) = word;
  }
}

// Both orientations (or 128 x 128 scales): a CTA takes 128 x 128 tiles, kTileRows rows a
// warp and 4 columns a lane, held in registers.  Row maxima are warp reductions, each
// row's scale worked out by one lane; column maxima meet in shared memory, each column's
// scale worked out by one thread.  A thread's 8 rows of a column are 8 consecutive bytes of the
// transposed matrix: they are turned round in a swizzled shared-memory tile and leave as
// 128-byte rows.
// Many CTAs one after another overlap loading, converting and storing better than a few that
// go from tile to tile with the next one's loads under way (8192 x 4096 bf16, both ways, two CTAs an SM:
// 36.5 against 47.3 us).  Values stay in the input's type until a conversion needs them, so
// that 40 registers do and three CTAs share an SM: 30.0 us, 4.5 TB/s; 32-bit input two: 40.7
// us (one: 54.8).
constexpr int kTileRows = 8;
constexpr int kTileWarps = 128 / kTileRows;

// Lane that works out row i's scale, and the row of a lane (kTileRows: none).
__device__ __forceinline__ int lane_of_row(int i) { return (i >> 1) * 8 + (i & 1); }
__device__ __forceinline__ int row_of_lane(int lane) { return (lane & 7) < 2 ? (lane >> 3) * 2 + (lane & 1) : kTileRows; }

// Largest magnitudes of the 8 rows, each in the lane of its row: two rows to a register, and
// lanes halve the rows they hold as they exchange (6 exchanges; one reduction a row would
// be 8 and as many selections more).  32-bit values: a reduction a row.
template <typename T>
__device__ __forceinline__ uint32_t row_maxima(const Four<T> (&v)[kTileRows], int lane) {
  if constexpr (sizeof(T) == 4) {
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
      Peak<T> row;
      row.take(v[i]);
      const uint32_t m = __reduce_max_sync(kAll, row.row());
      if (lane == lane_of_row(i)) mine = m;
    }
    return mine;
  } else {
    uint32_t k[4];  // rows 2i and 2i + 1
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = Peak<T>::most(v[2 * i].w.x & 0x7fff7fffu, v[2 * i].w.y & 0x7fff7fffu);
      const uint32_t b = Peak<T>::most(v[2 * i + 1].w.x & 0x7fff7fffu, v[2 * i + 1].w.y & 0x7fff7fffu);
      k[i] = Peak<T>::most(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    }
    const bool high = lane & 16, mid = lane & 8;
    const uint32_t o0 = __shfl_xor_sync(kAll, high ? k[0] : k[2], 16), o1 = __shfl_xor_sync(kAll, high ? k[1] : k[3], 16);
    const uint32_t k0 = Peak<T>::most(high ? k[2] : k[0], o0), k1 = Peak<T>::most(high ? k[3] : k[1], o1);
    uint32_t m = Peak<T>::most(mid ? k1 : k0, __shfl_xor_sync(kAll, mid ? k0 : k1, 8));
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) m = Peak<T>::most(m, __shfl_xor_sync(kAll, m, d));
    return Peak<T>::bits(lane & 1 ? m >> 16 : m & 0xffffu);
  }
}

// kTileRows rows' codes to q (inverse scales: in the rows' lanes).
template <bool E5M2, bool CAREFUL, typename T>
__device__ __forceinline__ void row_codes(const QuantArgs& a, const Four<T> (&v)[kTileRows], float inv_mine, uint32_t live,
                                          uint8_t* dst, int n) {
#pragma unroll
  for (int i = 0; i < kTileRows; ++i, dst += a.ldq) {
    const uint32_t c = codes4<E5M2, CAREFUL>(v[i].at(0), v[i].at(1), v[i].at(2), v[i].at(3),
                                             __shfl_sync(kAll, inv_mine, lane_of_row(i)));
    if ((live >> i) & 1u) store4(a, dst, c, n);
  }
}

// Codes of a lane's column j.
template <bool E5M2, bool CAREFUL, typename T>
__device__ __forceinline__ uint2 column_codes(const Four<T> (&v)[kTileRows], int j, float inv) {
  return make_uint2(codes4<E5M2, CAREFUL>(v[0].at(j), v[1].at(j), v[2].at(j), v[3].at(j), inv),
                    codes4<E5M2, CAREFUL>(v[4].at(j), v[5].at(j), v[6].at(j), v[7].at(j), inv));
}

template <typename T, bool E5M2, bool VEC>
__global__ void __launch_bounds__(32 * kTileWarps, sizeof(T) == 4 ? 2 : 3) quantize_tile_kernel(const QuantArgs a) {
  alignas(16) __shared__ uint32_t col_max[kTileWarps][128];
  alignas(16) __shared__ float col_inv[128];  // inverse scales of the columns
  __shared__ uint32_t tile_max[4], tile_byte;  // 128 x 128 scales: largest magnitudes of four stripes, the scale byte
  __shared__ uint4 turn[128 * 8];  // [column][8-byte piece of rows ^ (column / 4 % 16)]
  wait_prior_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cb = blockIdx.x, rb = blockIdx.y;  // past the matrix: only scale bytes, zero
  const int row0 = rb * 128 + warp * kTileRows, col = cb * 128 + 4 * lane;
  Four<T> v[kTileRows];
  uint32_t live = 0;  // rows that exist
  {
    int src[kTileRows];
    source_rows(a, row0, src);
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) live |= uint32_t(src[i] >= 0) << i;
    load_rows<T, VEC>(v, a, src, col);
  }
  bool careful = false;  // infinities or NaN: maxima over what is finite, careful conversions
  if (a.qt || a.block_rows > 1) {
    Peak<T> peak;
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) peak.take(v[i]);
    uint32_t cm[4] = {peak.column(0), peak.column(1), peak.column(2), peak.column(3)};
    const bool wild = max(max(cm[0], cm[1]), max(cm[2], cm[3])) >= kInf;
    if (wild) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cm[j] = 0;
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) cm[j] = max(cm[j], finite_bits(v[i].at(j)));
      }
    }
    *reinterpret_cast<uint4*>(&col_max[warp][4 * lane]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
    careful = __syncthreads_or(wild);
    // one thread a column: its scale, its scale byte
    if (threadIdx.x < 128) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < kTileWarps; ++w) m = max(m, col_max[w][threadIdx.x]);
      if (a.block_rows > 1) {  // one scale for the tile
        m = __reduce_max_sync(kAll, m);
        if (lane == 0) tile_max[warp] = m;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        m = max(max(tile_max[0], tile_max[1]), max(tile_max[2], tile_max[3]));
      }
      const uint32_t byte = scale_byte<E5M2>(m);
      col_inv[threadIdx.x] = inverse_scale(byte);
      const int c = cb * 128 + int(threadIdx.x);
      if (a.qt && c < a.cols_padded) {
        uint8_t* const s = a.sqt + scale_at(c, rb, a.qt_groups);
        if (DG_IN(a.dbg, s, 1, DBG_QUANTIZE)) *s = uint8_t(c < a.cols ? byte : 0u);
      }
      // (not into tile_max: a slower warp may still be reading it)
      if (a.block_rows > 1 && threadIdx.x == 0) tile_byte = byte;
    }
    __syncthreads();
  }
  const uint32_t tile_scale = a.block_rows > 1 ? tile_byte : 0u;
  const uint32_t peaks = a.q && a.block_rows == 1 ? row_maxima(v, lane) : 0u;
  if (a.q) {
    uint32_t mine = tile_scale;  // scale byte of the lane's row
    const int my_row = row0 + row_of_lane(lane);
    bool careful_rows = careful;
    if (a.block_rows == 1) {
      mine = peaks;
      careful_rows = __any_sync(kAll, mine >= kInf);
      if (careful_rows) {
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
          const uint32_t m = __reduce_max_sync(kAll, max(max(finite_bits(v[i].at(0)), finite_bits(v[i].at(1))),
                                                         max(finite_bits(v[i].at(2)), finite_bits(v[i].at(3)))));
          if (lane == lane_of_row(i)) mine = m;
        }
      }
      mine = scale_byte<E5M2>(mine);
    } else if (((live >> row_of_lane(lane)) & 1u) == 0u) {
      mine = 0;  // no such row, or a map that gives it no source
    }
    const float inv = a.block_rows == 1 ? inverse_scale(mine) : col_inv[0];
    uint8_t* const dst = a.q + int64_t(row0) * a.ldq + col;
    if (careful_rows)
      row_codes<E5M2, true>(a, v, inv, live, dst, a.cols - col);
    else
      row_codes<E5M2, false>(a, v, inv, live, dst, a.cols - col);
    if (row_of_lane(lane) < kTileRows && row0 < a.rows_padded) {
      uint8_t* const s = a.sq + scale_at(my_row, cb, a.q_groups);
      if (DG_IN(a.dbg, s, 1, DBG_QUANTIZE)) *s = uint8_t(mine);
    }
  }
  if (a.qt) {
    const float4 inv = *reinterpret_cast<const float4*>(&col_inv[4 * lane]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float by = j == 0 ? inv.x : j == 1 ? inv.y : j == 2 ? inv.z : inv.w;
      reinterpret_cast<uint2*>(turn)[(4 * lane + j) * 16 + (warp ^ (lane & 15))] =
          careful ? column_codes<E5M2, true>(v, j, by) : column_codes<E5M2, false>(v, j, by);
    }
    __syncthreads();
#pragma unroll
    for (int pass = 0; pass < 128 * 8 / (32 * kTileWarps); ++pass) {
      const int c = pass * 4 * kTileWarps + int(threadIdx.x >> 3), piece = threadIdx.x & 7;  // 16 bytes: two pieces of 8
      const int r = rb * 128 + piece * 16;
      if (cb * 128 + c >= a.cols || r >= a.rows) continue;
      const int f = (c >> 2) & 15;
      uint4 w = turn[c * 8 + (piece ^ (f >> 1))];
      if (f & 1) w = make_uint4(w.z, w.w, w.x, w.y);
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

template <typename T, bool E5M2, bool VEC>
cudaError_t launch(const QuantArgs& a, cudaStream_t s) {
  if (!a.qt && a.block_rows == 1) {
    const int64_t warps = int64_t(a.rows_padded / kRows) * a.q_groups;
    return launch_k(quantize_rows_kernel<T, E5M2, VEC>, dim3(unsigned((warps + 7) / 8)), dim3(256), 0, s, a.pdl, a);
  }
  // blocks past the matrix write the zero bytes that pad the scales to whole words
  const int col_blocks = a.q ? a.q_groups * 4 : (a.cols + 127) / 128;
  const int row_blocks = a.qt ? a.qt_groups * 4 : (a.rows + 127) / 128;
  return launch_k(quantize_tile_kernel<T, E5M2, VEC>, dim3(unsigned(col_blocks), unsigned(row_blocks)),
                  dim3(32 * kTileWarps), 0, s, a.pdl, a);
}

template <typename T>
cudaError_t launch_type(const QuantArgs& a, cudaStream_t s) {
  if (a.vec) return a.e5m2 ? launch<T, true, true>(a, s) : launch<T, false, true>(a, s);
  return a.e5m2 ? launch<T, true, false>(a, s) : launch<T, false, false>(a, s);
}

// Pieces of 16 bytes, loaded as the rows' alignment allows (T); a thread takes kItems of them,
// a CTA's width apart, whatever rows they belong to (a CTA a row: 45 us for 48 x 1744 rows of 616 bytes).
constexpr int kItems = 4;

template <typename T>
__global__ void __launch_bounds__(256) repack_kernel(const RepackArgs a, uint32_t pieces) {
  wait_prior_grid();
  const int z = int(blockIdx.z);
  if (a.counts && (!DG_IN(a.dbg, a.counts + z, 4, DBG_QUANTIZE) || __ldg(a.counts + z) <= 0)) return;
  const uint8_t* const in = a.in + z * a.group;
  uint8_t* const out = a.out + int64_t(z) * a.rows * a.ld_out;
  alignas(16) T v[kItems][16 / sizeof(T)];
  int64_t from[kItems], to[kItems];
  int n[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const uint64_t item = (uint64_t(blockIdx.x) * kItems + i) * 256 + threadIdx.x;
    const uint32_t r = uint32_t(item) / pieces, col = (uint32_t(item) - r * pieces) * 16;
    n[i] = item < uint64_t(a.rows) * pieces ? min(16, a.cols - int(col)) : 0;
    from[i] = int64_t(r) * a.ld + col;
    to[i] = int64_t(r) * a.ld_out + col;
#pragma unroll
    for (int j = 0; j < int(16 / sizeof(T)); ++j) {
      v[i][j] = 0;
      // (the last one of a row may reach past it: those byte by byte, below)
      if (int((j + 1) * sizeof(T)) <= n[i] && DG_IN(a.dbg, in + from[i] + j * sizeof(T), int(sizeof(T)), DBG_QUANTIZE))
        v[i][j] = __ldg(reinterpret_cast<const T*>(in + from[i]) + j);
    }
  }
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (n[i] <= 0 || !DG_IN(a.dbg, out + to[i], 16, DBG_QUANTIZE)) continue;
    const int whole = n[i] / int(sizeof(T)) * int(sizeof(T));
    *reinterpret_cast<uint4*>(out + to[i]) = *reinterpret_cast<const uint4*>(&v[i][0]);
    for (int b = whole; b < n[i]; ++b)
      if (DG_IN(a.dbg, in + from[i] + b, 1, DBG_QUANTIZE)) out[to[i] + b] = __ldg(in + from[i] + b);
  }
}

template <typename T>
cudaError_t launch_repack_type(const RepackArgs& a, cudaStream_t s) {
  const uint32_t pieces = uint32_t((a.cols + 15) / 16);
  const uint64_t items = uint64_t(a.rows) * pieces;
  return launch_k(repack_kernel<T>, dim3(unsigned((items + 256 * kItems - 1) / (256 * kItems)), 1, unsigned(a.groups)),
                  dim3(256), 0, s, a.pdl, a, pieces);
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
