// codes.cuh -- codes and their power-of-two scales: what the quantisers and the norm that writes
// codes share (the scale's rule: quantize.cu).
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

#include "kernels.h"

namespace dg {

constexpr uint32_t kAll = 0xffffffffu;

constexpr uint32_t kInf = 0x7f800000u;  // fp32 bits; those of infinities and NaN are at least that

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

}  // namespace dg
