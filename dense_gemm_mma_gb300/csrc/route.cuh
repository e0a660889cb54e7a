// route.cuh -- logits and scores of a token, a warp to it: what routing (route.cu) and the balance of its
// choices (balance.cu) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kernels.h"

namespace dg {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kNegInf = -__builtin_huge_valf();
// A number's order as an unsigned integer, -0 as 0 (positive: the sign bit set; negative: all bits flipped).
__device__ __forceinline__ uint32_t number_key(float f) {
  const uint32_t b = __float_as_uint(f + 0.f);
  return b ^ (uint32_t(int(b) >> 31) | 0x80000000u);
}

// The same for any float: NaN as minus infinity.
__device__ __forceinline__ uint32_t order_key(float f) { return number_key(f == f ? f : kNegInf); }

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float half_at(uint32_t pair, int i, int kind) {
  if (kind == OUT_BF16) return __uint_as_float(i & 1 ? pair & 0xffff0000u : pair << 16);
  const uint16_t h = uint16_t(i & 1 ? pair >> 16 : pair);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__device__ __forceinline__ uint32_t half_pair(float a, float b, int kind) {
  if (kind == OUT_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// NaN read as minus infinity.
__device__ __forceinline__ float masked(float f) { return f == f ? f : kNegInf; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, d));
  return v;
}

// Logit e of token t; what is not there is minus infinity.
__device__ __forceinline__ float logit(const RouteArgs& a, int t, int e) {
  if (e < 0 || e >= a.experts) return kNegInf;
  const int es = a.kind == OUT_F32 ? 4 : 2;
  const char* const p = static_cast<const char*>(a.logits) + (int64_t(t) * a.ldl + e) * es;
  if (!DG_IN(a.dbg, p, es, DBG_ROUTE)) return kNegInf;
  if (es == 4) return masked(*reinterpret_cast<const float*>(p));
  return masked(half_at(*reinterpret_cast<const uint16_t*>(p), 0, a.kind));
}

// A lane's experts: lane * run .. lane * run + run, run <= P.  Whole runs of a row on
// 16-byte boundaries (`wide`) are loaded 8 or 16 bytes at a time.
template <int P>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int t, int first, int run, bool wide, float (&x)[P]) {
  if constexpr (P >= 4) {
    if (wide && run == P && first + P <= a.experts) {
      const int es = a.kind == OUT_F32 ? 4 : 2;
      const char* const p = static_cast<const char*>(a.logits) + (int64_t(t) * a.ldl + first) * es;
      if (DG_IN(a.dbg, p, P * es, DBG_ROUTE)) {
        if (a.kind == OUT_F32) {
#pragma unroll
          for (int i = 0; i < P; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + 4 * i);
            x[i] = masked(v.x), x[i + 1] = masked(v.y), x[i + 2] = masked(v.z), x[i + 3] = masked(v.w);
          }
        } else {
#pragma unroll
          for (int i = 0; i < P; i += 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(p + 2 * i);
            x[i] = masked(half_at(v.x, 0, a.kind)), x[i + 1] = masked(half_at(v.x, 1, a.kind));
            x[i + 2] = masked(half_at(v.y, 0, a.kind)), x[i + 3] = masked(half_at(v.y, 1, a.kind));
          }
        }
        return;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = i < run ? logit(a, t, first + i) : kNegInf;
}

// What turns a token's logits into scores.  A masked expert (minus infinity) scores 0;
// a row with nothing else scores 0 throughout; of logits of plus infinity each takes an equal share.
struct Scorer {
  int sigmoid;
  float top, sum;  // softmax: largest logit, sum of exp(x - top)
  // `best`: the key of the lane's largest logit
  template <int P>
  __device__ __forceinline__ Scorer(const RouteArgs& a, const float (&x)[P], uint32_t best)
      : sigmoid(a.sigmoid), top(kNegInf), sum(0.f) {
    if (sigmoid) return;
    top = key_value(__reduce_max_sync(kAll, best));
    if (fabsf(top) < -kNegInf) {  // exp(-inf) is 0 and exp(0) is 1: nothing to look out for
#pragma unroll
      for (int i = 0; i < P; ++i) sum = __fadd_rn(sum, expf(__fsub_rn(x[i], top)));
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) sum = __fadd_rn(sum, power(x[i]));
    }
    sum = warp_sum(sum);
  }
  __device__ __forceinline__ float power(float x) const {  // softmax's numerator
    return x == kNegInf ? 0.f : x == top ? 1.f : expf(__fsub_rn(x, top));
  }
  __device__ __forceinline__ float score(float x) const {
    if (sigmoid) return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-x)));
    return sum > 0.f ? __fdiv_rn(power(x), sum) : 0.f;
  }
};

template <typename F>
cudaError_t by_experts(int experts, F f) {
  if (experts <= 32) return f(std::integral_constant<int, 1>{});
  if (experts <= 64) return f(std::integral_constant<int, 2>{});
  if (experts <= 128) return f(std::integral_constant<int, 4>{});
  if (experts <= 256) return f(std::integral_constant<int, 8>{});
  if (experts <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace
}  // namespace dg
