// route.cu -- routing of tokens to experts: scores, choice, weights; the order of the
// chosen rows by expert; the gradient of the scores.
//
// Scores of a token's logits x_i: softmax s_i = exp(x_i - max) / sum, or sigmoid
// s_i = 1 / (1 + exp(-x_i)).  The choice goes by a key: the logit itself where the order of the scores is all
// that counts (no bias, groups ranked by their best), else s_i + bias_i.  Weights of the chosen: s_i, over their
// sum if renormalised, times `scale`.
//
// What bounds it is latency for few tokens, then issuing instructions (reading the
// logits is a few microseconds at most): one warp a token, a run of consecutive experts per
// lane in registers, sorted by order-preserving integer keys.  A choice is then one warp
// maximum over the lanes' first keys: the lowest lane that has it holds the lowest expert that has it, and
// moves on to its next.  Scores are worked out only where something needs them.
// Measured, softmax, 16384 tokens, 8 of 128 experts: choice and weights 8.2 us, renormalised 9.0 (460 and 519 instructions a
// token), gradient 8.3 and 8.6 us (370 and 430); 16 tokens, sigmoid, 8 of 256 experts in groups: 4.1 us.
// Sums and products that make a key are written with the rounding intrinsics, so that no
// compiler contraction moves it by a bit: the choice depends on it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kernels.h"

namespace dg {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr float kNegInf = -__builtin_huge_valf();
// Keys of experts that are not there or taken, and of experts outside the chosen groups; every float's key is larger.
constexpr uint32_t kNone = 0, kOutside = 1;

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

// Sorts a lane's keys, largest first (an odd-even network of P rounds); ex[i] is the expert of
// key[i].  Equal keys keep the lower expert first: only a strictly larger key moves up.
template <int P>
__device__ __forceinline__ void sort_lane(uint32_t (&key)[P], int (&ex)[P]) {
#pragma unroll
  for (int round = 0; round < P; ++round)
#pragma unroll
    for (int i = round & 1; i + 1 < P; i += 2) {
      const bool up = key[i + 1] > key[i];
      const uint32_t k0 = key[i], k1 = key[i + 1];
      const int e0 = ex[i], e1 = ex[i + 1];
      key[i] = up ? k1 : k0, key[i + 1] = up ? k0 : k1;
      ex[i] = up ? e1 : e0, ex[i + 1] = up ? e0 : e1;
    }
}

// The warp's best expert; its lane moves on to its next one.
template <int P>
__device__ __forceinline__ int take_best(uint32_t (&key)[P], int (&ex)[P], int lane, uint32_t* value) {
  const uint32_t best = __reduce_max_sync(kAll, key[0]);
  *value = best;
  const int owner = __ffs(__ballot_sync(kAll, key[0] == best)) - 1;
  const int expert = __shfl_sync(kAll, ex[0], owner);
  if (lane == owner) {
#pragma unroll
    for (int i = 0; i + 1 < P; ++i) key[i] = key[i + 1], ex[i] = ex[i + 1];
    key[P - 1] = kNone;
  }
  return expert;
}

__device__ __forceinline__ uint32_t group_key(const RouteArgs& a, uint32_t best, uint32_t second) {
  return a.group_top == 2 && second != kNone ? order_key(__fadd_rn(key_value(best), key_value(second))) : best;
}

// The top_groups groups of the largest keys, ties to the lower group: bit g of the result.
// Group g's key is `mine` in lane g * every, and kNone elsewhere.
__device__ __forceinline__ uint32_t choose_groups(const RouteArgs& a, uint32_t mine, int every, int lane) {
  uint32_t chosen = 0;
  for (int i = 0; i < a.top_groups; ++i) {
    const uint32_t best = __reduce_max_sync(kAll, mine);
    const int owner = __ffs(__ballot_sync(kAll, mine == best)) - 1;
    chosen |= 1u << (owner / every);
    if (lane == owner) mine = kNone;
  }
  return chosen;
}

template <int P>
__global__ void __launch_bounds__(128) route_kernel(const RouteArgs a) {
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int t = int(blockIdx.x * 4 + (threadIdx.x >> 5));
  if (t >= a.tokens) return;
  const int run = (a.experts + 31) / 32, first = lane * run;
  float x[P];
  load_logits(a, t, first, run, a.wide, x);
  uint32_t key[P];
  int ex[P];
  uint32_t lane_best = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    key[i] = number_key(x[i]);
    ex[i] = first + i;
    lane_best = max(lane_best, key[i]);
  }
  const Scorer scorer(a, x, lane_best);
  const bool by_logit = a.bias == nullptr && a.group_top == 1;
  if (!by_logit) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (x[i] == kNegInf) continue;  // a masked expert stays minus infinity, whatever its bias
      float k = scorer.score(x[i]);
      if (a.bias && DG_IN(a.dbg, a.bias + ex[i], 4, DBG_ROUTE)) k = __fadd_rn(k, __ldg(a.bias + ex[i]));
      key[i] = order_key(k);
    }
  }
  if (run * 32 != a.experts || run != P) {  // what is not there
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i >= run || ex[i] >= a.experts) key[i] = kNone;
  }
  // Groups that are whole lanes (a power of two of them, every lane full): their best keys
  // meet in a few exchanges.  Others: one pair of warp maxima each.
  const bool by_lanes = a.experts % 32 == 0 && 32 % a.groups == 0;
  if (a.groups > 1 && !by_lanes) {
    const int per = a.experts / a.groups;
    uint32_t mine = kNone;
    for (int g = 0; g < a.groups; ++g) {
      uint32_t b1 = kNone, b2 = kNone;  // of this lane
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (ex[i] >= g * per && ex[i] < (g + 1) * per) {
          b2 = max(b2, min(b1, key[i]));
          b1 = max(b1, key[i]);
        }
      const uint32_t best = __reduce_max_sync(kAll, b1);
      // the best may be there more than once: only one lane gives its own up
      const int owner = __ffs(__ballot_sync(kAll, b1 == best)) - 1;
      const uint32_t second = __reduce_max_sync(kAll, lane == owner ? b2 : b1);
      if (lane == g) mine = group_key(a, best, second);
    }
    const uint32_t chosen = choose_groups(a, mine, 1, lane);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (key[i] != kNone && !((chosen >> (ex[i] / per)) & 1u)) key[i] = kOutside;
  }
  sort_lane(key, ex);
  if (a.groups > 1 && by_lanes) {
    const int every = 32 / a.groups;
    uint32_t b1 = key[0], b2 = kNone;
    if constexpr (P > 1) b2 = key[1];
    for (int d = 1; d < every; d <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(kAll, b1, d), o2 = __shfl_xor_sync(kAll, b2, d);
      b2 = max(min(b1, o1), max(b2, o2));
      b1 = max(b1, o1);
    }
    const uint32_t chosen = choose_groups(a, lane % every == 0 ? group_key(a, b1, b2) : kNone, every, lane);
    if (!((chosen >> (lane / every)) & 1u))
#pragma unroll
      for (int i = 0; i < P; ++i) key[i] = min(key[i], kOutside);
  }
  int expert = -1;  // lane j: choice j
  uint32_t best = kNone;
  for (int j = 0; j < a.top_k; ++j) {
    uint32_t k;
    const int e = take_best(key, ex, lane, &k);
    if (lane == j) expert = e, best = k;
  }
  // the chosen ones' scores, from the key where it is the logit, else from the logits again
  // (a few loads that hit L1)
  const float mine = !by_logit ? logit(a, t, expert) : expert >= 0 ? key_value(best) : kNegInf;
  float score = mine == kNegInf ? 0.f : scorer.score(mine);
  if (a.renormalize) {
    const float sum = warp_sum(score);
    score = sum > 0.f ? __fdiv_rn(score, sum) : 0.f;
  }
  if (lane < a.top_k) {
    const int64_t at = int64_t(t) * a.top_k + lane;
    if (DG_IN(a.dbg, a.weights + at, 4, DBG_ROUTE)) a.weights[at] = __fmul_rn(score, a.scale);
    if (DG_IN(a.dbg, a.indices + at, 4, DBG_ROUTE)) a.indices[at] = expert;
  }
}

// Without renormalising w_j = scale s_j, and with g_j = scale dw_j s_j
//   dx_i = g_i - s_i sum_j g_j (softmax), g_i (1 - s_i) = g_i / (1 + exp(x_i)) (sigmoid)
// where g_i is 0 for experts that were not chosen (the difference 1 - s_i of a rounded s_i would be 1% off at x_i = 12).  With it w_j = scale s_j / S, S the chosen scores' sum, and
//   g_j = scale (s_j / S) (dw_j - sum_i dw_i s_i / S)
// whose sum is 0 whatever dw: softmax's second term goes.  Written by the quotients s_j / S, which are at most 1, so
// that nothing overflows however small the chosen scores are ((dw_j - ...) / S does from S ~ 1e-38).
// The scores are computed again from the logits: reading them costs what reading kept scores would.
template <int P>
__global__ void __launch_bounds__(128) route_backward_kernel(const RouteArgs a) {
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int t = int(blockIdx.x * 4 + (threadIdx.x >> 5));
  if (t >= a.tokens) return;
  const int run = (a.experts + 31) / 32, first = lane * run;
  float x[P], dx[P];
  load_logits(a, t, first, run, a.wide, x);
  float lane_best = kNegInf;
#pragma unroll
  for (int i = 0; i < P; ++i) lane_best = fmaxf(lane_best, x[i]);
  const Scorer scorer(a, x, number_key(lane_best));
  int expert = -1;  // lane j: choice j; an index outside the experts takes no part
  float dw = 0.f;
  if (lane < a.top_k) {
    const int64_t at = int64_t(t) * a.top_k + lane;
    if (DG_IN(a.dbg, a.indices + at, 4, DBG_ROUTE)) expert = a.indices[at];
    if (DG_IN(a.dbg, a.dweights + at, 4, DBG_ROUTE)) dw = a.dweights[at];
    if (expert < 0 || expert >= a.experts) expert = -1, dw = 0.f;
  }
  const float chosen = logit(a, t, expert);
  const float sj = chosen == kNegInf ? 0.f : scorer.score(chosen);
  float gj = sj, through = 0.f;
  if (a.renormalize) {
    const float sum = warp_sum(sj);
    // a token whose one score is its sum has a weight of exactly 1, and a gradient of exactly 0
    const float w = sum > 0.f ? sj / sum : 0.f;
    const float dot = warp_sum(dw * w);
    gj = a.scale * w * (dw - dot);
  } else {
    gj *= a.scale * dw;
    through = warp_sum(gj);
  }
  // gj from lane j to the lane of its expert: through shared memory, or one after another
  // where two choices name the same expert (their sum then has an order)
  __shared__ float moved[4][32 * P];
  float* const mine = moved[threadIdx.x >> 5] + lane * P;
  const uint32_t same = __match_any_sync(kAll, expert >= 0 ? expert : -1 - lane);
  if (__any_sync(kAll, (same & (same - 1)) != 0)) {
#pragma unroll
    for (int i = 0; i < P; ++i) dx[i] = 0.f;
    for (int j = 0; j < a.top_k; ++j) {
      const int at = __shfl_sync(kAll, expert, j) - first;
      const float d = __shfl_sync(kAll, gj, j);
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (at == i && i < run) dx[i] += d;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) mine[i] = 0.f;
    __syncwarp();
    if (expert >= 0) moved[threadIdx.x >> 5][expert / run * P + expert % run] = gj;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < P; ++i) dx[i] = mine[i];
  }
  if (!a.sigmoid) {
    // (also where weights are renormalised and `through` is 0: a branch round it took two registers more than
    // the 32 with which 16 CTAs share an SM)
    const float by = scorer.sum > 0.f ? 1.f / scorer.sum * through : 0.f;
    if (fabsf(scorer.top) < -kNegInf) {
#pragma unroll
      for (int i = 0; i < P; ++i) dx[i] -= expf(x[i] - scorer.top) * by;
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) dx[i] -= scorer.power(x[i]) * by;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (dx[i] == 0.f) continue;  // (experts that were not chosen)
      dx[i] = __fdiv_rn(dx[i], __fadd_rn(1.f, expf(x[i])));
    }
  }
  const int es = a.kind == OUT_F32 ? 4 : 2;
  char* const dst = static_cast<char*>(a.dlogits) + (int64_t(t) * a.lddl + first) * es;
  if constexpr (P >= 4) {
    if (a.wide_out && run == P && first + P <= a.experts) {
      if (!DG_IN(a.dbg, dst, P * es, DBG_ROUTE)) return;
#pragma unroll
      for (int i = 0; i < P; i += 4) {
        if (a.kind == OUT_F32)
          *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(dx[i], dx[i + 1], dx[i + 2], dx[i + 3]);
        else
          *reinterpret_cast<uint2*>(dst + 2 * i) =
              make_uint2(half_pair(dx[i], dx[i + 1], a.kind), half_pair(dx[i + 2], dx[i + 3], a.kind));
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (i >= run || first + i >= a.experts || !DG_IN(a.dbg, dst + i * es, es, DBG_ROUTE)) continue;
    if (es == 4)
      *reinterpret_cast<float*>(dst + 4 * i) = dx[i];
    else
      *reinterpret_cast<uint16_t*>(dst + 2 * i) = uint16_t(half_pair(dx[i], 0.f, a.kind));
  }
}

template <typename F>
cudaError_t by_experts(int experts, F f) {
  if (experts <= 32) return f(std::integral_constant<int, 1>{});
  if (experts <= 64) return f(std::integral_constant<int, 2>{});
  if (experts <= 128) return f(std::integral_constant<int, 4>{});
  if (experts <= 256) return f(std::integral_constant<int, 8>{});
  if (experts <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

// ------------------------------------------------------------------- order
//
// A stable counting sort of the slots (token * top_k + choice) by expert.  Each CTA has a run of
// the slots, each warp a run of its CTA's: a first walk counts them by expert
// (lanes with the same expert find each other with match, one of them adds) and keeps each
// slot's place among its CTA's slots of its expert in pos; a second walk turns places into rows: first row of
// the expert + slots of earlier CTAs + place.  No atomics: the order is the slots' own.
//   up to kMapRun slots: one launch, one CTA
//   more: two launches, the CTAs' counts in between in plan workspace; every CTA
//         of the second sums up the counts of those before it (and of all) by itself.
// One launch on a cluster of eight CTAs took 36 us for 131072 slots of 128 experts, two launches of 64 CTAs 9.2 us.
constexpr int kMapThreads = 1024;
constexpr int kMapWarps = kMapThreads / 32;
constexpr int kAhead = 4;  // loads of a warp's slots that are in flight together

struct MapRun {  // a warp's slots [first, last), `first` a multiple of 32 from the CTA's start
  int64_t first, last;
};

__device__ __forceinline__ MapRun map_run(const RouteMapArgs& a, int block, int warp) {
  const int64_t from = int64_t(block) * a.run, to = min(int64_t(a.slots), from + a.run);
  const int per = a.run / a.warps;  // a multiple of 32
  MapRun r;
  r.first = warp < a.warps ? min(to, from + int64_t(warp) * per) : to;
  r.last = warp < a.warps ? min(to, r.first + per) : to;
  return r;
}

__device__ __forceinline__ int expert_of(const RouteMapArgs& a, int64_t slot, int64_t last) {
  if (slot >= last || !DG_IN(a.dbg, a.indices + slot, 4, DBG_ROUTE)) return -1;
  const int e = __ldg(a.indices + slot);
  return e >= 0 && e < a.experts ? e : -1;
}

// Every row holds no slot, until its slot says otherwise.
__device__ __forceinline__ void map_clear_rows(const RouteMapArgs& a, int block, int blocks) {
  for (int64_t r = 4 * (int64_t(block) * kMapThreads + threadIdx.x); r < a.rows; r += 4 * int64_t(blocks) * kMapThreads) {
    const int n = int(min(int64_t(4), a.rows - r));
    if (!DG_IN(a.dbg, a.rowmap + r, 4 * n, DBG_ROUTE)) continue;
    if (n == 4 && a.wide)
      *reinterpret_cast<int4*>(a.rowmap + r) = make_int4(-1, -1, -1, -1);
    else
      for (int i = 0; i < n; ++i) a.rowmap[r + i] = -1;
  }
}

// First walk of a CTA.  count: [warps][experts]; afterwards count[w][e] is the number of slots of e in
// warps before w, total[e] in the CTA.  A slot's place among its warp's is in pos.
__device__ __forceinline__ void map_count(const RouteMapArgs& a, const MapRun& r, int* count, int* total) {
  const int E = a.experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < E * a.warps; i += kMapThreads) count[i] = 0;
  __syncthreads();
  int* const mine = count + warp * E;
  for (int64_t s = r.first; s < r.last; s += 32 * kAhead) {
    int e[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) e[i] = expert_of(a, s + 32 * i + lane, r.last);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t slot = s + 32 * i + lane;
      const uint32_t same = __match_any_sync(kAll, e[i]);
      const int earlier = e[i] >= 0 ? mine[e[i]] : 0;
      __syncwarp();
      if (e[i] >= 0 && lane == __ffs(same) - 1) mine[e[i]] = earlier + __popc(same);
      __syncwarp();
      if (slot < r.last && DG_IN(a.dbg, a.pos + slot, 4, DBG_ROUTE))
        a.pos[slot] = earlier + __popc(same & ((1u << lane) - 1u));
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kMapThreads) {
    int sum = 0;
    for (int w = 0; w < a.warps; ++w) {
      const int n = count[w * E + e];
      count[w * E + e] = sum;
      sum += n;
    }
    total[e] = sum;
  }
}

// all[e] -> start[e], the first row of expert e: whole 128s of the experts before (experts <=
// kMapThreads: one a thread).  Block `writer` writes starts and counts.
__device__ __forceinline__ void map_starts(const RouteMapArgs& a, const int* all, int* start, int* warp_sums, bool writer) {
  const int e = threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = e < a.experts ? (all[e] + 127) & ~127 : 0;
  int sum = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kAll, sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sums[w];
  if (e < a.experts) {
    start[e] = before + sum - n;
    if (writer && DG_IN(a.dbg, a.starts + e, 4, DBG_ROUTE)) a.starts[e] = start[e];
    if (writer && DG_IN(a.dbg, a.counts + e, 4, DBG_ROUTE)) a.counts[e] = all[e];
  }
}

// Second walk: row of a slot = offset[expert] + place.
template <typename F>
__device__ __forceinline__ void map_place(const RouteMapArgs& a, const MapRun& r, F offset) {
  const int lane = threadIdx.x & 31;
  for (int64_t s = r.first; s < r.last; s += 32 * kAhead) {
    int e[kAhead], place[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t slot = s + 32 * i + lane;
      e[i] = expert_of(a, slot, r.last);
      place[i] = slot < r.last && DG_IN(a.dbg, a.pos + slot, 4, DBG_ROUTE) ? a.pos[slot] : 0;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t slot = s + 32 * i + lane;
      if (slot >= r.last || !DG_IN(a.dbg, a.pos + slot, 4, DBG_ROUTE)) continue;
      const int row = e[i] >= 0 ? offset(e[i]) + place[i] : -1;
      a.pos[slot] = row;
      if (row >= 0 && row < a.rows && DG_IN(a.dbg, a.rowmap + row, 4, DBG_ROUTE)) a.rowmap[row] = int(slot);
    }
  }
}

// ints of shared memory: totals, first rows and warp sums, then [warps][experts]
__host__ __device__ constexpr int map_ints(int experts, int warps) { return experts * (2 + warps) + 32; }

__global__ void __launch_bounds__(kMapThreads) route_map_kernel(const RouteMapArgs a) {
  extern __shared__ int map_shared[];
  int* const total = map_shared;
  int* const start = total + a.experts;
  int* const warp_sums = start + a.experts;
  int* const count = warp_sums + 32;
  const int warp = threadIdx.x >> 5;
  wait_prior_grid();
  map_clear_rows(a, 0, 1);
  const MapRun r = map_run(a, 0, warp);
  map_count(a, r, count, total);
  __syncthreads();
  map_starts(a, total, start, warp_sums, true);
  __syncthreads();
  const int* const mine = count + warp * a.experts;
  map_place(a, r, [&](int e) { return start[e] + mine[e]; });
}

// Two launches.  block_counts: [blocks][experts].
__global__ void __launch_bounds__(kMapThreads) route_map_count_kernel(const RouteMapArgs a) {
  extern __shared__ int map_shared[];
  int* const total = map_shared;
  int* const count = total + a.experts;
  const int block = int(blockIdx.x), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_prior_grid();
  map_clear_rows(a, block, int(gridDim.x));
  const MapRun r = map_run(a, block, warp);
  map_count(a, r, count, total);
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kMapThreads) {
    int* const c = a.block_counts + int64_t(block) * a.experts + e;
    if (DG_IN(a.dbg, c, 4, DBG_ROUTE)) *c = total[e];
  }
  // places among the CTA's slots
  const int* const mine = count + warp * a.experts;
  for (int64_t slot = r.first + lane; slot < r.last; slot += 32) {
    const int e = expert_of(a, slot, r.last);
    if (e >= 0 && DG_IN(a.dbg, a.pos + slot, 4, DBG_ROUTE)) a.pos[slot] += mine[e];
  }
}

__global__ void __launch_bounds__(kMapThreads) route_map_place_kernel(const RouteMapArgs a) {
  extern __shared__ int map_shared[];
  const int E = a.experts, blocks = int(gridDim.x), block = int(blockIdx.x), warp = threadIdx.x >> 5;
  int* const all = map_shared;
  int* const before = all + E;
  int* const start = before + E;
  int* const warp_sums = start + E;
  wait_prior_grid();
  for (int e = threadIdx.x; e < E; e += kMapThreads) all[e] = before[e] = 0;
  __syncthreads();
  // counts of all CTAs and of those before this one: 8 CTAs' counts of an expert a thread
  // (whole numbers: the order of the additions does not matter)
  const int parts = (blocks + 7) / 8;
  for (int i = threadIdx.x; i < parts * E; i += kMapThreads) {
    const int e = i % E, b0 = i / E * 8;
    int n[8], sum = 0, earlier = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int* const c = a.block_counts + int64_t(b0 + j) * E + e;
      n[j] = b0 + j < blocks && DG_IN(a.dbg, c, 4, DBG_ROUTE) ? __ldcg(c) : 0;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum += n[j];
      if (b0 + j < block) earlier += n[j];
    }
    if (sum) atomicAdd(all + e, sum);
    if (earlier) atomicAdd(before + e, earlier);
  }
  __syncthreads();
  map_starts(a, all, start, warp_sums, block == 0);
  __syncthreads();
  map_place(a, map_run(a, block, warp), [&](int e) { return start[e] + before[e]; });
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  return by_experts(a.experts, [&](auto p) {
    return launch_k(route_kernel<decltype(p)::value>, dim3(unsigned((a.tokens + 3) / 4)), dim3(128), 0, s, a.pdl, a);
  });
}

cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t s) {
  return by_experts(a.experts, [&](auto p) {
    return launch_k(route_backward_kernel<decltype(p)::value>, dim3(unsigned((a.tokens + 3) / 4)), dim3(128), 0, s,
                    a.pdl, a);
  });
}

constexpr int kMapRun = 2048;     // slots of a CTA, where there are not more than kMapBlocks of them
constexpr int kMapBlocks = 128;

static int map_blocks(int64_t slots) {
  return int(std::min<int64_t>(kMapBlocks, std::max<int64_t>(1, (slots + kMapRun - 1) / kMapRun)));
}

size_t route_map_workspace(int64_t slots, int64_t experts) {
  const int blocks = map_blocks(slots);
  return blocks > 1 ? size_t(blocks) * size_t(experts) * 4 : 0;
}

cudaError_t launch_route_map(RouteMapArgs a, cudaStream_t s) {
  const int blocks = map_blocks(a.slots);
  const int per_block = (a.slots + blocks - 1) / blocks;
  a.warps = std::max(1, std::min(kMapWarps, (per_block + 31) / 32));
  const int per_warp = ((per_block + a.warps - 1) / a.warps + 31) & ~31;
  a.run = per_warp * a.warps;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limits are set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit == 0 || (ready.load(std::memory_order_acquire) & bit) == 0) {
    const int most = map_ints(ROUTE_MAX_EXPERTS, kMapWarps) * 4;
    cudaError_t err = cudaFuncSetAttribute(route_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (err == cudaSuccess)
      err = cudaFuncSetAttribute(route_map_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (err != cudaSuccess) return err;
    ready.fetch_or(bit, std::memory_order_release);
  }
  const size_t smem = size_t(map_ints(a.experts, a.warps)) * 4;
  if (blocks == 1) return launch_k(route_map_kernel, dim3(1), dim3(kMapThreads), smem, s, a.pdl, a);
  const cudaError_t err = launch_k(route_map_count_kernel, dim3(unsigned(blocks)), dim3(kMapThreads), smem, s, a.pdl, a);
  if (err != cudaSuccess) return err;
  return launch_k(route_map_place_kernel, dim3(unsigned(blocks)), dim3(kMapThreads), size_t(3 * a.experts + 32) * 4, s,
                  a.pdl, a);
}

}  // namespace dg
