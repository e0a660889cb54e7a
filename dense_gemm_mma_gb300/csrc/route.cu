// route.cu -- routing of tokens to experts: scores, choice, weights; the order of the
// chosen rows by expert; the gradient of the scores.
//
// Scores of a token's logits x_i: softmax s_i = exp(x_i - max) / sum, or sigmoid
// s_i = 1 / (1 + exp(-x_i)).  The choice goes by a key: the logit itself where the order of the scores is all
// that counts (no bias, groups ranked by their best), else s_i + bias_i.  Weights of the chosen: s_i, over their
// sum if renormalised, times `scale`.
//
// What bounds it is latency, then reading the logits: one warp a token, its experts in
// registers (expert 32 i + lane in register i), each choice two warp reductions on
// order-preserving integer keys (largest key, then the lowest index that has it).
// Sums and products are written with the rounding intrinsics, so that no compiler
// contraction moves a key by a bit: the choice depends on it.
#include <cooperative_groups.h>
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

// A float's order as an unsigned integer; NaN as minus infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float f) {
  f = f == f ? f + 0.f : kNegInf;
  const uint32_t b = __float_as_uint(f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float load_logit(const void* p, int kind, int64_t i) {
  if (kind == OUT_F32) return static_cast<const float*>(p)[i];
  if (kind == OUT_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(kAll, v, d));
  return v;
}

// What turns a token's logits (NaN read as minus infinity) into scores.  A masked
// expert (minus infinity) scores 0; a row with nothing else scores 0 throughout.
struct Scorer {
  int sigmoid;
  float top, sum;  // softmax: largest logit, sum of exp(x - top)
  template <int P>
  __device__ __forceinline__ Scorer(const RouteArgs& a, const float (&x)[P]) : sigmoid(a.sigmoid), top(kNegInf), sum(0.f) {
    if (sigmoid) return;
#pragma unroll
    for (int i = 0; i < P; ++i) top = fmaxf(top, x[i]);
    top = key_value(__reduce_max_sync(kAll, order_key(top)));
#pragma unroll
    for (int i = 0; i < P; ++i) sum = __fadd_rn(sum, power(x[i]));
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

// Logit e of token t, NaN and what is not there as minus infinity.
__device__ __forceinline__ float logit(const RouteArgs& a, int t, int e) {
  if (e < 0 || e >= a.experts) return kNegInf;
  const int64_t at = int64_t(t) * a.ldl + e;
  if (!DG_IN(a.dbg, static_cast<const char*>(a.logits) + at * (a.kind == OUT_F32 ? 4 : 2), a.kind == OUT_F32 ? 4 : 2,
             DBG_ROUTE))
    return kNegInf;
  const float f = load_logit(a.logits, a.kind, at);
  return f == f ? f : kNegInf;
}

template <int P>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int t, int lane, float (&x)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = logit(a, t, 32 * i + lane);
}

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

// The warp's best expert, whose lane then moves on to its next one: the largest key, and
// among equal ones the lowest expert (lanes that have it are compared only if there are several).
template <int P>
__device__ __forceinline__ int take_best(uint32_t (&key)[P], int (&ex)[P], int lane) {
  const uint32_t best = __reduce_max_sync(kAll, key[0]);
  const uint32_t who = __ballot_sync(kAll, key[0] == best);
  int expert;
  if (who & (who - 1))
    expert = int(__reduce_min_sync(kAll, key[0] == best ? uint32_t(ex[0]) : 0xffffffffu));
  else
    expert = __shfl_sync(kAll, ex[0], __ffs(who) - 1);
  if (lane == (expert & 31)) {
#pragma unroll
    for (int i = 0; i + 1 < P; ++i) key[i] = key[i + 1], ex[i] = ex[i + 1];
    key[P - 1] = kNone;
  }
  return expert;
}

// Two largest keys among the experts of group g.
template <int P>
__device__ __forceinline__ void group_best(const uint32_t (&key)[P], int lane, int per, int g, uint32_t* first,
                                           uint32_t* second) {
  uint32_t b1 = kNone, b2 = kNone;  // of this lane
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = 32 * i + lane;
    if (e >= g * per && e < (g + 1) * per) {
      b2 = max(b2, min(b1, key[i]));
      b1 = max(b1, key[i]);
    }
  }
  *first = __reduce_max_sync(kAll, b1);
  const uint32_t owner = __ballot_sync(kAll, b1 == *first);
  // the best may be there more than once: only one lane gives its own up
  *second = __reduce_max_sync(kAll, lane == __ffs(owner) - 1 ? b2 : b1);
}

template <int P>
__global__ void __launch_bounds__(128) route_kernel(const RouteArgs a) {
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (t >= a.tokens) return;
  float x[P];
  load_logits(a, t, lane, x);
  const Scorer scorer(a, x);
  uint32_t key[P];
  const bool by_logit = a.bias == nullptr && a.group_top == 1;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = 32 * i + lane;
    float k = x[i];
    if (!by_logit && k != kNegInf) {  // a masked expert stays minus infinity, whatever its bias
      k = scorer.score(k);
      if (e < a.experts && a.bias && DG_IN(a.dbg, a.bias + e, 4, DBG_ROUTE)) k = __fadd_rn(k, __ldg(a.bias + e));
    }
    key[i] = e < a.experts ? order_key(k) : kNone;
  }
  if (a.groups > 1) {
    // Lane g holds group g's key; lanes are ranked, ties to the lower group.
    const int per = a.experts / a.groups;
    uint32_t mine = kNone;
    for (int g = 0; g < a.groups; ++g) {
      uint32_t b1, b2;
      group_best(key, lane, per, g, &b1, &b2);
      uint32_t k = b1;
      if (a.group_top == 2 && b2 != kNone) k = order_key(__fadd_rn(key_value(b1), key_value(b2)));
      if (lane == g) mine = k;
    }
    uint32_t chosen = 0;  // bit g: group g is in
    for (int i = 0; i < a.top_groups; ++i) {
      const uint32_t best = __reduce_max_sync(kAll, mine);
      const uint32_t who = __ballot_sync(kAll, mine == best && lane < a.groups && !((chosen >> lane) & 1u));
      const int g = __ffs(who) - 1;
      if (g < 0) break;
      chosen |= 1u << g;
      if (lane == g) mine = kNone;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = 32 * i + lane;
      if (e < a.experts && !((chosen >> (e / per)) & 1u)) key[i] = kOutside;
    }
  }
  int ex[P];
#pragma unroll
  for (int i = 0; i < P; ++i) ex[i] = 32 * i + lane;
  sort_lane(key, ex);
  int expert = -1;  // lane j: choice j
  for (int j = 0; j < a.top_k; ++j) {
    const int e = take_best(key, ex, lane);
    if (lane == j) expert = e;
  }
  // the chosen ones' scores, from their logits again (a few loads that hit L1)
  const float mine = logit(a, t, expert);
  float score = mine == kNegInf ? 0.f : scorer.score(mine);
  if (a.renormalize) {
    float sum = 0.f;
    for (int j = 0; j < a.top_k; ++j) sum = __fadd_rn(sum, __shfl_sync(kAll, score, j));
    score = sum > 0.f ? __fdiv_rn(score, sum) : 0.f;
  }
  if (lane < a.top_k) {
    const int64_t at = int64_t(t) * a.top_k + lane;
    if (DG_IN(a.dbg, a.weights + at, 4, DBG_ROUTE)) a.weights[at] = __fmul_rn(score, a.scale);
    if (DG_IN(a.dbg, a.indices + at, 4, DBG_ROUTE)) a.indices[at] = expert;
  }
}

// With S = the chosen scores' sum, w_j = scale s_j / S (or scale s_j):
//   ds_j = scale (dw_j - sum_i dw_i s_i / S) / S   (or scale dw_j)
//   dx_i = s_i (ds_i - sum_j ds_j s_j) (softmax), s_i (1 - s_i) ds_i (sigmoid).
// The scores are computed again from the logits: reading them costs what reading kept scores would.
template <int P>
__global__ void __launch_bounds__(128) route_backward_kernel(const RouteArgs a) {
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int t = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (t >= a.tokens) return;
  float x[P], ds[P];
  load_logits(a, t, lane, x);
  const Scorer scorer(a, x);
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
  float dsj = a.scale * dw;
  if (a.renormalize) {
    const float sum = warp_sum(sj);
    const float dot = warp_sum(dw * sj);
    dsj = sum > 0.f && expert >= 0 ? a.scale * (dw - dot / sum) / sum : 0.f;
  }
  const float through = warp_sum(dsj * sj);
#pragma unroll
  for (int i = 0; i < P; ++i) ds[i] = 0.f;
  for (int j = 0; j < a.top_k; ++j) {
    const int e = __shfl_sync(kAll, expert, j);
    const float d = __shfl_sync(kAll, dsj, j);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (e == 32 * i + lane) ds[i] += d;
  }
  const int es = a.kind == OUT_F32 ? 4 : 2;
  const float over = scorer.sum > 0.f ? 1.f / scorer.sum : 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = 32 * i + lane;
    if (e >= a.experts) continue;
    float d = 0.f;
    if (!a.sigmoid) {
      d = scorer.power(x[i]) * over * (ds[i] - through);
    } else if (ds[i] != 0.f) {  // (experts that were not chosen)
      const float s = scorer.score(x[i]);
      d = s * (1.f - s) * ds[i];
    }
    char* const dst = static_cast<char*>(a.dlogits) + (int64_t(t) * a.lddl + e) * es;
    if (!DG_IN(a.dbg, dst, es, DBG_ROUTE)) continue;
    if (a.kind == OUT_F32)
      *reinterpret_cast<float*>(dst) = d;
    else if (a.kind == OUT_BF16)
      *reinterpret_cast<__nv_bfloat16*>(dst) = __float2bfloat16_rn(d);
    else
      *reinterpret_cast<__half*>(dst) = __float2half_rn(d);
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
// A stable counting sort of the slots (token * top_k + choice) by expert, in one launch:
// a cluster of up to eight CTAs, each with a run of the slots, each warp with a run of
// its CTA's.  A warp counts its slots by expert (lanes with the same expert find each
// other with match, one of them adds), CTAs read each other's totals through
// distributed shared memory, and a second walk over the slots hands out rows:
// start of the expert + slots of earlier CTAs, warps and lanes (the place within the warp is
// kept in pos between the walks).  No atomics: the order is the slots' own.
constexpr int kMapThreads = 1024;
constexpr int kAhead = 8;  // loads of a warp's slots that are in flight together

// ints: four tables over the experts (this CTA's slots, all slots, slots of earlier
// CTAs, first row), then a count for each warp and expert
__host__ __device__ constexpr int map_ints(int experts, int warps) { return experts * (4 + warps) + 1; }

__global__ void __launch_bounds__(kMapThreads) route_map_kernel(const RouteMapArgs a, int ctas, int warps) {
  namespace cg = cooperative_groups;
  extern __shared__ int map_shared[];
  wait_prior_grid();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = ctas > 1 ? int(cluster.block_rank()) : 0;
  const int E = a.experts;
  int* const total = map_shared;
  int* const all = total + E;
  int* const before = all + E;
  int* const start = before + E;     // E + 1: [E] is the end of the last expert's rows
  int* const count = start + E + 1;  // [warps][E]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < E * warps; i += kMapThreads) count[i] = 0;
  // every row holds no slot, until its slot says otherwise (after the barriers below)
  for (int r = 4 * (rank * kMapThreads + int(threadIdx.x)); r < a.rows; r += 4 * ctas * kMapThreads) {
    const int n = min(4, a.rows - r);
    if (!DG_IN(a.dbg, a.rowmap + r, 4 * n, DBG_ROUTE)) continue;
    if (n == 4 && a.wide)
      *reinterpret_cast<int4*>(a.rowmap + r) = make_int4(-1, -1, -1, -1);
    else
      for (int i = 0; i < n; ++i) a.rowmap[r + i] = -1;
  }
  __syncthreads();
  // this warp's run of slots: a multiple of 32 (warps past `warps` have none)
  const int runs = ctas * warps;
  const int run = ((a.slots + runs - 1) / runs + 31) & ~31;
  const int64_t first = warp < warps ? int64_t(rank * warps + warp) * run : a.slots;
  const int64_t last = min(int64_t(a.slots), first + run);
  int* const mine = count + warp * E;
  auto expert_of = [&](int64_t slot) {
    if (slot >= last || !DG_IN(a.dbg, a.indices + slot, 4, DBG_ROUTE)) return -1;
    const int e = __ldg(a.indices + slot);
    return e >= 0 && e < E ? e : -1;
  };
  // first walk: a slot's place among its warp's slots of its expert, kept in pos
  for (int64_t s = first; s < last; s += 32 * kAhead) {
    int e[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) e[i] = expert_of(s + 32 * i + lane);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t slot = s + 32 * i + lane;
      const uint32_t same = __match_any_sync(kAll, e[i]);
      const int earlier = e[i] >= 0 ? mine[e[i]] : 0;
      __syncwarp();
      if (e[i] >= 0 && lane == __ffs(same) - 1) mine[e[i]] = earlier + __popc(same);
      __syncwarp();
      if (slot < last && DG_IN(a.dbg, a.pos + slot, 4, DBG_ROUTE))
        a.pos[slot] = earlier + __popc(same & ((1u << lane) - 1u));
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kMapThreads) {  // counts -> slots of earlier warps
    int sum = 0;
    for (int w = 0; w < warps; ++w) {
      const int n = count[w * E + e];
      count[w * E + e] = sum;
      sum += n;
    }
    total[e] = sum;
  }
  if (ctas > 1)
    cluster.sync();
  else
    __syncthreads();
  for (int e = threadIdx.x; e < E; e += kMapThreads) {
    int earlier = 0, sum = 0;
    for (int c = 0; c < ctas; ++c) {
      const int n = ctas > 1 ? *cluster.map_shared_rank(total + e, c) : total[e];
      if (c < rank) earlier += n;
      sum += n;
    }
    before[e] = earlier;
    all[e] = sum;
  }
  __syncthreads();
  if (warp == 0) {  // first rows: whole 128s of the experts before
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < E ? (all[e] + 127) & ~127 : 0;
      int sum = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kAll, sum, d);
        if (lane >= d) sum += o;
      }
      if (e < E) {
        start[e] = carry + sum - n;
        if (rank == 0 && DG_IN(a.dbg, a.starts + e, 4, DBG_ROUTE)) a.starts[e] = carry + sum - n;
        if (rank == 0 && DG_IN(a.dbg, a.counts + e, 4, DBG_ROUTE)) a.counts[e] = all[e];
      }
      carry += __shfl_sync(kAll, sum, 31);
    }
  }
  __syncthreads();
  // second walk: rows of this warp's slots
  for (int64_t s = first; s < last; s += 32 * kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t slot = s + 32 * i + lane;
      const int e = expert_of(slot);
      if (slot >= last || !DG_IN(a.dbg, a.pos + slot, 4, DBG_ROUTE)) continue;
      const int row = e >= 0 ? start[e] + before[e] + mine[e] + a.pos[slot] : -1;
      a.pos[slot] = row;
      if (row >= 0 && row < a.rows && DG_IN(a.dbg, a.rowmap + row, 4, DBG_ROUTE)) a.rowmap[row] = int(slot);
    }
  }
  if (ctas > 1) cluster.sync();  // no CTA leaves while another may still read its totals
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

cudaError_t launch_route_map(const RouteMapArgs& a, cudaStream_t s) {
  // 4096 slots a CTA, up to the portable cluster size
  const int ctas = std::max(1, std::min(8, (a.slots + 4095) / 4096));
  const int warps = std::max(1, std::min(kMapThreads / 32, (a.slots / ctas + 31) / 32));
  const int smem = map_ints(a.experts, warps) * 4;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaGetLastError();
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit == 0 || (ready.load(std::memory_order_acquire) & bit) == 0) {
    const cudaError_t err = cudaFuncSetAttribute(route_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 map_ints(ROUTE_MAX_EXPERTS, kMapThreads / 32) * 4);
    if (err != cudaSuccess) return err;
    ready.fetch_or(bit, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kMapThreads);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  attr[n].id = cudaLaunchAttributeClusterDimension;
  attr[n].val.clusterDim.x = unsigned(ctas);
  attr[n].val.clusterDim.y = 1;
  attr[n].val.clusterDim.z = 1;
  ++n;
  if (a.pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, route_map_kernel, a, ctas, warps);
}

}  // namespace dg
