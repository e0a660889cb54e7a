// balance.cu -- how evenly a router's choice spreads the tokens, and the gradient of the loss that keeps it even.
//
// With p[t, e] token t's share of expert e (softmax of its logits, or its sigmoids over their sum), over the m
// tokens that have a choice, n choices in all, c[e] of them expert e's:
//
//   P[e] = sum over t of p[t, e] / m      loss = scale E sum over e of (c[e] / n) P[e]
//   factor[e] = d loss / d p[t, e] = scale E c[e] / (n m)
//   d loss / d x[t, i] = p[t, i] (factor[i] - sum over e of factor[e] p[t, e]), for sigmoids times 1 - s[t, i]
//
// What bounds it is reading the logits once, for few tokens latency.  One warp a token, a run of experts a lane, as
// in the router (route.cuh): lanes keep the sums of their experts' shares from token to token, warps add theirs up
// in shared memory in a fixed order, CTAs through plan workspace, where the last one to arrive adds them in the
// order of their indices; counts are whole numbers, which may meet in any order.  The same bits every time.
// Measured: 16 tokens of 256 experts 3.5 us; 16384 of 128 9.3 us (while it took 10.5, the tokens were 4.8 of it, the parts and
// the count of those that are done 1.6 and the last CTA's sum 4); the gradient 5.3 us.
#include <algorithm>

#include "route.cuh"

namespace dg {
namespace {

// Warps of a CTA of the sums at most: with 16 or 32 experts a lane as many as there are registers for.
template <int P>
__host__ __device__ constexpr int balance_warps() {
  return P <= 8 ? 32 : 16;
}

// The lane's choice of the token's, -1 for none.
__device__ __forceinline__ int choice(const BalanceArgs& a, int t, int lane) {
  if (lane >= a.top_k) return -1;
  const int* const at = a.indices + int64_t(t) * a.top_k + lane;
  const int e = DG_IN(a.dbg, at, 4, DBG_ROUTE) ? __ldg(at) : -1;
  return e >= 0 && e < a.experts ? e : -1;
}

// A lane's experts' shares of a token, from its logits, the largest of which (of the token's) is `top`.  Masked experts
// (minus infinity) have none, a token of nothing else none at all; of logits of plus infinity (softmax) each takes an equal share.
// Sigmoids are taken times exp(-c), c = min(top, 0): 1 / (exp(c) + exp(c - x)), whose largest is 1/2 at least, so that a token
// whose sigmoids are all tiny, or 0 in fp32, has the shares that their ratio gives.
template <int P>
__device__ __forceinline__ void token_shares(const BalanceArgs& a, const float (&x)[P], float top, float (&p)[P]) {
  float sum = 0.f;
  if (a.sigmoid) {
    const float c = top == kNegInf ? 0.f : fminf(top, 0.f), ec = expf(c);
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = __fdividef(1.f, ec + expf(c - x[i]));  // (0 where exp(c - x) is past 2^126)
  } else if (fabsf(top) < -kNegInf) {  // exp(-inf) is 0: nothing to look out for
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = expf(x[i] - top);
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = x[i] == top && top > 0.f ? 1.f : 0.f;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) sum += p[i];
  sum = warp_sum(sum);
  const float by = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) p[i] *= by;
}

// What bounds few tokens, and half of the time of many, is the chain behind the last token, so it has few barriers: the
// warps' sums side by side in shared memory, a thread an expert adds them up; the choices' number and the loss's sum in one
// reduction.
template <int P>
__global__ void __launch_bounds__(32 * balance_warps<P>(), 1) balance_kernel(const BalanceArgs a) {
  constexpr int W = balance_warps<P>(), E = 32 * P;
  constexpr int ROWS = W * E <= 8192 ? W : 8192 / E;  // warps whose sums shared memory takes at once: all, or half
  __shared__ float room[ROWS * E];
  __shared__ int count[E];
  __shared__ int tokens;
  __shared__ float loss_sums[W];
  __shared__ int n_sums[W];
  __shared__ unsigned ticket;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int threads = int(blockDim.x), warps = threads >> 5;
  const int run = (a.experts + 31) / 32, first = lane * run;
  for (int e = threadIdx.x; e < E; e += threads) count[e] = 0;
  if (threadIdx.x == 0) tokens = 0;
  __syncthreads();
  wait_prior_grid();
  float acc[P];
#pragma unroll
  for (int i = 0; i < P; ++i) acc[i] = 0.f;
  int mine = 0;
  for (int64_t t = int64_t(blockIdx.x) * warps + warp; t < a.tokens; t += int64_t(gridDim.x) * warps) {
    float x[P], p[P];
    load_logits(a, int(t), first, run, a.wide, x);
    const int expert = choice(a, int(t), lane);
    if (!__any_sync(kAll, expert >= 0)) continue;
    if (expert >= 0) atomicAdd(count + expert, 1);
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < P; ++i) top = fmaxf(top, x[i]);
    top = key_value(__reduce_max_sync(kAll, number_key(top)));
    token_shares(a, x, top, p);
    ++mine;
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i] += p[i];
  }
  if (lane == 0 && mine) atomicAdd(&tokens, mine);
  auto put = [&](int row) {  // expert first + i of lane `lane`
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (i < run) room[row * E + first + i] = acc[i];
  };
  if constexpr (ROWS < W) {  // the upper half's sums to the lower half
    if (warp >= ROWS) put(warp - ROWS);
    __syncthreads();
    if (warp < ROWS && warp + ROWS < warps) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (i < run) acc[i] += room[warp * E + first + i];
    }
    __syncthreads();
  }
  if (warp < ROWS) put(warp);
  __syncthreads();
  int lots = min(ROWS, warps), stride = E;  // where the sums lie
  auto sum_of = [&](int e) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};  // (in eight chains: an order that depends on the sizes alone)
    int l = 0;
    for (; l + 8 <= lots; l += 8)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += room[(l + j) * stride + e];
    for (int j = 0; l < lots; ++l, ++j) v[0] += room[l * stride + e];
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
  };
  if (gridDim.x > 1) {
    float* const part = a.parts + int64_t(blockIdx.x) * a.experts;
    for (int e = threadIdx.x; e < a.experts; e += threads) {
      if (DG_IN(a.dbg, part + e, 4, DBG_ROUTE)) part[e] = sum_of(e);
      if (count[e] && DG_IN(a.dbg, a.counters + 2 + e, 4, DBG_ROUTE)) atomicAdd(a.counters + 2 + e, unsigned(count[e]));
    }
    if (threadIdx.x == 0 && DG_IN(a.dbg, a.counters + 1, 4, DBG_ROUTE)) atomicAdd(a.counters + 1, unsigned(tokens));
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) ticket = DG_IN(a.dbg, a.counters, 4, DBG_ROUTE) ? atomicAdd(a.counters, 1u) : 0u;
    __syncthreads();
    if (ticket != gridDim.x - 1) return;
    __threadfence();
    for (int e = threadIdx.x; e < a.experts; e += threads) {
      if (!DG_IN(a.dbg, a.counters + 2 + e, 4, DBG_ROUTE)) continue;
      count[e] = int(__ldcg(a.counters + 2 + e));
      a.counters[2 + e] = 0u;
    }
    if (threadIdx.x == 0) {
      tokens = int(__ldcg(a.counters + 1));
      a.counters[0] = a.counters[1] = 0u;
    }
    // the parts: every lots-th CTA's to a lot, a thread a lot of an expert; then the lots in their order
    lots = max(1, min(32, threads / a.experts));
    stride = a.experts;
    for (int i = threadIdx.x; i < lots * a.experts; i += threads) {
      const int e = i % a.experts, lot = i / a.experts;
      float s = 0.f;
      for (int c0 = lot; c0 < int(gridDim.x); c0 += 10 * lots) {  // (ten loads together, whatever is left)
        float v[10];
#pragma unroll
        for (int j = 0; j < 10; ++j) {
          const int c = c0 + j * lots;
          const float* const at = a.parts + int64_t(c) * a.experts + e;
          v[j] = c < int(gridDim.x) && DG_IN(a.dbg, at, 4, DBG_ROUTE) ? __ldcg(at) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 10; ++j) s += v[j];
      }
      room[i] = s;
    }
    __syncthreads();
  }
  // shares; n (whole numbers below 2^31) and the sum of counts times shares
  const float m = float(max(tokens, 1));
  int n = 0;
  float dot = 0.f;
  for (int e = threadIdx.x; e < a.experts; e += threads) {
    const float share = __fdiv_rn(sum_of(e), m);
    n += count[e];
    dot = fmaf(float(count[e]), share, dot);
    if (DG_IN(a.dbg, a.counts + e, 4, DBG_ROUTE)) a.counts[e] = count[e];
    if (DG_IN(a.dbg, a.shares + e, 4, DBG_ROUTE)) a.shares[e] = share;
  }
  const int active = min(warps, (a.experts + 31) / 32);  // warps that have experts
  if (warp < active) {
    n = __reduce_add_sync(kAll, n);
    dot = warp_sum(dot);
    if (lane == 0) n_sums[warp] = n, loss_sums[warp] = dot;
  }
  __syncthreads();
  n = 0;
  for (int w = 0; w < active; ++w) n += n_sums[w];
  const float by = __fdiv_rn(a.scale * float(a.experts), float(max(n, 1)));
  for (int e = threadIdx.x; e < a.experts; e += threads)
    if (DG_IN(a.dbg, a.factor + e, 4, DBG_ROUTE)) a.factor[e] = __fdiv_rn(by * float(count[e]), m);
  if (threadIdx.x == 0 && DG_IN(a.dbg, a.loss, 4, DBG_ROUTE)) {
    dot = 0.f;
    for (int w = 0; w < active; ++w) dot += loss_sums[w];
    *a.loss = by * dot;
  }
}

// The difference factor[i] - sum of factor[e] p[e] is taken from the factor of the token's surest expert on, whose
// own term is then exactly 0: a nearly sure token keeps the digits of its small gradient.
template <int P>
__global__ void __launch_bounds__(128) balance_backward_kernel(const BalanceArgs a) {
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int t = int(blockIdx.x * 4 + (threadIdx.x >> 5));
  if (t >= a.tokens) return;
  const int run = (a.experts + 31) / 32, first = lane * run;
  float x[P], p[P], f[P], old[P];
  load_logits(a, t, first, run, a.wide, x);
  const bool live = __any_sync(kAll, choice(a, t, lane) >= 0);
  const float dloss = a.dloss == nullptr ? 1.f : DG_IN(a.dbg, a.dloss, 4, DBG_ROUTE) ? __ldg(a.dloss) : 0.f;
  const int es = a.kind == OUT_F32 ? 4 : 2;
  char* const dst = static_cast<char*>(a.dlogits) + (int64_t(t) * a.lddl + first) * es;
  const bool whole = P >= 4 && a.wide_out && run == P && first + P <= a.experts;
  auto have = [&](int i) { return i < run && first + i < a.experts; };
  bool by_four = false;
  if constexpr (P >= 4) {
    by_four = whole && (reinterpret_cast<uintptr_t>(a.factor) & 15) == 0 && DG_IN(a.dbg, a.factor + first, 4 * P, DBG_ROUTE);
    if (by_four) {
#pragma unroll
      for (int i = 0; i < P; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(a.factor + first + i));
        f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
      }
    }
  }
  if (!by_four) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      f[i] = have(i) && DG_IN(a.dbg, a.factor + first + i, 4, DBG_ROUTE) ? __ldg(a.factor + first + i) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) old[i] = 0.f;
  if (a.accumulate) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (have(i) && DG_IN(a.dbg, dst + i * es, es, DBG_ROUTE))
        old[i] = es == 4 ? *reinterpret_cast<const float*>(dst + 4 * i)
                         : half_at(*reinterpret_cast<const uint16_t*>(dst + 2 * i), 0, a.kind);
  }
  float top = kNegInf, reference = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (x[i] > top) top = x[i], reference = f[i];
  const uint32_t key = number_key(top), best = __reduce_max_sync(kAll, key);
  token_shares(a, x, key_value(best), p);
  reference = __shfl_sync(kAll, reference, __ffs(__ballot_sync(kAll, key == best)) - 1);
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    f[i] -= reference;
    dot = fmaf(f[i], p[i], dot);
  }
  dot = warp_sum(dot);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float d = p[i] * (f[i] - dot);
    if (a.sigmoid) d = x[i] == kNegInf ? 0.f : __fdiv_rn(d, __fadd_rn(1.f, expf(x[i])));
    x[i] = live ? fmaf(dloss, d, old[i]) : old[i];
  }
  if constexpr (P >= 4) {
    if (whole) {
      if (!DG_IN(a.dbg, dst, P * es, DBG_ROUTE)) return;
#pragma unroll
      for (int i = 0; i < P; i += 4) {
        if (a.kind == OUT_F32)
          *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        else
          *reinterpret_cast<uint2*>(dst + 2 * i) = make_uint2(half_pair(x[i], x[i + 1], a.kind), half_pair(x[i + 2], x[i + 3], a.kind));
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if (!have(i) || !DG_IN(a.dbg, dst + i * es, es, DBG_ROUTE)) continue;
    if (es == 4)
      *reinterpret_cast<float*>(dst + 4 * i) = x[i];
    else
      *reinterpret_cast<uint16_t*>(dst + 2 * i) = uint16_t(half_pair(x[i], 0.f, a.kind));
  }
}

}  // namespace

static int warps_for(int64_t experts) { return experts <= 256 ? 32 : 16; }

// CTAs of the sums: one warp a token until every SM has a CTA.  (Two an SM, half the tokens a warp: 13.1 instead of 11.0 us for 16384
// tokens of 128 experts, twice the parts.)
int balance_ctas(int64_t tokens, int64_t experts, int sms) {
  const int64_t warps = warps_for(experts);
  return int(std::max<int64_t>(1, std::min<int64_t>(sms, (tokens + warps - 1) / warps)));
}

cudaError_t launch_balance(const BalanceArgs& a, int ctas, cudaStream_t s) {
  // (no more warps than tokens, but four)
  const int warps = std::max(4, std::min(warps_for(a.experts), a.tokens));
  return by_experts(a.experts, [&](auto p) {
    constexpr int P = decltype(p)::value;
    return launch_k(balance_kernel<P>, dim3(unsigned(ctas)), dim3(unsigned(32 * warps)), 0, s, a.pdl, a);
  });
}

cudaError_t launch_balance_backward(const BalanceArgs& a, cudaStream_t s) {
  return by_experts(a.experts, [&](auto p) {
    return launch_k(balance_backward_kernel<decltype(p)::value>, dim3(unsigned((a.tokens + 3) / 4)), dim3(128), 0, s, a.pdl, a);
  });
}

}  // namespace dg
