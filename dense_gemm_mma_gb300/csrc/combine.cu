// combine.cu -- the experts' rows back into tokens, and its gradients:
//
//   out[t] = sum_j w[t,j] Y[pos[t,j]]
//   dY[pos[t,j]] = w[t,j] dout[t]        dw[t,j] = <dout[t], Y[pos[t,j]]>
//
// Every row of Y belongs to one choice of one token, so the gradient of Y has one term
// and needs no atomics.  What bounds both is memory: each row of Y is read once (and of dY
// written once), each row of out or dout once.  16-byte loads, all k rows' of a piece in flight together.
// Measured, 8192 tokens of 4 rows of 2048 bf16: sum and gradients 79.6 us, 5.9 TB/s; of 1026 (4-byte loads) 73 us,
// of 1027 (by element; 2000 tokens) 16.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>
#include <type_traits>

#include "kernels.h"

namespace dg {
namespace {

constexpr uint32_t kAll = 0xffffffffu;
constexpr int kPiece = 8;   // columns of a thread

template <typename T>
__device__ __forceinline__ float to_f(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_f(float v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
  else return __float2bfloat16_rn(v);
}

template <typename T>
struct alignas(16) Piece {
  T v[kPiece];
};

// A warp takes 256 columns of a row at a time, a thread a piece of them.  WIDE, the bytes of a load:
//   16  eight neighbouring columns, rows on 16-byte boundaries, whole pieces: loads without a branch, so that the
//       pieces of all rows are in flight together
//   4   eight neighbouring columns, rows on 4-byte boundaries: a whole piece in words, the last one of a row by element
//   0   every 32nd column, so that a load of the warp is one run of memory
template <int WIDE>
struct Units {
  static constexpr int COLS = WIDE ? kPiece : 1;  // neighbouring columns of a thread
  static constexpr int STEP = WIDE ? 1 : 32;      // columns between values of a piece
  // Columns from a thread's first to its last, `left` in the row.
  static __device__ __forceinline__ int span(int left) { return min(left, (kPiece - 1) * STEP + 1); }
};

// A thread's piece, its first column at p, `left` columns from there to the end of the row; what does
// not exist is zero.
template <int WIDE, typename T>
__device__ __forceinline__ void load_piece(Piece<T>& o, const T* p, int left) {
#pragma unroll
  for (int i = 0; i < kPiece; ++i) o.v[i] = from_f<T>(0.f);
  if constexpr (WIDE == 16) {
    if (left > 0) o = *reinterpret_cast<const Piece<T>*>(p);
  } else if (WIDE == 4 && left >= kPiece) {
    uint32_t w[sizeof(Piece<T>) / 4];
#pragma unroll
    for (int i = 0; i < int(sizeof(w) / 4); ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    memcpy(&o, w, sizeof(w));
  } else {
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
      if (i * Units<WIDE>::STEP < left) o.v[i] = p[i * Units<WIDE>::STEP];
  }
}

template <int WIDE, typename T>
__device__ __forceinline__ void store_piece(const Piece<T>& o, T* p, int left) {
  if constexpr (WIDE == 16) {
    if (left > 0) *reinterpret_cast<Piece<T>*>(p) = o;
  } else if (WIDE == 4 && left >= kPiece) {
    uint32_t w[sizeof(Piece<T>) / 4];
    memcpy(w, &o, sizeof(w));
#pragma unroll
    for (int i = 0; i < int(sizeof(w) / 4); ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
      if (i * Units<WIDE>::STEP < left) p[i * Units<WIDE>::STEP] = o.v[i];
  }
}

__device__ __forceinline__ int row_of(const CombineArgs& a, int64_t slot) {
  if (!DG_IN(a.dbg, a.pos + slot, 4, DBG_COMBINE)) return -1;
  const int r = __ldg(a.pos + slot);
  return r < a.rows ? r : -1;  // negative: the choice has no row
}

// One thread a piece of a token's row.
template <typename TY, typename TO, int WIDE, int KC>
__global__ void __launch_bounds__(256) combine_kernel(const CombineArgs a) {
  wait_prior_grid();
  using U = Units<WIDE>;
  const int t = int(blockIdx.x), first = int(blockIdx.y * blockDim.x + threadIdx.x);
  const int col = first / 32 * (32 * kPiece) + first % 32 * U::COLS;
  const int left = a.cols - col;
  if (left <= 0) return;
  const int n = U::span(left);
  const TY* const y = static_cast<const TY*>(a.y) + col;
  float sum[kPiece];
#pragma unroll
  for (int i = 0; i < kPiece; ++i) sum[i] = 0.f;
  for (int j0 = 0; j0 < a.k; j0 += KC) {
    Piece<TY> p[KC];
    float w[KC];
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      const int64_t slot = int64_t(t) * a.k + j0 + j;
      const int r = j0 + j < a.k ? row_of(a, slot) : -1;
      const TY* const src = y + int64_t(max(r, 0)) * a.ldy;
      w[j] = r >= 0 && DG_IN(a.dbg, a.weights + slot, 4, DBG_COMBINE) ? __ldg(a.weights + slot) : 0.f;
      load_piece<WIDE>(p[j], src, r >= 0 && DG_IN(a.dbg, src, n * int(sizeof(TY)), DBG_COMBINE) ? left : 0);
    }
#pragma unroll
    for (int j = 0; j < KC; ++j)
#pragma unroll
      for (int i = 0; i < kPiece; ++i) sum[i] = fmaf(w[j], to_f(p[j].v[i]), sum[i]);
  }
  Piece<TO> o;
#pragma unroll
  for (int i = 0; i < kPiece; ++i) o.v[i] = from_f<TO>(sum[i]);
  TO* const dst = static_cast<TO*>(a.out) + int64_t(t) * a.ldo + col;
  if (DG_IN(a.dbg, dst, n * int(sizeof(TO)), DBG_COMBINE)) store_piece<WIDE>(o, dst, left);
}

// Gradients: WARPS warps a token (dout read once, its choices' rows side by side), each every
// WARPS-th 256 columns, their products added up in the warps' order; the warps after the
// tokens' clear the rows that hold no slot.
template <typename TY, typename TO, int WIDE, int KC, int WARPS>
__global__ void __launch_bounds__(256) combine_backward_kernel(const CombineArgs a) {
  using U = Units<WIDE>;
  __shared__ float part[WARPS > 1 ? WARPS : 1][KC];
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int share = WARPS > 1 ? int(threadIdx.x >> 5) : 0;  // this warp's part of the token's columns
  const int64_t index = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t warp = index / WARPS;  // (a whole CTA's warps have a token, or none has)
  if (warp >= a.tokens) {
    const int64_t r = index - int64_t(a.tokens) * WARPS;
    if (!a.rowmap || r >= a.rows || !DG_IN(a.dbg, a.rowmap + r, 4, DBG_COMBINE) || __ldg(a.rowmap + r) >= 0) return;
    Piece<TY> zero;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) zero.v[i] = from_f<TY>(0.f);
    TY* const dst = static_cast<TY*>(a.dy) + r * a.lddy;
    for (int col = lane * U::COLS; col < a.cols; col += 32 * kPiece) {
      const int left = a.cols - col;
      if (DG_IN(a.dbg, dst + col, U::span(left) * int(sizeof(TY)), DBG_COMBINE)) store_piece<WIDE>(zero, dst + col, left);
    }
    return;
  }
  const TO* const dout = static_cast<const TO*>(a.out) + warp * a.ldo;
  for (int j0 = 0; j0 < a.k; j0 += KC) {
    int row[KC];
    float w[KC], dot[KC];
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      const int64_t slot = warp * a.k + j0 + j;
      row[j] = j0 + j < a.k ? row_of(a, slot) : -1;
      // (a plain load: dweights may be the same array)
      w[j] = row[j] >= 0 && DG_IN(a.dbg, a.weights + slot, 4, DBG_COMBINE) ? a.weights[slot] : 0.f;
      dot[j] = 0.f;
    }
    for (int col = share * (32 * kPiece) + lane * U::COLS; col < a.cols; col += WARPS * 32 * kPiece) {
      const int left = a.cols - col, n = U::span(left);
      Piece<TO> g;
      load_piece<WIDE>(g, dout + col, DG_IN(a.dbg, dout + col, n * int(sizeof(TO)), DBG_COMBINE) ? left : 0);
      Piece<TY> y[KC];
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const TY* const src = static_cast<const TY*>(a.y) + int64_t(max(row[j], 0)) * a.ldy + col;
        load_piece<WIDE>(y[j], src, row[j] >= 0 && DG_IN(a.dbg, src, n * int(sizeof(TY)), DBG_COMBINE) ? left : 0);
      }
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        if (row[j] < 0) continue;
        Piece<TY> d;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
          const float f = to_f(g.v[i]);
          dot[j] = fmaf(f, to_f(y[j].v[i]), dot[j]);
          d.v[i] = from_f<TY>(w[j] * f);
        }
        TY* const dst = static_cast<TY*>(a.dy) + int64_t(row[j]) * a.lddy + col;
        if (DG_IN(a.dbg, dst, n * int(sizeof(TY)), DBG_COMBINE)) store_piece<WIDE>(d, dst, left);
      }
    }
#pragma unroll
    for (int j = 0; j < KC; ++j) {
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) dot[j] += __shfl_xor_sync(kAll, dot[j], s);
    }
    if constexpr (WARPS > 1) {
      if (j0 > 0) __syncthreads();  // the sums of the choices before have been read
#pragma unroll
      for (int j = 0; j < KC; ++j)
        if (lane == 0) part[share][j] = dot[j];
      __syncthreads();
      if (share > 0) continue;
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        dot[j] = 0.f;
        for (int w = 0; w < WARPS; ++w) dot[j] += part[w][j];
      }
    }
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      const int64_t slot = warp * a.k + j0 + j;
      if (lane == 0 && j0 + j < a.k && DG_IN(a.dbg, a.dweights + slot, 4, DBG_COMBINE)) a.dweights[slot] = dot[j];
    }
  }
}

// Tokens up to which the gradients take eight warps a token.  16-byte loads, 4 rows of 2048 bf16 a
// token: 20 tokens 3.7 us (one warp 7.1), 256 tokens 5.6 (7.4), 512 tokens 7.6 (7.4).  Narrower loads keep one warp busy for
// longer: 300 tokens of 7 rows of 1116, 6.9 us (one warp 15.1).
constexpr int few_tokens(int wide) { return wide == 16 ? 256 : 1024; }

template <typename TY, typename TO, int WIDE, int KC>
cudaError_t launch(const CombineArgs& a, bool backward, cudaStream_t s) {
  const int pieces = (a.cols + kPiece - 1) / kPiece;
  if (backward) {
    const bool few = a.tokens <= few_tokens(WIDE) && pieces > 32;
    const int64_t warps = int64_t(a.tokens) * (few ? 8 : 1) + (a.rowmap ? a.rows : 0);
    const dim3 grid(unsigned((warps + 7) / 8));
    if (few) return launch_k(combine_backward_kernel<TY, TO, WIDE, 8, 8>, grid, dim3(256), 0, s, a.pdl, a);
    return launch_k(combine_backward_kernel<TY, TO, WIDE, KC, 1>, grid, dim3(256), 0, s, a.pdl, a);
  }
  const int threads = pieces >= 256 ? 256 : (pieces + 31) / 32 * 32;
  return launch_k(combine_kernel<TY, TO, WIDE, KC>, dim3(unsigned(a.tokens), unsigned((pieces + threads - 1) / threads)),
                  dim3(unsigned(threads)), 0, s, a.pdl, a);
}

// KC, the choices of a token that are in flight together: its k rounded up, eight at most.
template <typename TY, typename TO>
cudaError_t launch_k_of(const CombineArgs& a, bool backward, cudaStream_t s) {
  if (a.wide == 0) return launch<TY, TO, 0, 4>(a, backward, s);
  if (a.wide == 4) return launch<TY, TO, 4, 4>(a, backward, s);
  if (a.k <= 2) return launch<TY, TO, 16, 2>(a, backward, s);
  if (a.k <= 4) return launch<TY, TO, 16, 4>(a, backward, s);
  return launch<TY, TO, 16, 8>(a, backward, s);
}

template <typename TY>
cudaError_t launch_y(const CombineArgs& a, bool backward, cudaStream_t s) {
  switch (a.o_kind) {
    case OUT_F32: return launch_k_of<TY, float>(a, backward, s);
    case OUT_BF16: return launch_k_of<TY, __nv_bfloat16>(a, backward, s);
    default: return launch_k_of<TY, __half>(a, backward, s);
  }
}

cudaError_t launch_any(const CombineArgs& a, bool backward, cudaStream_t s) {
  switch (a.y_kind) {
    case OUT_F32: return launch_y<float>(a, backward, s);
    case OUT_BF16: return launch_y<__nv_bfloat16>(a, backward, s);
    default: return launch_y<__half>(a, backward, s);
  }
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t s) { return launch_any(a, false, s); }
cudaError_t launch_combine_backward(const CombineArgs& a, cudaStream_t s) { return launch_any(a, true, s); }

}  // namespace dg
