// norm_ops.cpp -- the C ABI of the norm and its gradients (include/gemm.h): argument checks and launches.
#include "gemm.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <utility>

#include "ops.h"

using namespace dg;

namespace {

// A result that takes an input's own place: a lane reads its columns of a row before it writes them.
bool in_place(const void* out, int64_t ldo, gemm_type_t to, const void* in, int64_t ldi, gemm_type_t ti) {
  return out && out == in && ldo == ldi && to == ti;
}

// Bytes of loads and stores that each matrix's address (none: anything) and bytes between rows allow: 16, 4 or 0.
int access_of(std::initializer_list<std::pair<const void*, int64_t>> rows) {
  int wide = 16;
  for (const auto& m : rows)
    while (m.first && wide && (!aligned(m.first, size_t(wide)) || m.second % wide)) wide = wide == 16 ? 4 : 0;
  return wide;
}

// x_type and h_type, the sizes and the gain.
gemm_status_t check_norm(int64_t rows, int64_t cols, gemm_type_t x_type, gemm_type_t h_type, const void* gain, gemm_type_t g_type) {
  if (rows < 0 || cols < 0 || !is_float_type(x_type) || (h_type != x_type && h_type != GEMM_TYPE_F32)) return GEMM_ERR_INVALID_ARG;
  if (gain && g_type != x_type && g_type != GEMM_TYPE_F32) return GEMM_ERR_INVALID_ARG;
  if (!size_ok(rows) || cols > NORM_MAX_COLS) return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_status_t gemm_norm(gemm_plan_t plan, int64_t rows, int64_t cols, const void* X, int64_t ldx, gemm_type_t x_type,
                        const void* residual, int64_t ldr, gemm_type_t h_type, const void* gain, gemm_type_t g_type,
                        float eps, void* H, int64_t ldh, void* Y, int64_t ldy, gemm_type_t q_type, void* Q, int64_t ldq,
                        void* SQ, float* rstd, void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t st = check_norm(rows, cols, x_type, h_type, gain, g_type);
  if (st != GEMM_OK) return st;
  if (!(eps >= 0.f) || std::isinf(eps) || (Q == nullptr) != (SQ == nullptr) || (Q && !is_code_type(q_type)) ||
      (!H && !Y && !Q && !rstd))
    return GEMM_ERR_INVALID_ARG;
  const int64_t width = std::max<int64_t>(1, cols);
  if (ldx < width || (residual && ldr < width) || (H && ldh < width) || (Y && ldy < width) || (Q && ldq < width))
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (!X) return GEMM_ERR_INVALID_ARG;
  const int64_t xe = type_bytes(x_type), he = type_bytes(h_type), ge = gain ? type_bytes(g_type) : 1;
  if (!aligned(X, size_t(xe)) || !aligned(residual, size_t(he)) || !aligned(gain, size_t(ge)) || !aligned(H, size_t(he)) ||
      !aligned(Y, size_t(xe)) || !aligned(Q, 16) || !aligned(SQ, 16) || (Q && ldq % 16) || !aligned(rstd, 4))
    return GEMM_ERR_ALIGNMENT;
  const bool over_x = in_place(H, ldh, h_type, X, ldx, x_type) || in_place(Y, ldy, x_type, X, ldx, x_type);
  const bool over_r = in_place(H, ldh, h_type, residual, ldr, h_type) || in_place(Y, ldy, x_type, residual, ldr, h_type);
  const int64_t sq = Q ? scale_tiles(rows, cols) * 512 : 0;
  if (results_meet({region(H, H ? rows : 0, cols, ldh, he), region(Y, Y ? rows : 0, cols, ldy, xe),
                    region(Q, Q ? rows : 0, cols, ldq, 1), run_of(SQ, sq), run_of(rstd, rows * 4)},
                   {region(X, over_x ? 0 : rows, cols, ldx, xe), region(residual, residual && !over_r ? rows : 0, cols, ldr, he),
                    run_of(gain, cols * ge)}))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_norm %lldx%lld %s%s%s%s%s%s", (long long)rows, (long long)cols, type_name(x_type),
                       residual ? " residual" : "", H ? " H" : "", Y ? " Y" : "", Q ? " Q " : "", Q ? type_name(q_type) : "");
  DeviceGuard guard(plan->device);
  NormArgs a{};
  a.rows = int(rows);
  a.cols = int(cols);
  a.x = X;
  a.ldx = ldx;
  a.x_kind = type_kind(x_type);
  a.r = residual;
  a.ldr = ldr;
  a.h_kind = type_kind(h_type);
  a.gain = gain;
  a.g_kind = type_kind(g_type);
  a.eps = eps;
  a.h = H;
  a.ldh = ldh;
  a.y = Y;
  a.ldy = ldy;
  a.q = static_cast<uint8_t*>(Q);
  a.sq = static_cast<uint8_t*>(SQ);
  a.ldq = ldq;
  a.e5m2 = q_type == GEMM_TYPE_E5M2;
  a.q_groups = int(scale_groups(cols));
  a.rows_padded = int(std::min<int64_t>(round_up(rows, 128), kMaxDim));
  a.rstd = rstd;
  a.wide = access_of({{X, ldx * xe}, {residual, ldr * he}, {H, ldh * he}, {Y, ldy * xe}, {gain, 0}});
  a.pdl = plan->pdl;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(X, rows, cols, ldx, xe).matrix(residual, residual ? rows : 0, cols, ldr, he)
              .bytes(gain, gain ? cols * ge : 0).matrix(H, H ? rows : 0, cols, ldh, he).out_matrix(Y, Y ? rows : 0, cols, ldy, xe)
              .matrix(Q, Q ? rows : 0, cols, ldq, 1).bytes(SQ, sq).bytes(rstd, rstd ? rows * 4 : 0).s;
#endif
  return call.done(launched(launch_norm(a, plan->sms, static_cast<cudaStream_t>(stream))));
}

gemm_status_t gemm_norm_backward(gemm_plan_t plan, int64_t rows, int64_t cols, const void* dY, int64_t lddy,
                                 gemm_type_t x_type, const void* H, int64_t ldh, gemm_type_t h_type, const void* gain,
                                 gemm_type_t g_type, const float* rstd, const void* dH, int64_t lddh, void* dX, int64_t lddx,
                                 float* dgain, void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  const gemm_status_t st = check_norm(rows, cols, x_type, h_type, gain, g_type);
  if (st != GEMM_OK) return st;
  const int64_t width = std::max<int64_t>(1, cols);
  if (lddy < width || ldh < width || (dH && lddh < width) || lddx < width) return GEMM_ERR_INVALID_ARG;
  if (cols == 0 || (rows == 0 && !dgain)) return GEMM_OK;
  if (rows > 0 && (!dY || !H || !rstd || !dX)) return GEMM_ERR_INVALID_ARG;
  const int64_t xe = type_bytes(x_type), he = type_bytes(h_type), ge = gain ? type_bytes(g_type) : 1;
  if (!aligned(dY, size_t(xe)) || !aligned(H, size_t(he)) || !aligned(gain, size_t(ge)) || !aligned(rstd, 4) ||
      !aligned(dH, size_t(he)) || !aligned(dX, size_t(he)) || !aligned(dgain, 4))
    return GEMM_ERR_ALIGNMENT;
  const bool over_dy = in_place(dX, lddx, h_type, dY, lddy, x_type), over_dh = in_place(dX, lddx, h_type, dH, lddh, h_type);
  if (results_meet({region(dX, rows, cols, lddx, he), run_of(dgain, cols * 4)},
                   {region(H, rows, cols, ldh, he), run_of(gain, cols * ge), run_of(rstd, rows * 4)}) ||
      (!over_dy && overlaps(region(dX, rows, cols, lddx, he), region(dY, rows, cols, lddy, xe))) ||
      (dH && !over_dh && overlaps(region(dX, rows, cols, lddx, he), region(dH, rows, cols, lddh, he))) ||
      overlaps(run_of(dgain, cols * 4), region(dY, rows, cols, lddy, xe)) ||
      (dH && overlaps(run_of(dgain, cols * 4), region(dH, rows, cols, lddh, he))))
    return GEMM_ERR_INVALID_ARG;
  const CallScope call(plan, "gemm_norm_backward %lldx%lld %s%s%s", (long long)rows, (long long)cols, type_name(x_type),
                       dH ? " dH" : "", dgain ? " dgain" : "");
  DeviceGuard guard(plan->device);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = norm_backward_grid(type_kind(x_type), type_kind(h_type), rows, cols, plan->sms);
  const size_t ws = dgain ? size_t(grid) * size_t(norm_part_cols(cols)) * 4 : 0;
  if (ws > 0) {
    const gemm_status_t grown = ensure_ws(plan, ws, s);
    if (grown != GEMM_OK) return grown;
  }
  NormBackArgs a{};
  a.rows = int(rows);
  a.cols = int(cols);
  a.dy = dY;
  a.lddy = lddy;
  a.x_kind = type_kind(x_type);
  a.h = H;
  a.ldh = ldh;
  a.h_kind = type_kind(h_type);
  a.gain = gain;
  a.g_kind = type_kind(g_type);
  a.rstd = rstd;
  a.dh = dH;
  a.lddh = lddh;
  a.dx = dX;
  a.lddx = lddx;
  a.dgain = dgain;
  a.parts = static_cast<float*>(plan->ws);
  a.wide = access_of({{dY, lddy * xe}, {H, ldh * he}, {dH, lddh * he}, {dX, lddx * he}, {gain, 0}});
  a.pdl = plan->pdl;
#ifdef DG_DEBUG
  a.dbg = Spans(plan->err).matrix(dY, rows, cols, lddy, xe).matrix(H, rows, cols, ldh, he).bytes(gain, gain ? cols * ge : 0)
              .bytes(rstd, rows * 4).matrix(dH, dH ? rows : 0, cols, lddh, he).out_matrix(dX, rows, cols, lddx, he)
              .bytes(dgain, dgain ? cols * 4 : 0).bytes(plan->ws, int64_t(ws)).s;
#endif
  return call.done(launched(launch_norm_backward(a, grid, s)));
}

}  // extern "C"
