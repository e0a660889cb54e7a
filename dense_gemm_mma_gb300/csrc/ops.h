// ops.h -- what the C entries of the operators share (ops.cpp, norm_ops.cpp): sizes of types and
// scales, the checks that results have memory of their own, log lines and profiler ranges.  Internal to the library.
#pragma once

#include "gemm.h"

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "plan.h"

namespace dg {

inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

inline bool is_float_type(gemm_type_t t) { return t == GEMM_TYPE_BF16 || t == GEMM_TYPE_F16 || t == GEMM_TYPE_F32; }
inline bool is_code_type(gemm_type_t t) { return t == GEMM_TYPE_E4M3 || t == GEMM_TYPE_E5M2; }
inline int64_t type_bytes(gemm_type_t t) { return t == GEMM_TYPE_F32 ? 4 : is_code_type(t) ? 1 : 2; }

inline bool size_ok(int64_t n) { return n >= 0 && n <= kMaxDim; }

// Scale tiles (512 bytes) of a rows x cols matrix.
inline int64_t scale_groups(int64_t cols) { return std::max<int64_t>(1, ceil_div(cols, 512)); }
inline int64_t scale_tiles(int64_t rows, int64_t cols) { return std::max<int64_t>(1, ceil_div(rows, 128)) * scale_groups(cols); }

// The same of a 4-bit matrix, whose tiles are 128 rows of four blocks of 32.
inline int64_t mx4_scale_tiles(int64_t rows, int64_t cols) {
  return std::max<int64_t>(1, ceil_div(rows, 128)) * std::max<int64_t>(1, ceil_div(cols, 128));
}

// Every operator's launch goes through here: errors of the launch become a status.
inline gemm_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return GEMM_OK;
  cudaGetLastError();
  return GEMM_ERR_CUDA;
}

inline const char* type_name(gemm_type_t t) {
  static const char* kName[] = {"bf16", "f16", "f32", "tf32", "e4m3", "e5m2"};
  return int(t) >= 0 && int(t) < 6 ? kName[int(t)] : "?";
}

// A call under GEMM_NVTX (a range named after it, closed on every return) and GEMM_LOG (one line when it
// has succeeded).
class CallScope {
 public:
  CallScope(const gemm_plan* plan, const char* format, ...) __attribute__((format(printf, 3, 4)))
      : log_(plan->log), nvtx_(plan->nvtx) {
    if (!log_ && !nvtx_) return;
    va_list args;
    va_start(args, format);
    std::vsnprintf(text_, sizeof text_, format, args);
    va_end(args);
    if (nvtx_) nvtxRangePushA(text_);
  }
  CallScope(const CallScope&) = delete;
  CallScope& operator=(const CallScope&) = delete;
  ~CallScope() {
    if (nvtx_) nvtxRangePop();
  }
  gemm_status_t done(gemm_status_t st, const gemm_config_info_t* c = nullptr) const {
    if (!log_ || st != GEMM_OK || (c && c->path == GEMM_PATH_NONE)) return st;
    if (c)
      std::fprintf(stderr,
                   "gemm_log %s -> %s tile %dx%d cta/tile %d split %d stages %d grid %d sms %d tiles %lld launches %d "
                   "workspace %lld B\n",
                   text_, c->path == GEMM_PATH_SCALED_SLICED ? "scaled_sliced" : "scaled",
                   c->tile_m, c->tile_n, c->cta_per_tile, c->splitk, c->stages, c->grid, c->sms, (long long)c->tiles, c->launches,
                   (long long)c->workspace_bytes);
    else
      std::fprintf(stderr, "gemm_log %s\n", text_);
    return st;
  }

 private:
  const bool log_, nvtx_;
  char text_[160];
};

// A run of n bytes.
inline Region run_of(const void* p, int64_t n) { return region(p, p ? 1 : 0, n, 0, 1); }

// Rows of `ld` elements of es bytes from p allow 16-byte accesses where columns do.
inline bool rows_wide(const void* p, int64_t ld, int64_t es) { return aligned(p, 16) && (ld * es) % 16 == 0; }

// Does a result share a byte with an input or with another result?
inline bool results_meet(std::initializer_list<Region> results, std::initializer_list<Region> inputs) {
  for (const Region* r = results.begin(); r != results.end(); ++r) {
    for (const Region& i : inputs)
      if (overlaps(*r, i)) return true;
    for (const Region* o = results.begin(); o != r; ++o)
      if (overlaps(*r, *o)) return true;
  }
  return false;
}

}  // namespace dg
