// plan.h -- the plan object and the host helpers shared by the translation
// units that implement the C ABI (api.cpp, ops.cpp).  Internal to the library.
#pragma once

#include "gemm.h"

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <mutex>
#include <unordered_map>
#include <vector>

#include "kernels.h"

namespace dg {

// A tensor-core call as far as planning and descriptors are concerned.
struct TcKey {
  int64_t M, N, K, lda, ldb, ldc;
  uintptr_t A, B, C;
  int32_t dtype, ta, tb, beta_nz;
  uintptr_t Cin;  // the C that beta scales (C itself unless gemm_run_ex got a separate one)
  int64_t ldcin;
  int32_t cin_kind;
  bool operator==(const TcKey& o) const {
    return M == o.M && N == o.N && K == o.K && lda == o.lda && ldb == o.ldb && ldc == o.ldc &&
           A == o.A && B == o.B && C == o.C && dtype == o.dtype && ta == o.ta && tb == o.tb &&
           beta_nz == o.beta_nz && Cin == o.Cin && ldcin == o.ldcin && cin_kind == o.cin_kind;
  }
};

struct TcKeyHash {
  size_t operator()(const TcKey& k) const {
    uint64_t h = 1469598103934665603ull;
    auto mix = [&](uint64_t v) { h = (h ^ v) * 1099511628211ull; };
    mix(uint64_t(k.M)); mix(uint64_t(k.N)); mix(uint64_t(k.K)); mix(uint64_t(k.lda));
    mix(uint64_t(k.ldb)); mix(uint64_t(k.ldc)); mix(k.A); mix(k.B); mix(k.C);
    mix(uint64_t(k.dtype) | (uint64_t(k.ta) << 8) | (uint64_t(k.tb) << 16) | (uint64_t(k.beta_nz) << 24) |
        (uint64_t(k.cin_kind) << 32));
    mix(k.Cin); mix(uint64_t(k.ldcin));
    return size_t(h);
  }
};

// One tensor-core plan: tile width, kernel variant, K slices, and whether
// only the tail wave's tiles are split.
struct TcChoice {
  int bn = 256, mode = dg::TC_SOLO, s = 1;
  bool tail = false;
  double t = 1e300;  // estimated seconds
};

// The C that beta scales: the output itself, or gemm_run_ex's separate C.
struct CinRef {
  const void* ptr;
  int64_t ld;
  int kind;  // dg::OutKind
};

// Planner decision, encoded tensor maps and kernel parameters of one call.
struct TcEntry {
  gemm_config_info_t info;
  CUtensorMap ma, mb, mc, mw;  // A, B, C, split-K partial workspace
  dg::TcParams p;
  size_t ws_bytes;
  void* ws_ptr;  // workspace the partial map was encoded for (split-K)
};

}  // namespace dg

struct gemm_plan {
  int device = 0;
  int sms = 0;
  int* err = nullptr;  // device word, OR of wait codes (and, debug build, failed-check sites)
  int64_t last_err_bits = 0;  // the word the last gemm_plan_poll_error read
  void* ws = nullptr;  // workspace (split-K partials, GEMV partials, counts of the slots' order)
  size_t ws_bytes = 0;
  // Whether a captured graph holds the buffer's address: it then lives as long as the plan, in `kept`
  // once a larger one has taken its place.
  bool ws_in_graph = false, tws_in_graph = false, counters_in_graph = false;
  std::vector<void*> kept;
  unsigned* counters = nullptr;  // GEMV per-panel arrival counters: zero between calls
  void* tws = nullptr;  // K-major copies of TF32 operands stored M/N-major, copies of unaligned codes
  size_t tws_bytes = 0;
  size_t counter_count = 0;
  uint64_t watchdog_ns = 2000000000ull;
  // Kernels launch as programmatic dependents of the stream's previous kernel
  // (their launch and prologue overlap its tail); GEMM_PDL=0 turns this off.
  bool pdl = true;
  gemm_config_info_t last{};
  // Repeated calls with the same shapes, pointers and flags skip planning and
  // descriptor encoding (host time that would otherwise sit in front of the
  // kernels on the stream).
  std::unordered_map<dg::TcKey, dg::TcEntry, dg::TcKeyHash> tc_cache;
  // GEMM_LOG=1 (read at plan creation): one line per call on stderr.
  bool log = false;
  // GEMM_NVTX=1 (read at plan creation): every gemm_run / gemm_run_ex is an
  // NVTX range named after its shape and types, for profilers' timelines.
  bool nvtx = false;
  // Benchmark mode: the fastest measured choice per shape (key without pointers).
  bool autotune = false;
  std::unordered_map<dg::TcKey, dg::TcChoice, dg::TcKeyHash> tuned;
};

namespace dg {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int env_int(const char* name, int dflt) {
  const char* v = std::getenv(name);
  if (!v || !*v) return dflt;
  return std::atoi(v);
}

inline int type_kind(gemm_type_t t) {
  return t == GEMM_TYPE_F32 ? dg::OUT_F32 : (t == GEMM_TYPE_BF16 ? dg::OUT_BF16 : dg::OUT_F16);
}

// ------------------------------------------------------------- validation

// Floor division for a positive divisor.
inline int64_t floor_div(int64_t a, int64_t b) { return a >= 0 ? a / b : -((-a + b - 1) / b); }

// A row-major matrix as memory: `rows` rows of `width` bytes, `pitch` bytes
// apart, the first at byte address `base`.
struct Region {
  uint64_t base;
  int64_t rows, pitch, width;
};

inline Region region(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esize) {
  return Region{uint64_t(reinterpret_cast<uintptr_t>(p)), rows, ld * esize, cols * esize};
}

// Byte ranges of a call's buffers for the debug build's device checks
// (kernels.h, DbgSpans).  The release build passes them to no kernel.
// GEMM_DEBUG_SHRINK=n (read by the debug build only, for its tests) makes the
// output's range n bytes shorter, so that the checks of the last output
// elements fail while every access stays inside the caller's buffer.
// GEMM_DEBUG_SHRINK_INPUT does the same for the inputs that say so below.
struct Spans {
  dg::DbgSpans s{};
  int n = 0;
  explicit Spans(int* err) { s.err = err; }
  Spans& bytes(const void* p, int64_t len) {
    if (p != nullptr && len > 0 && n < dg::kDbgSpans) {
      s.lo[n] = uint64_t(reinterpret_cast<uintptr_t>(p));
      s.hi[n] = s.lo[n] + uint64_t(len);
      ++n;
    }
    return *this;
  }
  // rows x cols elements of esize bytes, rows ld elements apart
  Spans& matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esize) {
    if (rows <= 0 || cols <= 0) return *this;
    return bytes(p, ((rows - 1) * ld + cols) * esize);
  }
  // count elements of esize bytes, inc elements apart
  Spans& vector(const void* p, int64_t count, int64_t inc, int64_t esize) {
    return count > 0 ? bytes(p, ((count - 1) * inc + 1) * esize) : *this;
  }
  // the output: its range less GEMM_DEBUG_SHRINK bytes
  Spans& out_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esize) {
    const int at = n;
    matrix(p, rows, cols, ld, esize);
    return shrink(at);
  }
  // an input that a copy or the groups' kernels read, `len` bytes: its range less GEMM_DEBUG_SHRINK_INPUT bytes
  Spans& input(const void* p, int64_t len) {
    static const int64_t cut = [] {
      const char* v = std::getenv("GEMM_DEBUG_SHRINK_INPUT");
      return v ? std::max<int64_t>(0, std::atoll(v)) : int64_t(0);
    }();
    return bytes(p, len - std::min(cut, len));
  }
  Spans& out_vector(const void* p, int64_t count, int64_t inc, int64_t esize) {
    const int at = n;
    vector(p, count, inc, esize);
    return shrink(at);
  }
  Spans& shrink(int at) {
    static const int64_t cut = [] {
      const char* v = std::getenv("GEMM_DEBUG_SHRINK");
      return v ? std::max<int64_t>(0, std::atoll(v)) : int64_t(0);
    }();
    if (at < n) s.hi[at] -= std::min<uint64_t>(uint64_t(cut), s.hi[at] - s.lo[at]);
    return *this;
  }
};

// Do two matrices share a byte?  Row i of x and row k of y meet iff y's row
// starts before x's ends and ends after x's starts: -wy < d + k*Ly - i*Lx < wx
// with d = by - bx.  Exact in O(1) for equal pitches (row-interleaved slices
// of one parent, or a single row), where only t = k - i matters; with
// different pitches the rows of the shorter matrix are tested one by one, and
// past 2^20 such rows overlapping byte spans count as overlap.
inline bool overlaps(Region x, Region y) {
  if (x.rows <= 0 || y.rows <= 0 || x.width <= 0 || y.width <= 0) return false;
  const uint64_t xe = x.base + uint64_t(x.rows - 1) * uint64_t(x.pitch) + uint64_t(x.width);
  const uint64_t ye = y.base + uint64_t(y.rows - 1) * uint64_t(y.pitch) + uint64_t(y.width);
  if (xe <= y.base || ye <= x.base) return false;  // disjoint spans
  if (x.rows == 1 && y.rows == 1) return true;  // (whose pitches mean nothing, and may be 0)
  if (x.rows == 1) x.pitch = y.pitch;  // a single row fits any pitch
  if (y.rows == 1) y.pitch = x.pitch;
  if (x.pitch == y.pitch) {
    const int64_t L = x.pitch;
    const int64_t d = int64_t(y.base - x.base);  // the spans overlap: |d| < 2^63
    // integers t in the open interval ((-wy - d) / L, (wx - d) / L), and
    // t = k - i in [1 - rows_x, rows_y - 1] (each such t has a valid i, k)
    const int64_t lo = std::max<int64_t>(floor_div(-y.width - d, L) + 1, 1 - x.rows);
    const int64_t hi = std::min<int64_t>(-floor_div(d - x.width, L) - 1, y.rows - 1);
    return lo <= hi;
  }
  if (x.rows > y.rows) std::swap(x, y);
  if (x.rows > (int64_t(1) << 20)) return true;
  const int64_t d = int64_t(y.base - x.base);
  for (int64_t i = 0; i < x.rows; ++i) {
    // row i of x covers [s, s + wx) relative to y.base; rows k of y with
    // k*Ly < s + wx and k*Ly + wy > s
    const int64_t s = int64_t(i) * x.pitch - d;
    const int64_t k_lo = std::max<int64_t>(floor_div(s - y.width, y.pitch) + 1, 0);
    const int64_t k_hi = std::min<int64_t>(floor_div(s + x.width - 1, y.pitch), y.rows - 1);
    if (k_lo <= k_hi) return true;
  }
  return false;
}

// ------------------------------------------------------------ tensor maps

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// ------------------------------------------------------------- workspace

// Is `s` being captured?  (A query that fails, as for the legacy stream during another's capture, means no.)
inline bool capturing(cudaStream_t s) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &status) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return status != cudaStreamCaptureStatusNone;
}

// `bytes` of zeroed device memory allocated at once, not as a node of the graph that the calling thread
// is capturing: such memory would exist in that graph's launches only.
inline cudaError_t alloc_outside_capture(void** out, size_t bytes) {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // this thread may allocate meanwhile
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return e;
  cudaStream_t side = nullptr;
  e = cudaMalloc(out, bytes);
  if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&side, cudaStreamNonBlocking);
  if (e == cudaSuccess) e = cudaMemsetAsync(*out, 0, bytes, side);
  if (e == cudaSuccess) e = cudaStreamSynchronize(side);
  if (side) cudaStreamDestroy(side);
  if (e != cudaSuccess && *out) {
    cudaFree(*out);
    *out = nullptr;
  }
  cudaThreadExchangeStreamCaptureMode(&mode);
  return e;
}

// Make a plan buffer at least `bytes` long (multiples of `step`, zero-filled; stream-ordered on `s`, except in a
// capture).  What a captured graph works on is never freed or moved under it: a buffer that was used
// in a capture stays with the plan when it is replaced.
inline gemm_status_t ensure_buffer(gemm_plan* plan, void** buf, size_t* have, bool* in_graph, size_t bytes, size_t step,
                                   cudaStream_t s) {
  const bool graph = capturing(s);
  if (bytes <= *have) {
    *in_graph |= graph;
    return GEMM_OK;
  }
  const size_t nb = (bytes + step - 1) / step * step;
  if (*buf && (graph || *in_graph)) {
    try {
      plan->kept.push_back(*buf);
    } catch (...) {
      return GEMM_ERR_OUT_OF_MEMORY;
    }
  } else if (*buf) {
    cudaFreeAsync(*buf, s);
  }
  *buf = nullptr;
  *have = 0;
  *in_graph = graph;
  if ((graph ? alloc_outside_capture(buf, nb) : cudaMallocAsync(buf, nb, s)) != cudaSuccess) {
    cudaGetLastError();
    *buf = nullptr;
    return GEMM_ERR_OUT_OF_MEMORY;
  }
  if (!graph && cudaMemsetAsync(*buf, 0, nb, s) != cudaSuccess) return GEMM_ERR_CUDA;
  *have = nb;
  return GEMM_OK;
}

inline gemm_status_t ensure_ws(gemm_plan* plan, size_t bytes, cudaStream_t s) {
  return ensure_buffer(plan, &plan->ws, &plan->ws_bytes, &plan->ws_in_graph, bytes, size_t(1) << 20, s);
}

inline gemm_status_t ensure_tws(gemm_plan* plan, size_t bytes, cudaStream_t s) {
  return ensure_buffer(plan, &plan->tws, &plan->tws_bytes, &plan->tws_in_graph, bytes, size_t(1) << 20, s);
}

// The counters are zeroed once when allocated; every kernel that uses one
// leaves it at zero again.
inline gemm_status_t ensure_counters(gemm_plan* plan, size_t count, cudaStream_t s) {
  void* buf = plan->counters;
  size_t bytes = plan->counter_count * sizeof(unsigned);
  const gemm_status_t st = ensure_buffer(plan, &buf, &bytes, &plan->counters_in_graph, count * sizeof(unsigned),
                                         4096 * sizeof(unsigned), s);
  plan->counters = static_cast<unsigned*>(buf);
  plan->counter_count = bytes / sizeof(unsigned);
  return st;
}

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

}  // namespace dg
