"""ctypes binding of libdgemm_gb300.so (include/gemm.h).

Argument marshalling only: every function here forwards to the C entry point
of the same name; the torch helpers at the bottom turn tensors into pointers,
leading dimensions and flags.  There is no fallback: if the shared library is
missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
# GEMM_DEBUG=1 in the environment (read at the first load) selects the debug
# build: device-side bounds and copy-rule checks (include/gemm.h, gemm_debug_build).
LIB_PATH = os.path.join(_PKG, "libdgemm_gb300_debug.so" if os.environ.get("GEMM_DEBUG") == "1"
                        else "libdgemm_gb300.so")

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_ALIGNMENT = 2
GEMM_ERR_UNSUPPORTED = 3
GEMM_ERR_NO_DEVICE = 4
GEMM_ERR_OUT_OF_MEMORY = 5
GEMM_ERR_CUDA = 6
GEMM_ERR_TIMEOUT = 7
GEMM_ERR_DEBUG_CHECK = 8
# bits of the plan's error word (gemm_plan_last_error_bits)
DBG_FLAG = 1 << 30
DBG_SITES = {0: "tma", 1: "epilogue_store", 2: "epilogue_load", 3: "split_in_kernel", 4: "tile_reduce",
             5: "gemv", 6: "scale", 7: "transpose", 8: "scaled", 9: "quantize", 10: "route", 11: "combine"}

GEMM_OP_N, GEMM_OP_T = 0, 1
GEMM_TYPE_BF16, GEMM_TYPE_F16, GEMM_TYPE_F32, GEMM_TYPE_TF32 = 0, 1, 2, 3
GEMM_TYPE_E4M3, GEMM_TYPE_E5M2 = 4, 5
GEMM_SCORE_SOFTMAX, GEMM_SCORE_SIGMOID = 0, 1
GEMM_BF16_F32, GEMM_BF16_BF16, GEMM_F16_F32, GEMM_F16_F16, GEMM_TF32_F32 = 0, 1, 2, 3, 4
GEMM_ACT_NONE, GEMM_ACT_LEAKY_RELU, GEMM_ACT_RELU, GEMM_ACT_GELU, GEMM_ACT_SILU = 0, 1, 2, 3, 4

PATH_NAMES = {0: "none", 1: "tc", 2: "tc_splitk", 3: "gemv_rowdot", 4: "gemv_colstream",
              5: "gemv_generic", 6: "scale", 7: "tc_splitk_cluster", 8: "tc_tail_split",
              9: "scaled", 10: "scaled_sliced"}

DTYPES = {("bf16", "f32"): GEMM_BF16_F32, ("bf16", "bf16"): GEMM_BF16_BF16,
          ("f16", "f32"): GEMM_F16_F32, ("f16", "f16"): GEMM_F16_F16, ("tf32", "f32"): GEMM_TF32_F32}


class gemm_epilogue_t(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("slope", ctypes.c_float)]


class gemm_route_t(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("top_k", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class gemm_config_info_t(ctypes.Structure):
    _fields_ = [
        ("path", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
        ("tile_k", ctypes.c_int32), ("cta_per_tile", ctypes.c_int32), ("splitk", ctypes.c_int32),
        ("stages", ctypes.c_int32), ("raster_group", ctypes.c_int32), ("grid", ctypes.c_int32),
        ("sms", ctypes.c_int32), ("tiles", ctypes.c_int64), ("units", ctypes.c_int64),
        ("waves", ctypes.c_double), ("tail_fraction", ctypes.c_double),
        ("useful_fraction", ctypes.c_double), ("launches", ctypes.c_int32),
        ("tail_tiles", ctypes.c_int32), ("workspace_bytes", ctypes.c_int64),
    ]

    def as_dict(self) -> dict:
        d = {name: getattr(self, name) for name, _ in self._fields_}
        d["path"] = PATH_NAMES.get(self.path, str(self.path))
        return d


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gemm_status_string(status)}")


_lib = None

# name -> (restype, argtypes)
_I64, _VP, _F, _I32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int32
_SIGNATURES = {
    "gemm_plan_create": (_I32, [ctypes.POINTER(_VP), ctypes.c_int]),
    "gemm_run": (_I32, [_VP, _I64, _I64, _I64, _VP, _I64, _VP, _I64, _VP, _I64, _F, _F,
                        _I32, _I32, _I32, gemm_epilogue_t, _VP]),
    "gemm_plan_destroy": (_I32, [_VP]),
    "gemm_status_string": (ctypes.c_char_p, [_I32]),
    "gemm_plan_last_config": (_I32, [_VP, ctypes.POINTER(gemm_config_info_t)]),
    "gemm_plan_poll_error": (_I32, [_VP, _VP]),
    "gemm_plan_set_watchdog": (_I32, [_VP, ctypes.c_uint64]),
    "gemm_plan_selftest_watchdog": (_I32, [_VP, _VP]),
    "gemm_check_args": (_I32, [_I64, _I64, _I64, _VP, _I64, _VP, _I64, _VP, _I64, _F,
                               _I32, _I32, _I32, gemm_epilogue_t]),
    "gemm_choose_config": (_I32, [_I64, _I64, _I64, _I32, _I32, _I32, _I32,
                                  ctypes.POINTER(gemm_config_info_t)]),
    "gemm_quantization": (_I32, [_I64, _I64, _I32, _I32, _I32, _I32, _I32,
                                 ctypes.POINTER(gemm_config_info_t)]),
    "gemm_gemv_noalloc": (_I32, [_I64, _I64, _I64, _VP, _I64, _VP, _I64, _VP, _I64, _F, _F,
                                 _I32, _I32, _I32, gemm_epilogue_t, _VP]),
    "gemm_plan_set_autotune": (_I32, [_VP, ctypes.c_int]),
    "gemm_run_ex": (_I32, [_VP, _I64, _I64, _I64, _VP, _I64, _VP, _I64, _VP, _I64, _I32, _VP, _I64, _I32,
                           _F, _F, _I32, _I32, _I32, gemm_epilogue_t, _VP]),
    "gemm_check_args_ex": (_I32, [_I64, _I64, _I64, _VP, _I64, _VP, _I64, _VP, _I64, _I32, _VP, _I64, _I32,
                                  _F, _F, _I32, _I32, _I32, gemm_epilogue_t]),
    "gemm_plan_tuned_count": (_I32, [_VP, ctypes.POINTER(_I64)]),
    "gemm_plan_last_error_bits": (_I32, [_VP, ctypes.POINTER(_I64)]),
    "gemm_debug_build": (ctypes.c_int, []),
    "gemm_scale_bytes": (_I64, [_I64, _I64]),
    "gemm_quantize": (_I32, [_VP, _I64, _I64, _VP, _I64, _I32, _VP, _I64, _I64, _I32, _I32, _VP, _I64, _VP, _VP,
                             _I64, _VP, _VP]),
    "gemm_run_scaled": (_I32, [_VP, _I64, _I64, _I64, _VP, _I64, _VP, _I32, _VP, _I64, _VP, _I32, _VP, _I64, _I32,
                               _F, _F, gemm_epilogue_t, _VP]),
    "gemm_check_scaled": (_I32, [_I64, _I64, _I64, _VP, _I64, _VP, _I32, _VP, _I64, _VP, _I32, _VP, _I64, _I32,
                                 _F, _F, gemm_epilogue_t]),
    "gemm_run_grouped": (_I32, [_VP, _I64, _I64, _I64, _I64, _VP, _VP, _VP, _I64, _VP, _I32, _VP, _I64, _I64, _VP,
                                _I32, _VP, _I64, _I32, _F, _F, gemm_epilogue_t, _VP]),
    "gemm_run_grouped_k": (_I32, [_VP, _I64, _I64, _I64, _I64, _VP, _VP, _VP, _I64, _VP, _I32, _VP, _I64, _VP, _I32,
                                  _VP, _I64, _I64, _I32, _F, _F, gemm_epilogue_t, _VP]),
    "gemm_route": (_I32, [_VP, _I64, _I64, _VP, _I64, _I32, _VP, gemm_route_t, _VP, _VP, _VP]),
    "gemm_route_backward": (_I32, [_VP, _I64, _I64, _VP, _I64, _I32, gemm_route_t, _VP, _VP, _VP, _I64, _VP]),
    "gemm_route_rows": (_I64, [_I64, _I64, _I64]),
    "gemm_route_map": (_I32, [_VP, _I64, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _I64, _VP]),
    "gemm_combine": (_I32, [_VP, _I64, _I64, _I64, _I64, _VP, _I64, _I32, _VP, _VP, _VP, _I64, _I32, _VP]),
    "gemm_combine_backward": (_I32, [_VP, _I64, _I64, _I64, _I64, _VP, _I64, _I32, _VP, _I64, _I32, _VP, _VP, _VP,
                                     _VP, _I64, _VP, _VP]),
}


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the shared library (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is not built; run __graft_entry__.build() "
                               "(python -m dense_gemm_mma_gb300.build)")
        lib = ctypes.CDLL(p)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def exported_symbols() -> list[str]:
    return list(_SIGNATURES)


# ---------------------------------------------------------------- C entry points

def gemm_status_string(status: int) -> str:
    return load().gemm_status_string(status).decode()


def gemm_plan_create(device: int = 0) -> int:
    h = _VP()
    st = load().gemm_plan_create(ctypes.byref(h), device)
    if st != GEMM_OK:
        raise GemmError(st, "gemm_plan_create")
    return h.value


def gemm_plan_destroy(plan: int) -> int:
    return load().gemm_plan_destroy(plan)


def gemm_run(plan, M, N, K, A, lda, B, ldb, C, ldc, alpha, beta, dtype, transA, transB,
             act=GEMM_ACT_NONE, slope=0.0, stream=None) -> int:
    return load().gemm_run(plan, M, N, K, A, lda, B, ldb, C, ldc, alpha, beta, dtype,
                           transA, transB, gemm_epilogue_t(act, slope), stream)


def gemm_run_ex(plan, M, N, K, A, lda, B, ldb, C, ldc, c_type, D, ldd, d_type, alpha, beta, ab_type,
                transA, transB, act=GEMM_ACT_NONE, slope=0.0, stream=None) -> int:
    return load().gemm_run_ex(plan, M, N, K, A, lda, B, ldb, C, ldc, c_type, D, ldd, d_type, alpha, beta,
                              ab_type, transA, transB, gemm_epilogue_t(act, slope), stream)


def gemm_check_args_ex(M, N, K, A, lda, B, ldb, C, ldc, c_type, D, ldd, d_type, alpha, beta, ab_type,
                       transA, transB, act=GEMM_ACT_NONE, slope=0.0) -> int:
    return load().gemm_check_args_ex(M, N, K, A, lda, B, ldb, C, ldc, c_type, D, ldd, d_type, alpha, beta,
                                     ab_type, transA, transB, gemm_epilogue_t(act, slope))


def gemm_plan_last_config(plan) -> gemm_config_info_t:
    info = gemm_config_info_t()
    st = load().gemm_plan_last_config(plan, ctypes.byref(info))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_plan_last_config")
    return info


def gemm_plan_poll_error(plan, stream=None) -> int:
    return load().gemm_plan_poll_error(plan, stream)


def gemm_plan_last_error_bits(plan) -> int:
    v = _I64()
    st = load().gemm_plan_last_error_bits(plan, ctypes.byref(v))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_plan_last_error_bits")
    return v.value


def gemm_debug_build() -> int:
    return load().gemm_debug_build()


def debug_sites(bits: int) -> list[str]:
    """Names of the debug-build check sites set in an error word."""
    return [name for s, name in DBG_SITES.items() if bits & (1 << (16 + s))]


def gemm_plan_set_watchdog(plan, timeout_ns: int) -> int:
    return load().gemm_plan_set_watchdog(plan, timeout_ns)


def gemm_plan_selftest_watchdog(plan, stream=None) -> int:
    return load().gemm_plan_selftest_watchdog(plan, stream)


def gemm_check_args(M, N, K, A, lda, B, ldb, C, ldc, alpha, dtype, transA, transB,
                    act=GEMM_ACT_NONE, slope=0.0) -> int:
    return load().gemm_check_args(M, N, K, A, lda, B, ldb, C, ldc, alpha, dtype, transA,
                                  transB, gemm_epilogue_t(act, slope))


def gemm_choose_config(M, N, K, dtype, transA, transB, sms) -> gemm_config_info_t:
    info = gemm_config_info_t()
    st = load().gemm_choose_config(M, N, K, dtype, transA, transB, sms, ctypes.byref(info))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_choose_config")
    return info


def gemm_quantization(M, N, tile_m, tile_n, splitk, sms, ctas_per_sm=1) -> gemm_config_info_t:
    info = gemm_config_info_t()
    st = load().gemm_quantization(M, N, tile_m, tile_n, splitk, sms, ctas_per_sm,
                                  ctypes.byref(info))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_quantization")
    return info


def gemm_gemv_noalloc(M, N, K, A, lda, B, ldb, C, ldc, alpha, beta, dtype, transA, transB,
                      act=GEMM_ACT_NONE, slope=0.0, stream=None) -> int:
    return load().gemm_gemv_noalloc(M, N, K, A, lda, B, ldb, C, ldc, alpha, beta, dtype,
                                    transA, transB, gemm_epilogue_t(act, slope), stream)


def gemm_plan_set_autotune(plan, enable: bool) -> int:
    return load().gemm_plan_set_autotune(plan, int(bool(enable)))


def gemm_plan_tuned_count(plan) -> int:
    n = _I64()
    st = load().gemm_plan_tuned_count(plan, ctypes.byref(n))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_plan_tuned_count")
    return n.value


def gemm_scale_bytes(rows, cols) -> int:
    return load().gemm_scale_bytes(rows, cols)


def gemm_quantize(plan, rows, cols, X, ldx, x_type, rowmap, map_div, src_rows, q_type, block_rows, Q, ldq, SQ, QT,
                  ldqt, SQT, stream=None) -> int:
    return load().gemm_quantize(plan, rows, cols, X, ldx, x_type, rowmap, map_div, src_rows, q_type, block_rows, Q,
                                ldq, SQ, QT, ldqt, SQT, stream)


def gemm_run_scaled(plan, M, N, K, A, lda, SA, a_type, B, ldb, SB, b_type, D, ldd, d_type, alpha, beta,
                    act=GEMM_ACT_NONE, slope=0.0, stream=None) -> int:
    return load().gemm_run_scaled(plan, M, N, K, A, lda, SA, a_type, B, ldb, SB, b_type, D, ldd, d_type, alpha, beta,
                                  gemm_epilogue_t(act, slope), stream)


def gemm_check_scaled(M, N, K, A, lda, SA, a_type, B, ldb, SB, b_type, D, ldd, d_type, alpha, beta,
                      act=GEMM_ACT_NONE, slope=0.0) -> int:
    return load().gemm_check_scaled(M, N, K, A, lda, SA, a_type, B, ldb, SB, b_type, D, ldd, d_type, alpha, beta,
                                    gemm_epilogue_t(act, slope))


def gemm_run_grouped(plan, groups, rows, N, K, starts, counts, A, lda, SA, a_type, B, ldb, b_group, SB, b_type, D,
                     ldd, d_type, alpha, beta, act=GEMM_ACT_NONE, slope=0.0, stream=None) -> int:
    return load().gemm_run_grouped(plan, groups, rows, N, K, starts, counts, A, lda, SA, a_type, B, ldb, b_group, SB,
                                   b_type, D, ldd, d_type, alpha, beta, gemm_epilogue_t(act, slope), stream)


def gemm_run_grouped_k(plan, groups, M, N, rows, starts, counts, A, lda, SA, a_type, B, ldb, SB, b_type, D, ldd,
                       d_group, d_type, alpha, beta, act=GEMM_ACT_NONE, slope=0.0, stream=None) -> int:
    return load().gemm_run_grouped_k(plan, groups, M, N, rows, starts, counts, A, lda, SA, a_type, B, ldb, SB, b_type,
                                     D, ldd, d_group, d_type, alpha, beta, gemm_epilogue_t(act, slope), stream)


def gemm_route(plan, tokens, experts, logits, ldl, l_type, bias, route, weights, indices, stream=None) -> int:
    return load().gemm_route(plan, tokens, experts, logits, ldl, l_type, bias, route, weights, indices, stream)


def gemm_route_backward(plan, tokens, experts, logits, ldl, l_type, route, indices, dweights, dlogits, lddl,
                        stream=None) -> int:
    return load().gemm_route_backward(plan, tokens, experts, logits, ldl, l_type, route, indices, dweights, dlogits,
                                      lddl, stream)


def gemm_route_rows(tokens, top_k, experts) -> int:
    return load().gemm_route_rows(tokens, top_k, experts)


def gemm_route_map(plan, tokens, top_k, experts, indices, starts, counts, pos, rowmap, rows, stream=None) -> int:
    return load().gemm_route_map(plan, tokens, top_k, experts, indices, starts, counts, pos, rowmap, rows, stream)


def gemm_combine(plan, tokens, top_k, cols, rows, Y, ldy, y_type, pos, weights, out, ldo, out_type,
                 stream=None) -> int:
    return load().gemm_combine(plan, tokens, top_k, cols, rows, Y, ldy, y_type, pos, weights, out, ldo, out_type,
                               stream)


def gemm_combine_backward(plan, tokens, top_k, cols, rows, dout, ldo, out_type, Y, ldy, y_type, pos, weights, rowmap,
                          dY, lddy, dweights, stream=None) -> int:
    return load().gemm_combine_backward(plan, tokens, top_k, cols, rows, dout, ldo, out_type, Y, ldy, y_type, pos,
                                        weights, rowmap, dY, lddy, dweights, stream)


# ------------------------------------------------------------------ torch helpers

_types: dict = {}  # torch dtype -> gemm_type_t, filled at the first tensor
_array_types: dict = {}
_PLAIN = gemm_epilogue_t(GEMM_ACT_NONE, 0.0)


def _type_of(t) -> int:
    """gemm_type_t of a tensor."""
    if not _types:
        import torch
        _types.update({torch.bfloat16: GEMM_TYPE_BF16, torch.float16: GEMM_TYPE_F16, torch.float32: GEMM_TYPE_F32,
                       torch.float8_e4m3fn: GEMM_TYPE_E4M3, torch.float8_e5m2: GEMM_TYPE_E5M2})
    try:
        return _types[t.dtype]
    except KeyError:
        raise ValueError(f"no gemm_type_t for {t.dtype}") from None


def _matrix(t):
    """(pointer, rows, columns, ld) of a 2-D tensor whose rows are contiguous.  (These helpers run in
    front of every launch, and small launches wait for them: one look at each property.)"""
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError("expected a 2-D tensor with contiguous rows")
    if ld < cols or ld <= 0:  # only a row that is alone (or empty) has no use for its stride
        if rows > 1 and cols > 0:
            raise ValueError("rows share memory (an expanded tensor?): expected each on its own")
        ld = max(cols, 1)
    return t.data_ptr(), rows, cols, ld


def _matrices(t):
    """(pointer, matrices, rows, columns, ld, elements between matrices) of a 3-D stack of matrices
    whose rows are contiguous."""
    n, rows, cols = t.shape
    group, ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError("expected a 3-D stack of matrices with contiguous rows")
    some = n > 0 and rows > 0 and cols > 0
    if ld < cols or ld <= 0:
        if rows > 1 and some:
            raise ValueError("rows share memory (an expanded tensor?): expected each on its own")
        ld = max(cols, 1)
    if group < (rows - 1) * ld + cols:  # only a matrix that is alone (or empty) has no use for its stride
        if n > 1 and some:
            raise ValueError("the stack's matrices share memory or interleave: expected one after another")
        group = ld * rows
    return t.data_ptr(), n, rows, cols, ld, group


def _scales(t, rows: int, cols: int, groups: int = 1) -> int:
    """Pointer of the packed scale bytes of `groups` rows x cols matrices."""
    need = groups * 512 * (-(-rows // 128) or 1) * (-(-cols // 512) or 1)  # gemm_scale_bytes
    if t.element_size() != 1 or t.numel() < need or not t.is_contiguous():
        raise ValueError(f"scales are {need} contiguous bytes")
    return t.data_ptr()


def _array(t, n: int, dtype: str) -> int:
    """Pointer of at least n contiguous values ("int32" or "float32")."""
    if t.dtype is not _array_types.get(dtype):
        if not _array_types:
            import torch
            _array_types.update(int32=torch.int32, float32=torch.float32)
            return _array(t, n, dtype)
        raise ValueError(f"expected {dtype}")
    if t.numel() < n or not t.is_contiguous():
        raise ValueError(f"expected {n} contiguous {dtype}")
    return t.data_ptr()


def _epilogue(act, slope):
    return _PLAIN if act == GEMM_ACT_NONE else gemm_epilogue_t(act, slope)


def pack_scales(scales):
    """Packed scale bytes (include/gemm.h) of a rows x blocks uint8 tensor of E8M0 bytes,
    e.g. a checkpoint's power-of-two scales.  A 128 x 128 block's scale is repeated in its 128 rows."""
    import torch
    rows, blocks = scales.shape
    r, c = max(-(-rows // 128), 1) * 128, max(-(-blocks // 4), 1) * 4
    full = torch.zeros((r, c), dtype=torch.uint8, device=scales.device)
    full[:rows, :blocks] = scales
    return full.view(r // 128, 4, 32, c // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def unpack_scales(packed, rows: int, cols: int):
    """The rows x ceil(cols / 128) scale bytes of a packed rows x cols matrix."""
    r, c = max(-(-rows // 128), 1) * 128, max(-(-cols // 512), 1) * 4
    return packed[:r * c].view(r // 128, c // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r, c)[:rows, :-(-cols // 128)]


def _operand(t, trans: bool):
    """(pointer, ld) of a stored 2-D operand whose rows are contiguous."""
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("operands must be 2-D with contiguous rows")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError("rows share memory (an expanded tensor?): expected each on its own")
    return t.data_ptr(), max(t.stride(0), t.shape[1], 1)


class Plan:
    """Owns a gemm_plan_t on one device.  The calls take tensors of that device whose rows (and, in a stack, matrices)
    each have their own memory, in the order of their indices; others raise ValueError."""

    def __init__(self, device: int = 0):
        self.handle = gemm_plan_create(device)
        self.device = device
        self._current = None  # reads torch's current stream

    def close(self):
        if self.handle:
            gemm_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def run(self, A, B, C, *, alpha=1.0, beta=0.0, transA=False, transB=False,
            act=GEMM_ACT_NONE, slope=0.0, stream=None, M=None, N=None, K=None) -> int:
        """C <- act(alpha*op(A)@op(B) + beta*C) on torch tensors holding the
        STORED matrices (A is K x M when transA, B is N x K when transB)."""
        import torch
        # fp32 operands are read as TF32 by the tensor cores (GEMM_TF32_F32)
        in_t = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "tf32"}[A.dtype]
        out_t = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[C.dtype]
        if B.dtype != A.dtype:
            raise ValueError("A and B must have the same dtype")
        dtype = DTYPES[(in_t, out_t)]
        a, lda = _operand(A, transA)
        b, ldb = _operand(B, transB)
        c, ldc = _operand(C, False)
        M = C.shape[0] if M is None else M
        N = C.shape[1] if N is None else N
        K = (A.shape[0] if transA else A.shape[1]) if K is None else K
        if stream is None:
            stream = torch.cuda.current_stream(C.device).cuda_stream
        return gemm_run(self.handle, M, N, K, a, lda, b, ldb, c, ldc, alpha, beta, dtype,
                        int(transA), int(transB), act, slope, stream)

    def last_config(self) -> dict:
        return gemm_plan_last_config(self.handle).as_dict()

    def poll_error(self, stream=None) -> int:
        return gemm_plan_poll_error(self.handle, stream)

    # ------------------------------------------- block-scaled 8-bit products

    def _stream(self, stream):
        """The given stream, or torch's current one on the plan's device."""
        if stream is not None:
            return stream
        if self._current is None:
            import torch
            self._current = torch._C._cuda_getCurrentRawStream
        return self._current(self.device)

    def quantize(self, X, Q=None, SQ=None, QT=None, SQT=None, *, block_rows=1, rowmap=None, map_div=1,
                 stream=None) -> int:
        """X (rows x cols) -> 8-bit Q and scales SQ, and/or its transpose QT and scales SQT
        (float8_e4m3fn or float8_e5m2; scales gemm_scale_bytes uint8).  With rowmap (int32) row r
        of the result is X's row rowmap[r] // map_div (negative: none)."""
        x, src_rows, cols, ldx = _matrix(X)
        rows = src_rows if rowmap is None else rowmap.numel()
        q = sq = qt = sqt = None
        ldq = ldqt = 0
        if Q is not None:
            q, r, c, ldq = _matrix(Q)
            sq = _scales(SQ, rows, cols)
            if (r, c) != (rows, cols):
                raise ValueError("Q is rows x cols")
        if QT is not None:
            qt, c, r, ldqt = _matrix(QT)
            sqt = _scales(SQT, cols, rows)
            if (r, c) != (rows, cols) or (Q is not None and Q.dtype != QT.dtype):
                raise ValueError("QT is cols x rows, of Q's type")
        kind = Q if Q is not None else QT
        if kind is None:
            raise ValueError("neither Q nor QT")
        return load().gemm_quantize(self.handle, rows, cols, x, ldx, _type_of(X),
                                    None if rowmap is None else _array(rowmap, rows, "int32"), map_div, src_rows,
                                    _type_of(kind), block_rows, q, ldq, sq, qt, ldqt, sqt, self._stream(stream))

    def run_scaled(self, A, SA, B, SB, D, *, alpha=1.0, beta=0.0, act=GEMM_ACT_NONE, slope=0.0, stream=None) -> int:
        """D <- act(alpha * A @ B^T + beta * D) on 8-bit A (M x K), B (N x K) with packed scales SA, SB."""
        a, M, K, lda = _matrix(A)
        b, N, Kb, ldb = _matrix(B)
        d, Md, Nd, ldd = _matrix(D)
        if Kb != K or Md != M or Nd != N:
            raise ValueError("A is M x K, B is N x K and D is M x N")
        return load().gemm_run_scaled(self.handle, M, N, K, a, lda, _scales(SA, M, K), _type_of(A), b, ldb,
                                      _scales(SB, N, K), _type_of(B), d, ldd, _type_of(D), alpha, beta,
                                      _epilogue(act, slope), self._stream(stream))

    def run_grouped(self, A, SA, B, SB, D, starts, counts, *, alpha=1.0, beta=0.0, act=GEMM_ACT_NONE, slope=0.0,
                    stream=None) -> int:
        """Rows starts[e] .. starts[e] + counts[e] of A (rows x K) times B[e]^T (B groups x N x K, SB
        the groups' packed scales one after another) into the same rows of D (rows x N)."""
        a, rows, K, lda = _matrix(A)
        b, groups, N, Kb, ldb, b_group = _matrices(B)
        d, rows_d, Nd, ldd = _matrix(D)
        if Kb != K or rows_d != rows or Nd != N:
            raise ValueError("A is rows x K, B is groups x N x K and D is rows x N")
        return load().gemm_run_grouped(self.handle, groups, rows, N, K, _array(starts, groups, "int32"),
                                       _array(counts, groups, "int32"), a, lda, _scales(SA, rows, K), _type_of(A), b,
                                       ldb, b_group, _scales(SB, N, K, groups), _type_of(B), d, ldd, _type_of(D), alpha,
                                       beta, _epilogue(act, slope), self._stream(stream))

    def run_grouped_k(self, A, SA, B, SB, D, starts, counts, *, alpha=1.0, beta=0.0, act=GEMM_ACT_NONE, slope=0.0,
                      stream=None) -> int:
        """D[e] <- act(alpha * A_e @ B_e^T + beta * D[e]), A_e and B_e columns starts[e] .. starts[e] + counts[e]
        of A (M x rows) and B (N x rows); D groups x M x N."""
        a, M, rows, lda = _matrix(A)
        b, N, rows_b, ldb = _matrix(B)
        d, groups, Md, Nd, ldd, d_group = _matrices(D)
        if rows_b != rows or Md != M or Nd != N:
            raise ValueError("A is M x rows, B is N x rows and D is groups x M x N")
        return load().gemm_run_grouped_k(self.handle, groups, M, N, rows, _array(starts, groups, "int32"),
                                         _array(counts, groups, "int32"), a, lda, _scales(SA, M, rows), _type_of(A), b,
                                         ldb, _scales(SB, N, rows), _type_of(B), d, ldd, d_group, _type_of(D), alpha,
                                         beta, _epilogue(act, slope), self._stream(stream))

    # ----------------------------------------------------------- experts

    def route(self, logits, weights, indices, *, bias=None, score=GEMM_SCORE_SOFTMAX, groups=1, top_groups=1,
              group_top=1, renormalize=False, scale=1.0, stream=None) -> int:
        """logits (tokens x experts) -> each token's chosen experts (indices, tokens x top_k int32)
        and their weights (tokens x top_k float32)."""
        x, tokens, experts, ldl = _matrix(logits)
        n, k = weights.shape
        if n != tokens or indices.shape != weights.shape:
            raise ValueError("weights and indices are tokens x top_k")
        return load().gemm_route(self.handle, tokens, experts, x, ldl, _type_of(logits),
                                 None if bias is None else _array(bias, experts, "float32"),
                                 gemm_route_t(score, k, groups, top_groups, group_top, int(renormalize), scale),
                                 _array(weights, tokens * k, "float32"), _array(indices, tokens * k, "int32"),
                                 self._stream(stream))

    def route_backward(self, logits, indices, dweights, dlogits, *, score=GEMM_SCORE_SOFTMAX, renormalize=False,
                       scale=1.0, stream=None) -> int:
        """The gradient of the logits (dlogits) from the weights' (dweights) and the choice (indices)."""
        x, tokens, experts, ldl = _matrix(logits)
        d, nt, ne, lddl = _matrix(dlogits)
        n, k = indices.shape
        if (nt, ne) != (tokens, experts) or n != tokens or dlogits.dtype != logits.dtype or indices.shape != dweights.shape:
            raise ValueError("dlogits is like logits, dweights like indices")
        return load().gemm_route_backward(self.handle, tokens, experts, x, ldl, _type_of(logits),
                                          gemm_route_t(score, k, 1, 1, 1, int(renormalize), scale),
                                          _array(indices, tokens * k, "int32"), _array(dweights, tokens * k, "float32"), d,
                                          lddl, self._stream(stream))

    def route_map(self, indices, experts, starts, counts, pos, rowmap, *, stream=None) -> int:
        """The order of the slots of indices (tokens x top_k) by expert; rowmap has gemm_route_rows entries."""
        tokens, k = indices.shape
        return load().gemm_route_map(self.handle, tokens, k, experts, _array(indices, tokens * k, "int32"),
                                     _array(starts, experts, "int32"), _array(counts, experts, "int32"),
                                     _array(pos, tokens * k, "int32"), _array(rowmap, 0, "int32"), rowmap.numel(),
                                     self._stream(stream))

    def combine(self, Y, pos, weights, out, *, stream=None) -> int:
        """out[t] <- sum_j weights[t, j] * Y[pos[t, j]]."""
        y, rows, cols, ldy = _matrix(Y)
        o, nt, nc, ldo = _matrix(out)
        tokens, k = pos.shape
        if nt != tokens or nc != cols:
            raise ValueError("out is tokens x cols")
        return load().gemm_combine(self.handle, tokens, k, cols, rows, y, ldy, _type_of(Y), _array(pos, tokens * k, "int32"),
                                   _array(weights, tokens * k, "float32"), o, ldo, _type_of(out), self._stream(stream))

    def combine_backward(self, dout, Y, pos, weights, dY, dweights, *, rowmap=None, stream=None) -> int:
        """dY[pos[t, j]] <- weights[t, j] * dout[t], dweights[t, j] <- <dout[t], Y[pos[t, j]]>; with rowmap the
        rows of dY that hold no slot are cleared."""
        y, rows, cols, ldy = _matrix(Y)
        g, nt, nc, ldo = _matrix(dout)
        d, nr, ncd, lddy = _matrix(dY)
        tokens, k = pos.shape
        if (nt, nc) != (tokens, cols) or (nr, ncd) != (rows, cols) or dY.dtype != Y.dtype:
            raise ValueError("dout is tokens x cols, dY like Y")
        return load().gemm_combine_backward(self.handle, tokens, k, cols, rows, g, ldo, _type_of(dout), y, ldy, _type_of(Y),
                                            _array(pos, tokens * k, "int32"), _array(weights, tokens * k, "float32"),
                                            None if rowmap is None else _array(rowmap, rows, "int32"), d, lddy,
                                            _array(dweights, tokens * k, "float32"), self._stream(stream))
