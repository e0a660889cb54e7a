"""The 4-bit products and quantisers, the norm and the balance loss in the debug build of the library (device-side checks of every
plain global access and every TMA coordinate, include/gemm.h: gemm_debug_build), run in child processes because the binding
loads one library per process.

- Their own tests pass under the checks, and no check fails.
- With the output's range taken 4 bytes short (GEMM_DEBUG_SHRINK), each kernel skips the store of its last
  output and reports its site; nothing else is missing.
"""
import pytest

from tests.test_debug_ops import _run

pytestmark = pytest.mark.gpu


def test_operators_pass_their_tests_under_the_checks():
    _run(["-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_mx4_gpu.py", "tests/test_norm_gpu.py",
          "tests/test_balance_gpu.py", "-k", "row_map or dequantize or (test_quantize and (129 or 2050)) or (test_product and (33 or 129 or 513 or 4096)) or "
          "test_grouped or address or tiles or in_place or test_codes or (test_norm and (513 or 2050 or 20000)) or "
          "(test_gradients and (513 or 2050 or 20000)) or (test_balance and (256 or 128 or 1024))"])


def test_skipped_and_reported():
    assert _run(["-m", "tests.more_debug_ops"], GEMM_DEBUG_SHRINK="4").strip().startswith("ok")
