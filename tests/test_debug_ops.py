"""The block-scaled products, the quantiser, routing and the weighted sum in the debug
build of the library (device-side checks of every plain global access and every TMA
coordinate, include/gemm.h: gemm_debug_build), run in child processes because the
binding loads one library per process.

- Their own tests pass under the checks, and no check fails.
- With the output's range taken 4 bytes short (GEMM_DEBUG_SHRINK), each kernel skips
  the store of its last output and reports its site; nothing else is missing.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(args, **more):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_gemm_mma_gb300 import build
    build.build(debug=True)
    env = {k: v for k, v in os.environ.items() if not k.startswith("GEMM_")}
    r = subprocess.run([sys.executable, *args], cwd=ROOT, env=dict(env, GEMM_DEBUG="1", **more), capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    return r.stdout


def test_operators_pass_their_tests_under_the_checks():
    _run(["-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_scaled_gpu.py", "tests/test_experts_gpu.py",
          "-k", "row_map or (test_quantize and 129) or (test_product and (33 or 129 or 513)) or test_grouped or address or "
                "units or test_route or test_combine"])


def test_skipped_and_reported():
    assert _run(["-m", "tests.debug_ops"], GEMM_DEBUG_SHRINK="4").strip().startswith("ok")


def test_inputs_skipped_and_reported():
    assert _run(["-m", "tests.debug_inputs"], GEMM_DEBUG_SHRINK_INPUT="4").strip().startswith("ok")


def test_edges_pass_under_the_checks():
    _run(["-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_scaled_gpu.py", "tests/test_experts_gpu.py",
          "-k", "copied or square or meet or share or between or in_place"])
