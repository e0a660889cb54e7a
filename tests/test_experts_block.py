"""The experts' block of examples/experts_block.py, forward and backward, against the
same block in 32 bits.

An E4M3 code is off by at most 2^-4 of its value, 0.026 of it on the root mean square; a sum
of products of two such operands is off by 0.037 of its norm, and a result behind n products
one after another by 0.037 sqrt(n) where the errors are independent.  out and dw2 stand behind
two (dw2: one product of two results with codes of their own), dx, dw1 behind four, the
logits' gradient behind two and a difference between choices that doubles them.  Bounds: twice that.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("shape", [dict(), dict(tokens=37, experts=6, top_k=3, hidden=136, inner=264), dict(tokens=1, experts=4, top_k=1)])
def test_experts_block(shape):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("experts_block", os.path.join(ROOT, "examples", "experts_block.py"))
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    errors = block.compare(**shape)
    bound = {"out": 0.105, "out (serving)": 0.105, "dw2": 0.105, "dx": 0.15, "dw1": 0.15, "dlogits": 0.21}
    if shape.get("top_k") == 1:  # one renormalised weight is 1 whatever the logits: their gradient is 0
        errors.pop("dlogits")
    for name, e in errors.items():
        assert e <= bound[name], (name, errors)
