"""The layer of examples/experts_layer.py, forward, backward and served in 4 bits, against the same layer in 32 bits.

h and y are one bf16 rounding off (2^-9 of the norm at most, root mean square of a uniform half step less); the loss is a sum of fp32
shares of logits that stand behind y's rounding.  An E4M3 code is off by 0.026 of its value on the root mean square, a product of two such
operands by 0.037 of its norm, and a result behind n products one after another by 0.037 sqrt(n) where the errors are
independent: out and dw2 two, dx and dgain (which sum dy, behind four), dw1 four, the logits' gradient two and a difference between
choices that doubles them; the projection one.  Bounds: twice that.  E2M1 with a scale for each 32: a code's step is 1/4 to 1/2 of its value
between 1 and 6 and the scale wastes up to half of the range: at most 0.13 of the norm on the root mean square for normal values (a step of 2
at 4 to 6, 1 at 2 to 4, 0.5 below: steps / sqrt(12) over the block's root mean square, which is 1.2 to 3 of the scale).  Served, the weights are the same
on both sides, the tokens and the hidden values are quantised: 0.13 sqrt(2), bound twice that.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BOUND = {"h": 2.0 ** -8, "y": 2.0 ** -8, "loss": 0.01, "out": 0.105, "dw2": 0.105, "dx": 0.15, "dgain": 0.15, "dw1": 0.15, "dlogits": 0.21,
         "projection": 0.075, "out (4 bits)": 0.37}


@pytest.mark.parametrize("shape", [dict(), dict(tokens=37, experts=6, top_k=3, hidden=136, inner=264), dict(tokens=1, experts=4, top_k=2)])
def test_experts_layer(shape):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("experts_layer", os.path.join(ROOT, "examples", "experts_layer.py"))
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    errors = layer.compare(**shape)
    assert set(errors) == set(BOUND)
    for name, e in errors.items():
        assert e <= BOUND[name], (name, errors)
