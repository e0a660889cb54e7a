"""Sigmoid shares of tokens whose logits are all far below zero: shares are a ratio, which has its value however small the
sigmoids themselves are (in fp32 they are 0 below about -103, and below -87 no normal numbers).  Against 64 bits (tests/more_ref.py),
in which sigmoids reach down to -700.

Tolerance as in test_balance_gpu.py, with u = 2^-24 and d the largest spread of a token's logits: each score is the reciprocal of a sum
of two exponentials of differences, (d + 12) u off at most; a share (60 + d) u; the mean adds T / 16 + 200 roundings, the gradient
three times a share's and 80 u.
"""
import numpy as np
import pytest

from tests import more_ref as ref
from tests.test_balance_gpu import HALF, Call, U, dtype, g, near, plan  # noqa: F401  (g, plan: fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(4, 1), (60, 6), (256, 8), (1000, 4)])
@pytest.mark.parametrize("top", [-20.0, -60.0, -86.0, -90.0, -104.0, -300.0, "mixed"])
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_low_logits(plan, g, E, k, top, name):  # noqa: F811
    import torch
    T = 70
    rng = np.random.default_rng(E)
    base = rng.choice([3.0, -5.0, -45.0, -87.5, -95.0, -650.0], (T, 1)) if top == "mixed" else np.full((T, 1), top)
    logits = torch.from_numpy(base - 12 * rng.random((T, E))).to(dtype(name)).cuda()
    x64 = logits.double().cpu().numpy()
    index = rng.integers(0, E, (T, k))
    index[::7] = -1
    indices = torch.from_numpy(index.astype(np.int32)).cuda()
    c = Call(g, plan, logits, indices, "sigmoid")
    counts, shares, factor, loss, p, live = ref.balance(x64, index, "sigmoid")
    off = (60 + (x64.max(1) - x64.min(1)).max()) * U
    mean = off + (T / 16 + 200) * U
    near(c.shares, shares, shares * mean)
    assert abs(float(c.shares.double().sum()) - 1) < mean  # every token that takes part has shares
    near(c.factor, factor, factor * 8 * U)
    near(c.loss, loss, loss * (mean + 60 * U))
    dx = torch.empty_like(logits)
    assert plan.balance_backward(logits, indices, c.factor, dx, **c.how) == g.GEMM_OK
    f = c.factor.double().cpu().numpy()
    want = ref.balance_backward(x64, index, f, 1.0, "sigmoid")
    size = p * (np.abs(f) + (np.abs(f) * p).sum(1, keepdims=True)) * live[:, None]
    near(dx, want, size * (3 * off + 80 * U) + np.abs(want) * HALF[name] + (2.0 ** -24 if name == "f16" else 1e-37))
    assert plan.poll_error() == g.GEMM_OK


def test_lowest_logits(plan, g):  # noqa: F811
    """Further down than 64 bits reach: logits of the type's lowest value among others, and nothing but them."""
    import torch
    low = torch.finfo(torch.float32).min
    logits = torch.full((4, 8), low, device="cuda")
    logits[0, :2] = torch.tensor([-1000.0, -1000.0])
    logits[1, 3] = 2.0
    logits[3] = float("-inf")  # masked: no shares
    shares = []
    for t in range(4):
        index = torch.full((4, 1), -1, dtype=torch.int32, device="cuda")
        index[t] = 5
        c = Call(g, plan, logits, index, "sigmoid")
        shares.append(c.shares.cpu())
        dx = torch.empty_like(logits)
        assert plan.balance_backward(logits, index, c.factor, dx, **c.how) == g.GEMM_OK
        assert torch.isfinite(dx).all() and torch.isfinite(c.loss).all()
    assert (shares[0][:2] - 0.5).abs().max() <= 4 * U and (shares[0][2:] == 0).all()
    assert abs(float(shares[1][3]) - 1) <= 4 * U and float(shares[1].sum() - shares[1][3]) == 0
    assert (shares[2] - 0.125).abs().max() <= 4 * U
    assert (shares[3] == 0).all()
