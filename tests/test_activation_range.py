"""SiLU and GELU behind 4-bit products over the whole range in which they are not their limits: arguments -96 to 96 in steps of 1/16, each an
exact sum of products, through every kernel.

Tolerance, relative to the result: the exponent's rounding, 1.25 |x| 2^-24 (SiLU) or 1.125 x^2 2^-24 (GELU), 2^-16 at most; 2^-20 for the
rest (the exponential's, the reciprocal's and the polynomial's own errors, each 2^-22); half a step of the result.  Below -87.3 SiLU may be 0 in
place of numbers below 2^-119 (the reciprocal of 1 + exp(-x) is no normal number there); GELU's exponential ends where its result is
no normal bf16 number (2^-126).
"""
import numpy as np
import pytest

from tests import more_ref as ref
from tests import scaled_ref
from tests.test_mx4_gpu import ROUND, float_rows, g, plan  # noqa: F401  (g, plan: fixtures)

pytestmark = pytest.mark.gpu

K = 1312


@pytest.mark.parametrize("kernel", ["tile", "pair", "sliced"])
@pytest.mark.parametrize("act", [3, 4])
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_every_sixteenth(plan, g, monkeypatch, kernel, act, out):  # noqa: F811
    import torch
    monkeypatch.setenv("GEMM_SCALED_KERNEL", kernel)
    n = 16 * 96 + 1
    code, byte = np.zeros((n, K), int), np.full((n, K // 32), 127)
    for k in range(11):  # bit k of the row's number: codes 0.5, 1, 2, 4 (1, 2, 4, 6 in E2M1's order) times a scale of its block
        block, j = divmod(k, 4)
        code[:, 32 * block + j] = np.where(np.arange(n) >> k & 1, (1, 2, 4, 6)[j], 0)
        byte[:, block] = 127 - 3 + 4 * block
    w = np.zeros((16, K), int)
    w[:, :96] = np.where(np.arange(16)[:, None] % 2 == 0, 2, 10)  # 1 and -1
    wb = np.full((16, K // 32), 127)
    a, b = (ref.scaled4(ref.decode4(ref.pack4(c), K), s) for c, s in ((code, byte), (w, wb)))
    x = a @ b.T
    assert np.array_equal(x[:, 0], np.arange(n) / 16) and np.array_equal(x[:, 1], -np.arange(n) / 16)
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    _, D = float_rows(n, 16, out)
    assert plan.run_mx4(dev(ref.pack4(code)), dev(ref.pack_scales4(byte, K)), dev(ref.pack4(w)), dev(ref.pack_scales4(wb, K)), D, K=K, act=act) == g.GEMM_OK
    assert plan.poll_error() == g.GEMM_OK and plan.last_config()["stages"] == (6 if kernel == "pair" else plan.last_config()["stages"])
    got, want = D.double().cpu().numpy(), scaled_ref.act(x, act)
    part = np.minimum(1.25 * np.abs(x) * 2.0 ** -24 if act == 4 else 1.125 * x * x * 2.0 ** -24, 2.0 ** -16)
    least = 2.0 ** -25 if out == "f16" else 2.0 ** -126 if act == 3 else np.where(x < -87.3, 2.0 ** -119, 2.0 ** -134)
    tol = np.abs(want) * (part + 2.0 ** -20 + ROUND[out]) + least
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (x[bad][:4], got[bad][:4], want[bad][:4])
    assert (got[:, ::2] == got[:, :1]).all() and (got[:, 1::2] == got[:, 1:2]).all()
