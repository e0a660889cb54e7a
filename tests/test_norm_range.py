"""Rows at the ends of what the norm's sum of squares holds: it is fp32, and its limits are those that include/gemm.h states."""
import pytest

from tests.test_norm_gpu import g, plan  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["float32", "bfloat16"])
@pytest.mark.parametrize("N", [64, 4096, 20000])
def test_sum_of_squares(plan, g, name, N):  # noqa: F811
    import torch
    t = getattr(torch, name)
    x = torch.ones((5, N), dtype=t, device="cuda")
    x[0] *= 2.0 ** 64 / 2 ** (N.bit_length() / 2)  # the sum of squares is 2^126 to 2^127: held
    x[1] *= 2.0 ** 64  # 2^128 and more: past the largest number
    x[2] *= 2.0 ** -54  # squares are normal numbers
    x[3] *= 2.0 ** -80  # squares are 0 in fp32
    Y, rstd, dx = torch.empty_like(x), torch.empty(5, device="cuda"), torch.empty_like(x)
    assert plan.norm(x, Y=Y, rstd=rstd, eps=0.0) == g.GEMM_OK
    near = 2.0 ** -7 if name == "bfloat16" else 2.0 ** -18
    for r in (0, 2, 4):
        assert (Y[r].double() - 1).abs().max() <= near
    assert rstd[1] == 0 and (Y[1] == 0).all()
    assert torch.isinf(rstd[3])
    assert plan.norm(x, Y=Y, rstd=rstd, eps=1e-6) == g.GEMM_OK
    assert rstd[1] == 0 and abs(float(rstd[3]) - 1e3) < 1e-3 and torch.isfinite(Y).all()
    assert plan.norm_backward(torch.ones_like(x), x, None, rstd, dx) == g.GEMM_OK
    assert torch.isfinite(dx).all() and (dx[1] == 0).all()
