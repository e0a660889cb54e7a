"""Run by test_more_debug.py with the debug build and GEMM_DEBUG_SHRINK=4: each operator's output range is taken 4 bytes
short, so the check of its last plain store fails, the store is skipped, and every other element is written."""
from __future__ import annotations

import os

import torch

from dense_gemm_mma_gb300 import gemm
from tests.debug_ops import site


def main():
    assert gemm.gemm_debug_build() == 1 and os.environ.get("GEMM_DEBUG_SHRINK") == "4"
    plan = gemm.Plan(0)
    new = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    scales = lambda r, k: new(gemm.gemm_mx_scale_bytes(r, k))  # noqa: E731

    for kernel in ("sliced", "tile", "pair"):  # N = 130: the last columns go through plain stores
        os.environ["GEMM_SCALED_KERNEL"] = kernel
        D = torch.full((40, 132), float("nan"), device="cuda")
        assert plan.run_mx4(new(40, 128), scales(40, 256), new(130, 128), scales(130, 256), D[:, :130]) == 0
        site(plan, "scaled")
        missing = torch.isnan(D[:, :130])
        assert missing[39, 129] and missing.sum() <= 4, (kernel, int(missing.sum()))  # (a store is up to four columns)
    del os.environ["GEMM_SCALED_KERNEL"]

    x = torch.ones((128, 130), device="cuda")
    q, qt = torch.full((128, 80), 0x99, dtype=torch.uint8, device="cuda"), torch.full((130, 64), 0x99, dtype=torch.uint8, device="cuda")
    assert plan.quantize_mx4(x, q[:, :65], scales(128, 130)) == 0
    site(plan, "quantize")
    # a row is 65 bytes, stored as 16 words and a byte: the four bytes at its end, 61 to 64, lie in the last word (60 to 63) and in the byte
    assert (q[:, :65] == 0x99).sum() == 5 and (q[127, 60:65] == 0x99).all()
    assert plan.quantize_mx4(x, q[:, :65], scales(128, 130), qt, scales(130, 128)) == 0
    site(plan, "quantize")
    assert (qt == 0x99).sum() == 16  # the last store: 16 bytes
    v = torch.full((128, 130), float("nan"), device="cuda")
    assert plan.dequantize(new(128, 80)[:, :65], scales(128, 130), v) == 0
    site(plan, "quantize")
    assert torch.isnan(v).sum() == 2  # the last piece of the last row

    for cols in (30, 2050, 9000):
        x = torch.ones((5, cols), device="cuda")
        y, h, rstd = torch.full((5, cols), float("nan"), device="cuda"), torch.empty_like(x), torch.empty(5, device="cuda")
        assert plan.norm(x, Y=y, residual=x, H=h, rstd=rstd) == 0
        site(plan, "norm")
        assert torch.isnan(y[:4]).sum() == 0 and 1 <= torch.isnan(y[4]).sum() <= 8 and torch.isnan(y[4, -1])
        dx, dgain = torch.full((5, cols), float("nan"), device="cuda"), torch.empty(cols, device="cuda")
        assert plan.norm_backward(x, h, None, rstd, dx, dgain=dgain) == 0
        site(plan, "norm")
        assert torch.isnan(dx[:4]).sum() == 0 and 1 <= torch.isnan(dx[4]).sum() <= 8 and torch.isnan(dx[4, -1])
        assert torch.isfinite(dgain).all()

    for T in (5, 500):
        logits, index = torch.randn((T, 16), device="cuda"), torch.zeros((T, 2), dtype=torch.int32, device="cuda")
        counts = torch.empty(16, dtype=torch.int32, device="cuda")
        shares, factor, loss = (torch.full((n,), float("nan"), device="cuda") for n in (16, 16, 1))
        assert plan.balance(logits, index, counts, shares, factor, loss) == 0
        site(plan, "route")
        assert torch.isnan(factor).sum() == 1 and torch.isnan(factor[15]) and torch.isfinite(shares).all() and torch.isfinite(loss).all()
        dl = torch.full((T, 17), float("nan"), device="cuda")
        assert plan.balance_backward(logits, index, torch.ones(16, device="cuda"), dl[:, :16]) == 0
        site(plan, "route")
        assert torch.isnan(dl[:, :16]).sum() == 1
    print("ok")


if __name__ == "__main__":
    main()
