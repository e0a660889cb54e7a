"""Run by test_debug_ops.py with the debug build and GEMM_DEBUG_SHRINK=4: each operator's
output range is taken 4 bytes short, so the check of its last plain store fails, the
store is skipped, and every other element is written."""
from __future__ import annotations

import os

import torch

from dense_gemm_mma_gb300 import gemm


def site(plan, name):
    assert plan.poll_error() == gemm.GEMM_ERR_DEBUG_CHECK, name
    bits = gemm.gemm_plan_last_error_bits(plan.handle)
    assert bits & gemm.DBG_FLAG and gemm.debug_sites(bits) == [name] and (bits & 0xFFFF) == 0, (name, hex(bits))


def main():
    assert gemm.gemm_debug_build() == 1 and os.environ.get("GEMM_DEBUG_SHRINK") == "4"
    plan = gemm.Plan(0)
    ints = lambda *n: torch.full(n, -7, dtype=torch.int32, device="cuda")  # noqa: E731
    codes = lambda r, k: torch.zeros((r, k), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    scales = lambda r, k: torch.zeros(gemm.gemm_scale_bytes(r, k), dtype=torch.uint8, device="cuda")  # noqa: E731

    for kernel in ("sliced", "tile", "pair"):  # N = 130: the last columns go through plain stores
        os.environ["GEMM_SCALED_KERNEL"] = kernel
        D = torch.full((40, 132), float("nan"), device="cuda")
        assert plan.run_scaled(codes(40, 256), scales(40, 256), codes(130, 256), scales(130, 256), D[:, :130]) == 0
        site(plan, "scaled")
        missing = torch.isnan(D[:, :130])
        assert missing[39, 129] and missing.sum() <= 4, (kernel, int(missing.sum()))  # (a store is up to four columns)

    x = torch.ones((128, 130), device="cuda")
    qt = torch.full((130, 128), 0x11, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    assert plan.quantize(x, codes(128, 144)[:, :130], scales(128, 130), qt, scales(130, 128)) == 0
    site(plan, "quantize")
    assert (qt.view(torch.uint8) == 0x11).sum() == 16  # the last store: 16 bytes

    logits, w, i = torch.randn((5, 16), device="cuda"), torch.zeros((5, 2), device="cuda"), ints(5, 2)
    assert plan.route(logits, w, i) == 0
    site(plan, "route")
    assert (i == -7).sum() == 1 and i[4, 1] == -7
    chosen = torch.zeros((5, 2), dtype=torch.int32, device="cuda")
    dl = torch.full((5, 17), float("nan"), device="cuda")
    assert plan.route_backward(logits, chosen, w, dl[:, :16]) == 0
    site(plan, "route")
    assert torch.isnan(dl[:, :16]).sum() == 1
    rows = gemm.gemm_route_rows(5, 2, 16)
    rowmap = ints(rows)
    assert plan.route_map(chosen, 16, ints(16), ints(16), ints(5, 2), rowmap) == 0
    site(plan, "route")
    assert (rowmap == -7).sum() <= 4 and rowmap[-1] == -7

    Y, pos, out = torch.randn((8, 30), device="cuda"), torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.full((3, 30), float("nan"), device="cuda")
    wt = torch.ones((3, 2), device="cuda")
    assert plan.combine(Y, pos, wt, out) == 0
    site(plan, "combine")
    assert torch.isnan(out).sum() == 6  # the last piece of the last row
    pos = torch.tensor([[0, 1], [2, 3], [4, 7]], dtype=torch.int32, device="cuda")
    dY = torch.full((8, 30), float("nan"), device="cuda")
    assert plan.combine_backward(torch.ones_like(out), Y, pos, wt, dY, torch.empty_like(wt)) == 0
    site(plan, "combine")
    assert torch.isnan(dY[7]).sum() == 6 and torch.isnan(dY[[0, 1, 2, 3, 4]]).sum() == 0
    print("ok")


if __name__ == "__main__":
    main()
