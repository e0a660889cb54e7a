"""Run by test_debug_ops.py with the debug build and GEMM_DEBUG_SHRINK_INPUT=4: the ranges of the groups' starts
and counts, and of codes that are copied, are taken 4 bytes short, so that the checks of their last
loads fail; the loads are skipped and reported, and nothing else goes missing."""
from __future__ import annotations

import os

import torch

from dense_gemm_mma_gb300 import gemm
from tests.debug_ops import site


def main():
    assert gemm.gemm_debug_build() == 1 and os.environ.get("GEMM_DEBUG_SHRINK_INPUT") == "4"
    plan = gemm.Plan(0)
    ones = lambda *n: torch.full(n, 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    scales = lambda r, k, e=1: torch.full((e * gemm.gemm_scale_bytes(r, k),), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    E, N, K = 3, 64, 256
    starts = torch.tensor([0, 128, 256], dtype=torch.int32, device="cuda")
    counts = torch.tensor([100, 128, 70], dtype=torch.int32, device="cuda")
    for kernel in ("sliced", "tile", "pair"):  # the last group counts as empty
        os.environ["GEMM_SCALED_KERNEL"] = kernel
        D = torch.zeros((384, N), device="cuda")
        assert plan.run_grouped(ones(384, K), scales(384, K), ones(E, N, K), scales(N, K, E), D, starts, counts) == 0
        site(plan, "scaled")
        assert (D[:100] == K).all() and (D[128:256] == K).all() and (D[100:128] == 0).all() and (D[256:] == 0).all(), kernel
    for kernel in ("tile", "pair"):
        os.environ["GEMM_SCALED_KERNEL"] = kernel
        D = torch.full((E, N, N), 5.0, device="cuda")
        assert plan.run_grouped_k(ones(N, 384), scales(N, 384), ones(N, 384), scales(N, 384), D, starts, counts) == 0
        site(plan, "scaled")
        assert (D[0] == 128).all() and (D[1] == 128).all() and (D[2] == 0).all(), kernel
    del os.environ["GEMM_SCALED_KERNEL"]
    # copies of codes: rows `ld` bytes apart, loads of 8, 4 and 1 bytes; the last 4 bytes (or the word that holds them) read as 0
    K = 40
    for ld, lost in ((40, 8), (44, 4), (41, 4)):
        A = torch.full((20 * ld,), 0x38, dtype=torch.uint8, device="cuda").as_strided((20, K), (ld, 1)).view(torch.float8_e4m3fn)
        D = torch.zeros((20, N), device="cuda")
        assert plan.run_scaled(A, scales(20, K), ones(N, 48)[:, :K], scales(N, K), D) == 0
        site(plan, "quantize")
        assert (D[:19] == K).all() and (D[19] == K - lost).all(), (ld, D[19, 0].item())
    print("ok")


if __name__ == "__main__":
    main()
