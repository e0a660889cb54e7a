"""GEMM_LOG and GEMM_NVTX at plan creation for the block-scaled products, the quantiser, routing and the weighted
sum: one line for each successful call that launches something, none without, none for a refused call; the
results are the same bits."""
import pytest

from tests.test_scaled_gpu import g  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def calls(gm, plan):
    """Every operator once, and their results."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    f8 = torch.float8_e4m3fn
    ints = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    T, E, k, N = 40, 8, 2, 64
    x = torch.randn((T, N), generator=gen, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn((T, E), generator=gen, device="cuda")
    w, i, pos, starts, counts = torch.zeros((T, k), device="cuda"), ints(T, k), ints(T, k), ints(E), ints(E)
    rowmap = ints(gm.gemm_route_rows(T, k, E))
    rows = rowmap.numel()
    new = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    q, sq, qt, st = new(rows, N), new(gm.gemm_scale_bytes(rows, N)), new(N, rows), new(gm.gemm_scale_bytes(N, rows))
    W = torch.randint(0x30, 0x40, (E, N, N), generator=gen, device="cuda").to(torch.uint8)
    SW = torch.full((E * gm.gemm_scale_bytes(N, N),), 120, dtype=torch.uint8, device="cuda")
    Y, D, G, out = (torch.zeros(s, device="cuda") for s in ((rows, N), (rows, N), (E, N, N), (T, N)))
    dl, dw, dY = torch.zeros_like(logits), torch.zeros_like(w), torch.zeros_like(Y)
    assert plan.route(logits, w, i, bias=torch.zeros(E, device="cuda"), score=gm.GEMM_SCORE_SIGMOID, groups=4, top_groups=2, renormalize=True) == 0
    assert plan.route_map(i, E, starts, counts, pos, rowmap) == 0
    assert plan.quantize(x, q.view(f8), sq, qt.view(f8), st, rowmap=rowmap, map_div=k) == 0
    assert plan.run_scaled(q.view(f8), sq, W[0].view(f8), SW, D) == 0
    assert plan.run_grouped(q.view(f8), sq, W.view(f8), SW, Y, starts, counts) == 0
    assert plan.run_grouped_k(qt.view(f8), st, qt.view(f8), st, G, starts, counts) == 0
    assert plan.combine(Y, pos, w, out) == 0
    assert plan.combine_backward(out, Y, pos, w, dY, dw, rowmap=rowmap) == 0
    assert plan.route_backward(logits, i, dw, dl, score=gm.GEMM_SCORE_SIGMOID, renormalize=True) == 0
    assert plan.run_scaled(q[:0].view(f8), sq, W[0].view(f8), SW, D[:0]) == 0  # nothing to do: no line
    assert plan.run_scaled(q.view(f8), sq, W[0].view(f8), SW, D, act=9) == gm.GEMM_ERR_INVALID_ARG
    torch.cuda.synchronize()
    return w, i, pos, starts, counts, rowmap, q, sq, qt, st, D, Y, G, out, dY, dw, dl


def test_a_line_for_each_call(g, monkeypatch, capfd):
    import torch
    quiet = calls(g, g.Plan(0))
    assert "gemm_log" not in capfd.readouterr().err
    monkeypatch.setenv("GEMM_LOG", "1")
    monkeypatch.setenv("GEMM_NVTX", "1")
    plan = g.Plan(0)
    loud = calls(g, plan)
    lines = [line for line in capfd.readouterr().err.splitlines() if line.startswith("gemm_log")]
    rows = quiet[5].numel()
    want = ["gemm_route 40x8 f32 sigmoid top 2 groups 2 of 4 bias renormalized", "gemm_route_map 40x2 experts 8 rows %d" % rows,
            "gemm_quantize %dx64 bf16->e4m3 block 1x128 Q QT by map" % rows, "gemm_run_scaled %dx64x64 groups 1 e4m3 e4m3->f32 -> scaled" % rows,
            "gemm_run_grouped %dx64x64 groups 8 e4m3 e4m3->f32 -> scaled" % rows, "gemm_run_grouped_k 64x64x%d groups 8 e4m3 e4m3->f32 -> scaled" % rows,
            "gemm_combine 40x2x64 rows %d f32->f32" % rows, "gemm_combine_backward 40x2x64 rows %d f32->f32 by map" % rows,
            "gemm_route_backward 40x8 f32 sigmoid top 2 renormalized"]
    assert len(lines) == len(want) and all(line.startswith("gemm_log " + w) for line, w in zip(lines, want)), lines
    assert all(torch.equal(a, b) for a, b in zip(quiet, loud))
