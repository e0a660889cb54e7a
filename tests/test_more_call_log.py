"""GEMM_LOG and GEMM_NVTX at plan creation for the 4-bit products and quantisers, the norm and the balance loss: one line for each
successful call that launches something, none without, none for a refused call; the results are the same bits.  And the
path of a plan's calls one behind another on another stream than torch's default one."""
import pytest

from tests.test_scaled_gpu import g  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def calls(gm, plan, stream=None):
    """Every operator once, and their results."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    ints = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    new = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device="cuda")  # noqa: E731
    T, E, k, N = 40, 8, 2, 64
    x = torch.randn((T, N), generator=gen, device="cuda", dtype=torch.bfloat16)
    h, y, dx, v = (torch.zeros_like(x) for _ in range(4))
    rstd, dgain = torch.zeros(T, device="cuda"), torch.zeros(N, device="cuda")
    q8, s8 = new(T, N).view(torch.float8_e4m3fn), new(gm.gemm_scale_bytes(T, N))
    logits = torch.randn((T, E), generator=gen, device="cuda")
    w, i, pos, starts, counts = torch.zeros((T, k), device="cuda"), ints(T, k), ints(T, k), ints(E), ints(E)
    rowmap = ints(gm.gemm_route_rows(T, k, E))
    rows = rowmap.numel()
    load, shares, factor, loss, dl = ints(E), *(torch.zeros(n, device="cuda") for n in (E, E, 1)), torch.zeros_like(logits)
    q, sq, qt, st = new(rows, N // 2), new(gm.gemm_mx_scale_bytes(rows, N)), new(N, rows // 2), new(gm.gemm_mx_scale_bytes(N, rows))
    W = torch.randint(0, 256, (E, N, N // 2), generator=gen, device="cuda").to(torch.uint8)
    SW = torch.full((E * gm.gemm_mx_scale_bytes(N, N),), 125, dtype=torch.uint8, device="cuda")
    D, Y = torch.zeros((rows, N), device="cuda"), torch.zeros((rows, N), device="cuda")
    torch.cuda.synchronize()
    on = {"stream": stream}
    assert plan.norm(x, None, Y=y, Q=q8, SQ=s8, residual=x, H=h, rstd=rstd, **on) == 0
    assert plan.route(logits, w, i, **on) == 0
    assert plan.route_map(i, E, starts, counts, pos, rowmap, **on) == 0
    assert plan.balance(logits, i, load, shares, factor, loss, **on) == 0
    assert plan.balance_backward(logits, i, factor, dl, accumulate=True, **on) == 0
    assert plan.quantize_mx4(y, q, sq, qt, st, rowmap=rowmap, map_div=k, **on) == 0
    assert plan.run_mx4(q, sq, W[0], SW, D, **on) == 0
    assert plan.run_grouped_mx4(q, sq, W, SW, Y, starts, counts, **on) == 0
    assert plan.dequantize(q8, s8, v, **on) == 0
    assert plan.norm_backward(y, h, None, rstd, dx, dgain=dgain, **on) == 0
    assert plan.run_mx4(q[:0], sq, W[0], SW, D[:0], **on) == 0  # nothing to do: no line
    assert plan.run_mx4(q, sq, W[0], SW, D, act=9, **on) == gm.GEMM_ERR_INVALID_ARG
    torch.cuda.synchronize()
    return y, h, rstd, q8.view(torch.uint8), s8, load, shares, factor, loss, dl, q, sq, qt, st, D, Y, v, dx, dgain, rowmap


def test_a_line_for_each_call(g, monkeypatch, capfd):
    import torch
    quiet = calls(g, g.Plan(0))
    assert "gemm_log" not in capfd.readouterr().err
    monkeypatch.setenv("GEMM_LOG", "1")
    monkeypatch.setenv("GEMM_NVTX", "1")
    loud = calls(g, g.Plan(0))
    lines = [line for line in capfd.readouterr().err.splitlines() if line.startswith("gemm_log")]
    rows = quiet[-1].numel()
    want = ["gemm_norm 40x64 bf16 residual H Y Q e4m3", "gemm_route 40x8", "gemm_route_map 40x2", "gemm_balance 40x8 f32 softmax top 2",
            "gemm_balance_backward 40x8 f32 softmax top 2 accumulated", "gemm_quantize_mx %dx64 bf16->mx4 Q QT by map" % rows,
            "gemm_run_mx %dx64x64 groups 1 mx4 mx4->f32 -> scaled" % rows, "gemm_run_grouped_mx %dx64x64 groups 8 mx4 mx4->f32 -> scaled" % rows,
            "gemm_dequantize 40x64 e4m3->bf16", "gemm_norm_backward 40x64 bf16 dgain"]
    assert len(lines) == len(want) and all(line.startswith("gemm_log " + w) for line, w in zip(lines, want)), lines
    assert all(torch.equal(a, b) for a, b in zip(quiet, loud))


def test_on_another_stream(g):
    import torch
    plan, stream = g.Plan(0), torch.cuda.Stream()
    assert all(torch.equal(a, b) for a, b in zip(calls(g, g.Plan(0)), calls(g, plan, stream.cuda_stream)))
    assert plan.poll_error() == 0


def test_without_programmatic_launches(g, monkeypatch):
    import torch
    want = calls(g, g.Plan(0))
    monkeypatch.setenv("GEMM_PDL", "0")
    assert all(torch.equal(a, b) for a, b in zip(want, calls(g, g.Plan(0))))
