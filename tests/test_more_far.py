"""Rows that lie further apart than 32 bits count: the norm, the 4-bit quantiser, the values of codes, the 4-bit product and the
balance loss give the bits that they give on rows close together."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from dense_gemm_mma_gb300 import gemm
    return gemm


def far(x, ld):
    """x with its rows ld elements apart (views of one buffer past 2^32 bytes)."""
    import torch
    buf = torch.empty((x.shape[0] - 1) * ld + x.shape[1], dtype=x.dtype, device="cuda")
    v = buf.as_strided(x.shape, (ld, 1))
    v.copy_(x)
    return v


def test_far_rows(g):
    import torch
    plan = g.Plan(0)
    R, N, ld = 5, 264, (1 << 30) + 8  # 4 * 2^30 elements: past 2^32 elements and, 16 bits each, 2^33 bytes
    x = torch.randn((R, N), device="cuda", dtype=torch.bfloat16)
    xf = far(x, ld)
    y, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(R, device="cuda")
    assert plan.norm(x, Y=y, residual=x, H=h, rstd=rstd) == g.GEMM_OK
    yf = far(torch.zeros_like(x), ld)
    assert plan.norm(xf, Y=yf, residual=xf) == g.GEMM_OK
    assert torch.equal(yf, y)
    dx, dgain, dgain2 = torch.empty_like(x), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    assert plan.norm_backward(x, h, None, rstd, dx, dgain=dgain) == g.GEMM_OK
    assert plan.norm_backward(xf, h, None, rstd, yf, dgain=dgain2) == g.GEMM_OK
    assert torch.equal(yf, dx) and torch.equal(dgain2, dgain)

    new = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    size = g.gemm_mx_scale_bytes(R, N)
    q, s, q2, s2 = new(R, 144)[:, :132], new(size), new(R, 144)[:, :132], new(size)
    assert plan.quantize_mx4(x, q, s) == g.GEMM_OK and plan.quantize_mx4(xf, q2, s2) == g.GEMM_OK
    assert torch.equal(q, q2) and torch.equal(s, s2)
    v = torch.empty_like(x)
    assert plan.dequantize(q, s, v) == g.GEMM_OK and plan.dequantize(q, s, yf) == g.GEMM_OK
    assert torch.equal(yf, v)
    del xf, yf
    qf = far(q, (1 << 31) - 16)  # 2^33 bytes
    assert plan.dequantize(qf, s, v.zero_()) == g.GEMM_OK
    D, D2 = torch.empty((R, R + 3), device="cuda"), torch.empty((R, R + 3), device="cuda")
    assert plan.run_mx4(q, s, q, s, D[:, :R].as_strided((R, R), (8, 1)), K=N) == g.GEMM_OK
    for kernel_operand in ((qf, q), (q, qf)):
        assert plan.run_mx4(kernel_operand[0], s, kernel_operand[1], s, D2[:, :R], K=N) == g.GEMM_OK
        assert torch.equal(D2[:, :R], D[:, :R])
    del qf

    E = 16
    logits = torch.randn((R, E), device="cuda")
    lf = far(logits, ld)
    index = torch.zeros((R, 2), dtype=torch.int32, device="cuda")
    outs = []
    for lg in (logits, lf):
        c, p, f, loss = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E, device="cuda"), torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
        assert plan.balance(lg, index, c, p, f, loss) == g.GEMM_OK
        dl = torch.zeros_like(logits)
        assert plan.balance_backward(lg, index, f, dl) == g.GEMM_OK
        outs.append((c, p, f, loss, dl))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert plan.balance_backward(logits, index, outs[0][2], lf) == g.GEMM_OK
    assert torch.equal(lf, outs[0][4])
    assert plan.poll_error() == g.GEMM_OK
