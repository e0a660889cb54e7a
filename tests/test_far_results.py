"""Results whose rows lie further apart than 32 bits count have the bits of results close together: values of far codes, far
codes and transposed codes of the 4-bit quantiser, far sums, codes and gradients of the norm; and a norm's result beside its
codes, rows with NaN and infinities among them."""
import pytest

from tests.test_more_far import far, g  # noqa: F401  (g: a fixture)

pytestmark = pytest.mark.gpu

LD = (1 << 30) + 8  # elements; of bytes: four times that


def bits(t):
    import torch
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def test_values_of_far_codes(g):  # noqa: F811
    import torch
    plan = g.Plan(0)
    R, N = 5, 264
    x = torch.randn((R, N), device="cuda", dtype=torch.bfloat16)
    q, s = torch.zeros((R, N // 2), dtype=torch.uint8, device="cuda"), torch.empty(g.gemm_mx_scale_bytes(R, N), dtype=torch.uint8, device="cuda")
    q8, s8 = torch.zeros((R, 272), dtype=torch.uint8, device="cuda")[:, :N].view(torch.float8_e4m3fn), torch.empty(g.gemm_scale_bytes(R, N), dtype=torch.uint8, device="cuda")
    assert plan.quantize_mx4(x, q, s) == g.GEMM_OK and plan.quantize(x, q8, s8) == g.GEMM_OK
    for codes, scales in ((q, s), (q8, s8)):
        near, got = torch.zeros_like(x), torch.zeros_like(x)
        assert plan.dequantize(codes, scales, near) == g.GEMM_OK
        away = far(codes.view(torch.uint8), (1 << 31) - 16).view(codes.dtype)
        assert plan.dequantize(away, scales, got) == g.GEMM_OK
        assert torch.equal(got, near) and got.abs().max() > 0
    assert plan.poll_error() == g.GEMM_OK


def test_far_codes(g):  # noqa: F811
    import torch
    plan = g.Plan(0)
    R, N, ld = 5, 70, (1 << 31) - 16  # Q: past 2^32 bytes at its third row; QT: 70 rows, so that these are nearer one another
    new = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    for name in (torch.bfloat16, torch.float32):
        x = torch.randn((R, N), device="cuda").to(name)
        q, qt, s, st = new(R, 35), new(N, 3), new(g.gemm_mx_scale_bytes(R, N)), new(g.gemm_mx_scale_bytes(N, R))
        assert plan.quantize_mx4(x, q, s, qt, st) == g.GEMM_OK
        for both in (False, True):
            away, s2 = far(new(R, 35), ld), torch.empty_like(s)
            away_t, st2 = far(new(N, 3), (1 << 27) + 1), torch.empty_like(st)
            assert plan.quantize_mx4(x, away, s2, *((away_t, st2) if both else (None, None))) == g.GEMM_OK
            assert torch.equal(away, q) and torch.equal(s2, s)
            if both:
                assert torch.equal(away_t, qt) and torch.equal(st2, st)
            del away, away_t
    assert plan.poll_error() == g.GEMM_OK


def test_far_norm(g):  # noqa: F811
    import torch
    plan = g.Plan(0)
    R, N = 5, 264
    x, r, dy = (torch.randn((R, N), device="cuda", dtype=torch.bfloat16) for _ in range(3))
    H, Y, rstd, dx, dgain = torch.empty_like(x), torch.empty_like(x), torch.empty(R, device="cuda"), torch.empty_like(x), torch.empty(N, device="cuda")
    codes = lambda: torch.zeros((R, 272), dtype=torch.uint8, device="cuda")[:, :N]  # noqa: E731
    q, s = codes(), torch.empty(g.gemm_scale_bytes(R, N), dtype=torch.uint8, device="cuda")
    assert plan.norm(x, Y=Y, Q=q.view(torch.float8_e4m3fn), SQ=s, residual=r, H=H, rstd=rstd) == g.GEMM_OK
    assert plan.norm_backward(dy, H, None, rstd, dx, dgain=dgain, dH=r) == g.GEMM_OK
    hf, qf, s2 = far(torch.zeros_like(x), LD), far(codes(), (1 << 31) - 16), torch.empty_like(s)
    assert plan.norm(x, Q=qf.view(torch.float8_e4m3fn), SQ=s2, residual=r, H=hf) == g.GEMM_OK
    assert torch.equal(hf, H) and torch.equal(qf, q) and torch.equal(s2, s)
    got, again = far(torch.zeros_like(x), LD), torch.empty_like(dgain)
    assert plan.norm_backward(dy, hf, None, rstd, got, dgain=again, dH=r) == g.GEMM_OK
    assert torch.equal(got, dx) and torch.equal(again, dgain)
    del hf, qf
    into = far(r, LD)  # a far gradient past the norm, and dX in its place
    assert plan.norm_backward(dy, H, None, rstd, into, dH=into) == g.GEMM_OK
    assert torch.equal(into, dx)
    del into, got
    x = torch.randn((3, 9000), device="cuda", dtype=torch.bfloat16)  # rows that are read twice
    H, Y, rstd, dx = torch.empty_like(x), torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty_like(x)
    assert plan.norm(x, Y=Y, H=H, rstd=rstd) == g.GEMM_OK and plan.norm_backward(Y, H, None, rstd, dx) == g.GEMM_OK
    hf, got = far(torch.zeros_like(x), 2 * LD), far(torch.zeros_like(x), 2 * LD)
    assert plan.norm(x, Y=Y, H=hf) == g.GEMM_OK and torch.equal(hf, H)
    assert plan.norm_backward(Y, hf, None, rstd, got) == g.GEMM_OK and torch.equal(got, dx)
    assert plan.poll_error() == g.GEMM_OK


@pytest.mark.parametrize("R,N", [(5, 128), (33, 2050), (130, 513), (129, 640), (7, 9000)])
@pytest.mark.parametrize("name", ["bfloat16", "float32"])
def test_result_beside_its_codes(g, R, N, name):  # noqa: F811
    """Y written together with codes is Y written alone, and the 32-bit result rounded once; NaN where that has NaN."""
    import torch
    plan, t = g.Plan(0), getattr(torch, name)
    x, r = torch.randn((R, N), device="cuda").to(t), (0.1 * torch.randn((R, N), device="cuda")).to(t)
    x[4, 3], x[3, 0] = float("nan"), float("inf")
    gain = (1 + 0.3 * torch.randn(N, device="cuda")).to(t)
    q = torch.empty((R, -(-N // 16) * 16), dtype=torch.uint8, device="cuda")[:, :N].view(torch.float8_e4m3fn)
    s = torch.empty(g.gemm_scale_bytes(R, N), dtype=torch.uint8, device="cuda")
    Y, alone, y32 = torch.empty_like(x), torch.empty_like(x), torch.empty((R, N), device="cuda")
    assert plan.norm(x, gain, Y=Y, Q=q, SQ=s, residual=r) == g.GEMM_OK
    assert plan.norm(x, gain, Y=alone, residual=r) == g.GEMM_OK
    assert plan.norm(x.float(), gain.float(), Y=y32, residual=r.float(), Q=q, SQ=s) == g.GEMM_OK
    nan = torch.isnan(y32)
    assert nan[4].all() and nan[3, 0] and int(nan.sum()) == N + 1 and (y32[3, 1:] == 0).all()
    want = y32.to(t)
    assert torch.equal(torch.isnan(Y), nan) and torch.equal(bits(Y.masked_fill(nan, 0)), bits(want.masked_fill(nan, 0)))
    # the same row's sum of squares is added in another order where the shapes of the two kernels differ: 100 u of the sum, 55 u of the root
    a, b = alone.masked_fill(nan, 0).double(), Y.masked_fill(nan, 0).double()
    step = 2.0 ** -7 if name == "bfloat16" else 2.0 ** -18
    assert torch.equal(torch.isnan(alone), nan) and ((a - b).abs() <= b.abs() * step + 1e-37).all()
    assert plan.poll_error() == g.GEMM_OK
