"""The norm and its gradients on the GPU against 64-bit numpy (tests/more_ref.py).

Tolerance, with u = 2^-24: h is one rounding off (u).  A row's sum of squares has positive terms only; a lane adds at most 64 of them one
after another, then five exchanges and at most 16 warps: 85 u; the mean, eps and the reciprocal root add 3 u and halve what came before:
rstd is off by less than 50 u.  y adds three roundings, h * rstd * gain: 55 u of its size, below 2^-18, and its type's half a step.
dx = rstd (g - xhat mean(g xhat)) + dh: the mean is off by 90 u of the mean of |g xhat|, xhat by 50 u, the products and sums by a few more:
150 u of rstd (|g| + |xhat| mean |g xhat|) + |dh|, below 2^-16.  dgain: a sum of R terms, each 55 u off, in any order: (R + 60) u of the sum of their sizes.
The 64-bit form gets the kernel's own H and rstd where the gradients do.
"""
import numpy as np
import pytest

from tests import more_ref as ref

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f32": 1e-37, "f16": 2.0 ** -24, "bf16": 1e-37}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def g():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from dense_gemm_mma_gb300 import gemm
    return gemm


@pytest.fixture(scope="module")
def plan(g):
    return g.Plan(0)


def dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[name]


def room(n, width, name, extra=0, fill=-3.0):
    """(buffer, n x width view): rows on 16-byte boundaries, `extra` elements more apart."""
    import torch
    per = 16 // torch.empty((), dtype=dtype(name)).element_size()
    buf = torch.full((n, -(-width // per) * per + extra), fill, dtype=dtype(name), device="cuda")
    return buf, buf[:, :width]


def on(x, name, extra=0):
    import torch
    _, v = room(*x.shape, name, extra)
    v.copy_(torch.from_numpy(np.asarray(x)))
    return v


def wide(t):
    return t.double().cpu().numpy()


def near(got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


SHAPES = [(1, 1), (3, 7), (1, 4096), (5, 512), (33, 513), (130, 1024), (17, 2050), (300, 264), (4, 8200), (2, 20000), (3, 32768)]


@pytest.mark.parametrize("R,N", SHAPES)
@pytest.mark.parametrize("x_name,h_name,g_name", [("bf16", "bf16", "bf16"), ("f16", "f16", "f32"), ("f32", "f32", "f32"), ("bf16", "f32", "f32"), ("f16", "f32", "f16")])
@pytest.mark.parametrize("extra", [0, 1])
def test_norm(plan, g, R, N, x_name, h_name, g_name, extra):
    import torch
    rng = np.random.default_rng(R * 31 + N)
    X = on(rng.standard_normal((R, N)) * 10.0 ** rng.integers(-3, 3, (R, 1)), x_name, extra)
    res = on(rng.standard_normal((R, N)), h_name, extra)
    gain = torch.from_numpy(1 + 0.3 * rng.standard_normal(N)).to(dtype(g_name)).cuda()
    if R > 2:
        X[1], res[1] = 0, 0
    ybuf, Y = room(R, N, x_name, extra)
    hbuf, H = room(R, N, h_name, extra)
    rstd = torch.empty(R, device="cuda")
    for with_r, with_g, eps in ((True, True, 1e-5), (False, True, 0.5), (True, False, 1e-6)):
        assert plan.norm(X, gain if with_g else None, Y=Y, residual=res if with_r else None, H=H, rstd=rstd, eps=eps) == g.GEMM_OK
        h, rs, y = ref.norm(wide(X), wide(res) if with_r else None, wide(gain) if with_g else None, float(np.float32(eps)))
        near(wide(H), h, np.abs(h) * (HALF[h_name] + U) + LEAST[h_name])
        near(wide(rstd), rs, rs * 50 * U)
        near(wide(Y), y, np.abs(y) * (HALF[x_name] + 2.0 ** -18) + LEAST[x_name])
        assert (ybuf[:, N:] == -3).all() and (hbuf[:, N:] == -3).all()
    first = Y.clone()
    assert plan.norm(X, None, Y=Y, residual=res, eps=1e-6) == g.GEMM_OK  # without what is not wanted: the same bits
    assert torch.equal(first, Y)
    assert plan.poll_error() == g.GEMM_OK


@pytest.mark.parametrize("R,N", [(1, 4096), (3, 7), (33, 2050), (130, 513), (5, 128), (1, 9000), (129, 640)])
@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_codes(plan, g, R, N, name, fmt):
    """The codes and scales that the quantiser makes of the 32-bit result, bit for bit."""
    import torch
    rng = np.random.default_rng(R + N)
    x = rng.standard_normal((R, N)) * np.where(rng.random((1, N)) < 0.02, 100, 1)
    x[:, N // 2:] *= 1e-3
    if N > 130:
        x[R // 2, 128:] = 0
    X, res = on(x, name), on(rng.standard_normal((R, N)) * 0.1, name)
    if R > 4:
        X[4, 3] = float("nan")
        X[3, 0] = float("inf")
    gain = torch.from_numpy(1 + 0.3 * rng.standard_normal(N)).to(dtype(name)).cuda()
    ft = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt]
    ld = -(-N // 16) * 16

    def codes():
        return (torch.full((R, ld), 0xA5, dtype=torch.uint8, device="cuda"),
                torch.full((g.gemm_scale_bytes(R, N),), 0xEE, dtype=torch.uint8, device="cuda"))

    q, s = codes()
    _, Y = room(R, N, name)
    _, H = room(R, N, name)
    assert plan.norm(X, gain, Q=q[:, :N].view(ft), SQ=s, residual=res, H=H, Y=Y) == g.GEMM_OK
    y32 = torch.empty((R, N), device="cuda")
    q2, s2 = codes()
    assert plan.norm(X.float(), gain.float(), Y=y32, residual=res.float()) == g.GEMM_OK
    assert plan.quantize(y32, q2[:, :N].view(ft), s2) == g.GEMM_OK
    assert torch.equal(s, s2)
    assert torch.equal(q, q2)
    assert torch.equal(Y.view(torch.int16 if name == "bf16" else torch.int32), y32.to(dtype(name)).view(torch.int16 if name == "bf16" else torch.int32)) or R > 4
    alone, s3 = codes()
    assert plan.norm(X, gain, Q=alone[:, :N].view(ft), SQ=s3, residual=res) == g.GEMM_OK
    assert torch.equal(alone, q) and torch.equal(s3, s)


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_in_place(plan, g, name):
    import torch
    x, r = torch.randn((70, 1032), device="cuda").to(dtype(name)), torch.randn((70, 1032), device="cuda").to(dtype(name))
    Y, H = torch.empty_like(x), torch.empty_like(x)
    assert plan.norm(x, Y=Y, residual=r, H=H) == g.GEMM_OK
    a, b = x.clone(), r.clone()
    assert plan.norm(a, Y=a, residual=b, H=b) == g.GEMM_OK  # the usual form between two layers
    assert torch.equal(a, Y) and torch.equal(b, H)
    a, b = x.clone(), r.clone()
    assert plan.norm(a, Y=b, residual=b, H=a) == g.GEMM_OK
    assert torch.equal(b, Y) and torch.equal(a, H)
    rstd, dgain = torch.empty(70, device="cuda"), torch.empty(1032, device="cuda")
    plan.norm(x, Y=Y, residual=r, H=H, rstd=rstd)
    dy, dh, dx = torch.randn_like(x), torch.randn_like(x), torch.empty_like(x)
    assert plan.norm_backward(dy, H, None, rstd, dx, dgain=dgain, dH=dh) == g.GEMM_OK
    for over in (dy, dh):
        y2, h2 = dy.clone(), dh.clone()
        into = y2 if over is dy else h2
        again = torch.empty_like(dgain)
        assert plan.norm_backward(y2, H, None, rstd, into, dgain=again, dH=h2) == g.GEMM_OK
        assert torch.equal(into, dx) and torch.equal(again, dgain)


@pytest.mark.parametrize("R,N", SHAPES + [(0, 40), (2000, 520)])
@pytest.mark.parametrize("x_name,h_name,g_name", [("bf16", "bf16", "bf16"), ("f16", "f32", "f32"), ("f32", "f32", "f32")])
@pytest.mark.parametrize("extra", [0, 1])
def test_gradients(plan, g, R, N, x_name, h_name, g_name, extra):
    import torch
    rng = np.random.default_rng(R * 13 + N)
    H, dy = on(rng.standard_normal((R, N)) * 3, h_name, extra), on(rng.standard_normal((R, N)), x_name, extra)
    dh = on(rng.standard_normal((R, N)), h_name, extra)
    gain = torch.from_numpy(1 + 0.3 * rng.standard_normal(N)).to(dtype(g_name)).cuda()
    rstd = torch.from_numpy((1 / np.sqrt((wide(H) ** 2).mean(1) + 1e-6)).astype(np.float32)).cuda()
    for with_g, with_h in ((True, True), (False, False), (True, False)):
        buf, dx = room(R, N, h_name, extra)
        dgain = torch.full((N,), float("nan"), device="cuda")
        args = (dy, H, gain if with_g else None, rstd, dx)
        assert plan.norm_backward(*args, dgain=dgain, dH=dh if with_h else None) == g.GEMM_OK
        want, wgain, size, gsize = ref.norm_backward(wide(dy), wide(H), wide(gain) if with_g else None, wide(rstd), wide(dh) if with_h else None)
        near(wide(dx), want, size * 2.0 ** -16 + np.abs(want) * HALF[h_name] + LEAST[h_name])
        near(wide(dgain), wgain, gsize * (R + 60) * U + 1e-37)
        assert (buf[:, N:] == -3).all()
        alone, again = torch.empty_like(dx), torch.empty_like(dgain)
        assert plan.norm_backward(*args[:4], alone, dH=dh if with_h else None) == g.GEMM_OK  # without the gain's
        assert torch.equal(alone, dx)
        plan.norm_backward(*args[:4], alone, dgain=again, dH=dh if with_h else None)
        assert torch.equal(again, dgain)  # the same bits every time
    assert plan.poll_error() == g.GEMM_OK


def test_gradients_against_differences(plan, g):
    """The sum of w * y, as the kernel computes it in fp32, moves with x and gain as the gradients say."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    x, gain, w = rand(4, 40), 1 + 0.2 * rand(40), rand(4, 40)
    Y, H, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(4, device="cuda")

    def loss(x, gain):
        assert plan.norm(x, gain, Y=Y, H=H, rstd=rstd) == g.GEMM_OK
        return float((Y.double() * w.double()).sum())

    loss(x, gain)
    dx, dgain = torch.empty_like(x), torch.empty_like(gain)
    assert plan.norm_backward(w, H, gain, rstd, dx, dgain=dgain) == g.GEMM_OK
    step = 2.0 ** -7  # curvature ~ step^2 |d3| / 6 ~ 1e-5; rounding: 160 values 55 u off over 2 steps ~ 1e-4 at worst
    for k in range(6):
        d, dg = rand(4, 40), rand(40)
        d, dg = d / d.norm(), dg / dg.norm()
        diff = (loss(x + step * d, gain) - loss(x - step * d, gain)) / (2 * step)
        assert abs(diff - float((dx * d).sum())) < 2e-3
        diff = (loss(x, gain + step * dg) - loss(x, gain - step * dg)) / (2 * step)
        assert abs(diff - float((dgain * dg).sum())) < 2e-3


def test_rows_without_a_norm(plan, g):
    """Zeros with eps, infinities and NaN stay in their rows."""
    import torch
    x = torch.randn((6, 600), device="cuda")
    x[1], x[2, 5], x[3, 7] = 0, float("inf"), float("nan")
    Y, rstd = torch.empty_like(x), torch.empty(6, device="cuda")
    assert plan.norm(x, Y=Y, rstd=rstd, eps=1e-6) == g.GEMM_OK
    assert (Y[1] == 0).all() and abs(float(rstd[1]) - 1e3) < 1e-3
    assert rstd[2] == 0 and torch.isnan(Y[2, 5]) and (Y[2, :5] == 0).all()
    assert torch.isnan(rstd[3]) and torch.isnan(Y[3]).all()
    assert torch.isfinite(Y[[0, 1, 4, 5]]).all()


def test_on_a_stream_and_in_a_graph(g):
    """A plan's first calls, workspace included, captured; replayed with new inputs."""
    import torch
    plan = g.Plan(0)
    x, r, dy = (torch.zeros((500, 520), device="cuda") for _ in range(3))
    Y, H, dx = (torch.empty_like(x) for _ in range(3))
    rstd, dgain = torch.empty(500, device="cuda"), torch.empty(520, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        assert plan.norm(x, Y=Y, residual=r, H=H, rstd=rstd) == g.GEMM_OK
        assert plan.norm_backward(dy, H, None, rstd, dx, dgain=dgain) == g.GEMM_OK
    rng = np.random.default_rng(2)
    for _ in range(2):
        for t in (x, r, dy):
            t.copy_(torch.from_numpy(rng.standard_normal((500, 520))))
        graph.replay()
        torch.cuda.synchronize()
        _, rs, y = ref.norm(wide(x), wide(r), None, 1e-6)
        near(wide(Y), y, np.abs(y) * 2.0 ** -17 + 1e-37)
        want, wgain, size, gsize = ref.norm_backward(wide(dy), wide(H), None, wide(rstd), None)
        near(wide(dx), want, size * 2.0 ** -16)
        near(wide(dgain), wgain, gsize * 560 * U)


def test_refusals(plan, g):
    import torch
    x, r, y, h = (torch.zeros((8, 64), device="cuda") for _ in range(4))
    gain, rstd, dgain = torch.ones(64, device="cuda"), torch.zeros(8, device="cuda"), torch.zeros(64, device="cuda")
    q, s = torch.zeros((8, 64), dtype=torch.uint8, device="cuda"), torch.zeros(512, dtype=torch.uint8, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    call = lambda **c: g.gemm_norm(*{**dict(  # noqa: E731
        plan=plan.handle, rows=8, cols=64, X=p(x), ldx=64, x_type=2, residual=p(r), ldr=64, h_type=2, gain=p(gain), g_type=2, eps=1e-6,
        H=p(h), ldh=64, Y=p(y), ldy=64, q_type=4, Q=p(q), ldq=64, SQ=p(s), rstd=p(rstd)), **c}.values())
    assert call() == g.GEMM_OK and call(rows=0, X=None) == g.GEMM_OK and call(cols=0) == g.GEMM_OK
    assert call(H=p(r)) == g.GEMM_OK and call(Y=p(x)) == g.GEMM_OK and call(H=p(x), Y=p(r)) == g.GEMM_OK
    for bad in ({"plan": None}, {"rows": -1}, {"cols": -1}, {"x_type": 4}, {"h_type": 0}, {"g_type": 1}, {"eps": -1.0}, {"eps": float("nan")},
                {"eps": float("inf")}, {"SQ": None}, {"Q": None}, {"q_type": 2}, {"H": None, "Y": None, "Q": None, "SQ": None, "rstd": None},
                {"ldx": 63}, {"ldr": 63}, {"ldh": 63}, {"ldy": 63}, {"ldq": 48}, {"X": None}, {"H": p(y)}, {"Y": p(x) + 256}, {"H": p(x), "Y": p(x)},
                {"rstd": p(gain)}, {"rstd": p(x)}, {"Q": p(x)}, {"SQ": p(q)}, {"H": p(x), "ldh": 72}, {"Y": p(gain)}):
        assert call(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    for bad in ({"X": p(x) + 2}, {"Q": p(q) + 8}, {"ldq": 72}, {"SQ": p(s) + 4}, {"rstd": p(rstd) + 1}):
        assert call(**bad) == g.GEMM_ERR_ALIGNMENT, bad
    assert call(cols=32769, ldx=2 ** 16, ldr=2 ** 16, ldh=2 ** 16, ldy=2 ** 16, ldq=2 ** 16) == g.GEMM_ERR_UNSUPPORTED
    back = lambda **c: g.gemm_norm_backward(*{**dict(  # noqa: E731
        plan=plan.handle, rows=8, cols=64, dY=p(y), lddy=64, x_type=2, H=p(h), ldh=64, h_type=2, gain=p(gain), g_type=2, rstd=p(rstd),
        dH=p(r), lddh=64, dX=p(x), lddx=64, dgain=p(dgain)), **c}.values())
    assert back() == g.GEMM_OK and back(dX=p(y)) == g.GEMM_OK and back(dX=p(r)) == g.GEMM_OK and back(rows=0, dgain=None) == g.GEMM_OK
    for bad in ({"plan": None}, {"rows": -1}, {"x_type": 4}, {"h_type": 1}, {"dY": None}, {"H": None}, {"rstd": None}, {"dX": None}, {"dX": p(h)},
                {"dX": p(y) + 256}, {"dgain": p(gain)}, {"dgain": p(y)}, {"dgain": p(x)}, {"lddx": 63}, {"dX": p(r), "lddx": 72}):
        assert back(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    assert back(dX=p(x) + 2) == g.GEMM_ERR_ALIGNMENT
    with pytest.raises(ValueError):
        plan.norm(x, gain[:60], Y=y)
    with pytest.raises(ValueError):
        plan.norm(x, gain, Y=y.bfloat16())
    with pytest.raises(ValueError):
        plan.norm(x, gain, Y=y[:, :60])
    with pytest.raises(ValueError):
        plan.norm_backward(y, h, gain, rstd, x.bfloat16())
