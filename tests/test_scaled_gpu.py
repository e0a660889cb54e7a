"""The quantiser and the block-scaled products on the GPU against 64-bit numpy
(tests/scaled_ref.py).

Quantiser: codes and scale bytes are whole numbers and have to be equal.

Products, tolerance: the tensor core multiplies 8-bit values exactly and adds the 32
products of an MMA into an fp32 accumulator, K/32 times.  With S = sum |a b| (an upper bound
of every partial sum), each of the K/32 additions, and the sum inside an MMA, is off by
at most two units of 2^-23 S: (K/32 + 1) * 2^-22 * S, to which the K slices of a cluster add
eight more additions.  alpha, beta and the activation (slope at most 1.13, expf and
erfcf to 2^-20) scale that and add 2^-20 of the result; the result's rounding adds half a unit:
2^-24, 2^-11 (f16) or 2^-8 (bf16) of its size, and f16's least step.
"""
import itertools
import os

import numpy as np
import pytest

from tests import scaled_ref as ref

pytestmark = pytest.mark.gpu

ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


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
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
            "e5m2": torch.float8_e5m2}[name]


def rows_of(n, width, name, fill=None, extra=0):
    """n x width view of a buffer whose rows start on 16-byte boundaries; the buffer is filled with `fill` bytes."""
    import torch
    es = torch.empty((), dtype=dtype(name)).element_size()
    ld = -(-max(width, 1) * es // 16) * 16 // es + extra
    buf = torch.full((n * ld * es,), 0 if fill is None else fill, dtype=torch.uint8, device="cuda").view(dtype(name)).view(n, ld)
    return buf, buf[:, :width]


def operand(rng, rows, K, fmt, spread=4):
    """Random codes (device view, packed scales, element values in 64 bits)."""
    import torch
    codes = rng.integers(0, 256, (rows, K))
    bad = np.isnan(ref.decode(codes, fmt)) | np.isinf(ref.decode(codes, fmt))
    codes[bad] = 0
    if fmt == "e5m2":  # keep the sums within fp32: magnitudes up to 2^4
        codes = np.where(np.abs(ref.decode(codes, fmt)) > 16, codes & 0xBF, codes)
    byte = rng.integers(127 - spread, 127 + spread, (rows, -(-K // 128)))
    buf, view = rows_of(rows, K, fmt, fill=0x7F)  # NaN beyond the rows' ends: not to be read as operands
    view.view(torch.uint8).copy_(torch.from_numpy(codes.astype(np.uint8)))
    return view, torch.from_numpy(ref.pack(byte, K)).cuda(), ref.scaled(ref.decode(codes, fmt), byte)


def expect(a, b, alpha=1.0, beta=0.0, c=None, act=0, slope=0.0):
    """(result in 64 bits, what its accumulator may be off by)."""
    y = alpha * (a @ b.T)
    off = abs(alpha) * (np.abs(a) @ np.abs(b).T) * (a.shape[1] / 32 + 9) * 2.0 ** -22
    if beta:
        y = y + beta * c
        off = off + np.abs(beta * c) * 2.0 ** -22
    return ref.act(y, act, slope), off * 1.13


def near(got, want, off, out):
    got = got.double().cpu().numpy()
    tol = off + np.abs(want) * (2.0 ** -20 + ROUND[out]) + (2.0 ** -24 if out == "f16" else 1e-37)
    if out == "f16":  # past f16's largest value the result rounds to infinity
        got, want = (np.where(np.abs(v) >= 65520, np.sign(v) * 65520, v) for v in (got, want))
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


# ------------------------------------------------------------------ quantiser

def values(rng, R, K, name):
    import torch
    x = rng.standard_normal((R, K)) * 10.0 ** rng.integers(-5, 4, (R, 1))
    x[:, :: 7] *= 50
    if R > 2:
        x[2] = 0
    if K > 130:
        x[R // 2, 128:] = 1e-30 if name != "f16" else 6e-8  # a block of the smallest values
    x.reshape(-1)[:: 97] = 448.0  # on the rounding's edges: the largest code, a tie, just past it
    if R > 5:
        x[5, : K // 2] = np.resize([1.75, 1.8125, 1.8126, 3.5, 1.0, -0.0], K // 2)
    if R > 6 and K > 3:
        x[6, 1], x[6, 2], x[6, K - 1] = np.inf, np.nan, -np.inf
    return torch.from_numpy(x).to(dtype(name))


@pytest.mark.parametrize("R,K", [(1, 1), (1, 128), (7, 127), (33, 2050), (127, 129), (128, 512), (129, 640), (300, 517)])
@pytest.mark.parametrize("name", ["bf16", "f16", "f32"])
def test_quantize(plan, g, R, K, name):
    import torch
    rng = np.random.default_rng(R * 1000 + K)
    x = values(rng, R, K, name)
    for fmt, block, both, odd in itertools.product(("e4m3", "e5m2"), (1, 128), (False, True), (False, True)):
        buf, xd = rows_of(R, K, name, extra=1 if odd else 0)  # odd rows: no wide loads
        xd.copy_(x)
        want, byte = ref.quantize(x.double().numpy(), fmt, block)
        qbuf, q = rows_of(R, K, fmt, fill=0xA5)
        sq = torch.full((g.gemm_scale_bytes(R, K),), 0xEE, dtype=torch.uint8, device="cuda")
        tbuf, qt = rows_of(K, R, fmt, fill=0xA5)
        st = torch.full((g.gemm_scale_bytes(K, R),), 0xEE, dtype=torch.uint8, device="cuda")
        assert plan.quantize(xd, q, sq, *((qt, st) if both else ()), block_rows=block) == 0
        got = ref.decode(q.view(torch.uint8).cpu().numpy(), fmt)
        np.testing.assert_array_equal(got, want)
        np.testing.assert_array_equal(sq.cpu().numpy(), ref.pack(byte, K))
        assert (qbuf.view(torch.uint8)[:, K:] == 0xA5).all()
        if both:
            want_t, byte_t = ref.quantize(x.double().numpy().T, fmt, block)
            np.testing.assert_array_equal(ref.decode(qt.view(torch.uint8).cpu().numpy(), fmt), want_t)
            np.testing.assert_array_equal(st.cpu().numpy(), ref.pack(byte_t, R))
            assert (tbuf.view(torch.uint8)[:, R:] == 0xA5).all()
    assert plan.poll_error() == 0


def test_quantize_through_a_row_map(plan, g):
    import torch
    rng = np.random.default_rng(5)
    T, k, K = 50, 3, 300
    x = values(rng, T, K, "bf16")
    rows = 700
    rowmap = np.full(rows, -1)
    rowmap[rng.permutation(rows)[:T * k]] = np.arange(T * k)
    rowmap[0], rowmap[1] = T * k, 2 ** 31 - 1  # past X: no row
    src = np.where((rowmap >= 0) & (rowmap < T * k), rowmap // k, -1)
    moved = np.where((src >= 0)[:, None], x.double().numpy()[src], 0.0)
    for both in (False, True):
        qbuf, q = rows_of(rows, K, "e4m3", fill=0xA5)
        sq = torch.full((g.gemm_scale_bytes(rows, K),), 0xEE, dtype=torch.uint8, device="cuda")
        _, qt = rows_of(K, rows, "e4m3", fill=0xA5)
        st = torch.full((g.gemm_scale_bytes(K, rows),), 0xEE, dtype=torch.uint8, device="cuda")
        assert plan.quantize(x.cuda(), q, sq, *((qt, st) if both else ()), map_div=k,
                             rowmap=torch.from_numpy(rowmap.astype(np.int32)).cuda()) == 0
        want, byte = ref.quantize(moved, "e4m3")
        got = ref.decode(q.view(torch.uint8).cpu().numpy(), "e4m3")
        np.testing.assert_array_equal(got[src >= 0], want[src >= 0])
        assert (q.view(torch.uint8)[torch.from_numpy(src < 0).cuda()] == 0xA5).all()  # rows without a source: left
        np.testing.assert_array_equal(sq.cpu().numpy(), ref.pack(byte, K))
        if both:
            want, byte = ref.quantize(moved.T, "e4m3")
            np.testing.assert_array_equal(ref.decode(qt.view(torch.uint8).cpu().numpy(), "e4m3"), want)
            np.testing.assert_array_equal(st.cpu().numpy(), ref.pack(byte, rows))


@pytest.mark.parametrize("name,fmt", [("bf16", "e4m3"), ("f32", "e5m2")])
def test_quantize_square_scales_with_every_sm_full(plan, g, name, fmt):
    """128 x 128 scales of both orientations while several CTAs share an SM and their warps are held up: a
    tile's largest value lies in its first 32 columns, so that a warp of the other columns that took the scale
    from anything but the whole tile would choose a smaller one.  The same bits every time."""
    import torch
    rng = np.random.default_rng(12)
    R, K = 3000, 2500
    x = rng.standard_normal((R, K))
    for b in range(0, K, 128):
        x[rng.integers(0, 128) % min(128, R):: 128, b + rng.integers(0, min(32, K - b))] = 1000.0 * (1 + b)
    _, xd = rows_of(R, K, name)
    xd.copy_(torch.from_numpy(x))
    want, byte = ref.quantize(xd.double().cpu().numpy(), fmt, 128)
    want_t, byte_t = ref.quantize(xd.double().cpu().numpy().T, fmt, 128)
    first = None
    for _ in range(8):
        _, q = rows_of(R, K, fmt)
        _, qt = rows_of(K, R, fmt)
        sq = torch.full((g.gemm_scale_bytes(R, K),), 0xEE, dtype=torch.uint8, device="cuda")
        st = torch.full((g.gemm_scale_bytes(K, R),), 0xEE, dtype=torch.uint8, device="cuda")
        assert plan.quantize(xd, q, sq, qt, st, block_rows=128) == 0
        got = [v.view(torch.uint8).contiguous().cpu() for v in (q, sq, qt, st)]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    np.testing.assert_array_equal(ref.decode(first[0].numpy(), fmt), want)
    np.testing.assert_array_equal(first[1].numpy(), ref.pack(byte, K))
    np.testing.assert_array_equal(ref.decode(first[2].numpy(), fmt), want_t)
    np.testing.assert_array_equal(first[3].numpy(), ref.pack(byte_t, R))


@pytest.mark.parametrize("both", [False, True])
def test_square_scales_through_a_row_map(plan, g, both):
    """With 128 x 128 scales too, a row without a source has scale bytes of 0, and its codes are left; it
    takes no part in its block's scale, and its column of the transposed matrix is zero."""
    import torch
    rng = np.random.default_rng(13)
    T, k, K, rows = 90, 2, 300, 500
    x = values(rng, T, K, "bf16")
    rowmap = np.full(rows, -1)
    rowmap[rng.permutation(rows - 200)[:T * k]] = np.arange(T * k)  # (the last tile has no row at all)
    rowmap[rows - 1] = T * k  # past X
    src = np.where((rowmap >= 0) & (rowmap < T * k), rowmap // k, -1)
    moved = np.where((src >= 0)[:, None], x.double().numpy()[src], 0.0)
    _, q = rows_of(rows, K, "e4m3", fill=0xA5)
    sq = torch.full((g.gemm_scale_bytes(rows, K),), 0xEE, dtype=torch.uint8, device="cuda")
    _, qt = rows_of(K, rows, "e4m3", fill=0xA5)
    st = torch.full((g.gemm_scale_bytes(K, rows),), 0xEE, dtype=torch.uint8, device="cuda")
    assert plan.quantize(x.cuda(), q, sq, *((qt, st) if both else ()), map_div=k, block_rows=128,
                         rowmap=torch.from_numpy(rowmap.astype(np.int32)).cuda()) == 0
    want, byte = ref.quantize(moved, "e4m3", 128)
    got = ref.decode(q.view(torch.uint8).cpu().numpy(), "e4m3")
    np.testing.assert_array_equal(got[src >= 0], want[src >= 0])
    assert (q.view(torch.uint8)[torch.from_numpy(src < 0).cuda()] == 0xA5).all()
    byte[src < 0] = 0
    np.testing.assert_array_equal(sq.cpu().numpy(), ref.pack(byte, K))
    if both:
        want, byte = ref.quantize(moved.T, "e4m3", 128)
        np.testing.assert_array_equal(ref.decode(qt.view(torch.uint8).cpu().numpy(), "e4m3"), want)
        np.testing.assert_array_equal(st.cpu().numpy(), ref.pack(byte, rows))


def test_quantize_refusals(plan, g):
    import torch
    x = torch.zeros((8, 64), device="cuda", dtype=torch.bfloat16)
    q = torch.zeros((8, 64), device="cuda", dtype=torch.float8_e4m3fn)
    s = torch.zeros(512, device="cuda", dtype=torch.uint8)
    call = lambda **c: g.gemm_quantize(*{**dict(  # noqa: E731
        plan=plan.handle, rows=8, cols=64, X=x.data_ptr(), ldx=64, x_type=0, rowmap=None, map_div=1, src_rows=8, q_type=4,
        block_rows=1, Q=q.data_ptr(), ldq=64, SQ=s.data_ptr(), QT=None, ldqt=0, SQT=None), **c}.values())
    assert call() == g.GEMM_OK and call(rows=0) == g.GEMM_OK and call(cols=0) == g.GEMM_OK
    for bad in ({"rows": -1}, {"x_type": 4}, {"q_type": 0}, {"block_rows": 2}, {"Q": None}, {"SQ": None}, {"ldx": 63},
                {"ldq": 48}, {"X": None}, {"Q": x.data_ptr()}, {"SQ": q.data_ptr()}, {"QT": q.data_ptr()}):
        assert call(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    for bad in ({"Q": q.data_ptr() + 8}, {"ldq": 72}, {"SQ": s.data_ptr() + 4}, {"X": x.data_ptr() + 1}):
        assert call(**bad) == g.GEMM_ERR_ALIGNMENT, bad
    assert call(rows=2 ** 24) == g.GEMM_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        plan.quantize(x, q, s[:100])


def test_quantize_refuses_runs_of_bytes_that_meet(plan, g):
    """Scales over scales, over the map or over a single row: runs of bytes without a pitch."""
    import torch
    x = torch.zeros((1, 64), device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(64, device="cuda", dtype=torch.uint8)
    qt = torch.zeros(64 * 16, device="cuda", dtype=torch.uint8)
    s = torch.zeros(4096, device="cuda", dtype=torch.uint8)
    base, rowmap = s.data_ptr(), s.data_ptr() + 2048
    call = lambda **c: g.gemm_quantize(*{**dict(  # noqa: E731
        plan=plan.handle, rows=1, cols=64, X=x.data_ptr(), ldx=64, x_type=0, rowmap=rowmap, map_div=1, src_rows=1, q_type=4,
        block_rows=1, Q=q.data_ptr(), ldq=64, SQ=base, QT=qt.data_ptr(), ldqt=16, SQT=base + 512), **c}.values())
    assert call() == g.GEMM_OK
    for bad in ({"SQT": base}, {"SQT": base + 496}, {"SQ": rowmap - 496}, {"SQT": rowmap}, {"SQ": q.data_ptr()}, {"Q": base + 480},
                {"SQ": x.data_ptr()}):
        assert call(**bad) == g.GEMM_ERR_INVALID_ARG, bad


# ------------------------------------------------------------------- products

KERNELS = [None, "tile", "pair", "sliced"]
SHAPES = [(1, 1, 1), (1, 300, 130), (2, 128, 1024), (31, 257, 515), (33, 96, 640), (64, 640, 2050), (95, 200, 128), (128, 130, 127),
          (129, 127, 777), (200, 520, 1500), (300, 264, 384), (513, 776, 300)]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(plan, g, monkeypatch, kernel, M, N, K):
    import torch
    if kernel:
        monkeypatch.setenv("GEMM_SCALED_KERNEL", kernel)
    rng = np.random.default_rng(M + 7 * N + 31 * K)
    for n, (fa, fb, out, alpha, beta, act) in enumerate([
            ("e4m3", "e4m3", "bf16", 1.0, 0.0, 0), ("e5m2", "e4m3", "f32", 0.5, -1.5, 0), ("e4m3", "e5m2", "f16", 2.0 ** -8, 0.0, 4),
            ("e4m3", "e4m3", "f32", 2.0 ** -6, 0.0, 1 + M % 3), ("e5m2", "e5m2", "bf16", 2.0 ** -6, 0.75, 2)]):
        if kernel == "sliced":
            monkeypatch.setenv("GEMM_SCALED_SLICES", str((1, 2, 3, 5, 8)[n]))
        A, SA, a = operand(rng, M, K, fa)
        B, SB, b = operand(rng, N, K, fb)
        buf, D = rows_of(M, N, out, fill=0x7F)
        c = None
        if beta:
            c = rng.standard_normal((M, N))
            D.copy_(torch.from_numpy(c))
            c = D.double().cpu().numpy()
        st = plan.run_scaled(A, SA, B, SB, D, alpha=alpha, beta=beta, act=act, slope=0.25)
        assert st == 0
        want, off = expect(a, b, alpha, beta, c, act, 0.25)
        near(D, want, off, out)
        assert (buf.view(torch.uint8).view(M, -1)[:, N * buf.element_size():] == 0x7F).all()  # nothing past a row's end
        path = plan.last_config()["path"]
        assert kernel is None or path == ("scaled_sliced" if kernel == "sliced" else "scaled")
    assert plan.poll_error() == 0


@pytest.mark.parametrize("by,off", [(8, 0), (8, 8), (4, 4), (1, 3)])
def test_operands_at_any_address(plan, by, off):
    """Code matrices whose rows the TMA cannot address are copied first."""
    import torch
    rng = np.random.default_rng(by + off)
    M, N, K, E = 70, 140, 328 + by, 3
    A, SA, a = operand(rng, M, K, "e4m3", spread=1)
    Bs = [operand(rng, N, K, "e4m3", spread=1) for _ in range(E)]

    def moved(t):
        flat = torch.full((t.numel() + off,), 0x7F, dtype=torch.uint8, device="cuda")[off:]
        flat.copy_(t.reshape(-1))
        return flat.view(t.shape).view(torch.float8_e4m3fn)

    A2 = moved(A.view(torch.uint8).contiguous())
    B2 = moved(torch.stack([b.view(torch.uint8) for b, _, _ in Bs]))
    _, D = rows_of(M, N, "f32")
    assert plan.run_scaled(A2, SA, B2[1], Bs[1][1], D) == 0
    near(D, *expect(a, Bs[1][2]), "f32")
    rows = 128 * E
    A3, SA3, a3 = operand(rng, rows, K, "e4m3", spread=1)
    starts, counts = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 128, 256], [5, 0, 100]))
    _, D = rows_of(rows, N, "f32", fill=0)
    assert plan.run_grouped(moved(A3.view(torch.uint8).contiguous()), SA3, B2, torch.stack([s for _, s, _ in Bs]), D, starts, counts) == 0
    for s, n, e in ((0, 5, 0), (256, 100, 2)):
        near(D[s:s + n], *expect(a3[s:s + n], Bs[e][2]), "f32")
    assert plan.poll_error() == 0


@pytest.mark.parametrize("K", [328, 41, 12, 8, 345])
@pytest.mark.parametrize("ld,off", [(8, 0), (8, 8), (4, 4), (1, 0), (1, 3)])
def test_copied_codes(plan, K, ld, off):
    """Rows `ld` bytes past a multiple of 16 apart, from an address `off` bytes past one: copied first, by words as wide as both
    allow, the last word of a row in part; and the call says so."""
    import torch
    rng = np.random.default_rng(K + ld + off)
    M, N, E = 50, 70, 3
    A, SA, a = operand(rng, M, K, "e5m2", spread=1)
    Bs = [operand(rng, N, K, "e4m3", spread=1) for _ in range(E)]
    pitch = -(-K // 16) * 16 + ld

    def moved(t, *lead):
        flat = torch.full((t.numel() // K * pitch + off,), 0x7F, dtype=torch.uint8, device="cuda")[off:]
        view = flat.view(*lead, pitch)[..., :K]
        view.copy_(t)
        assert view.data_ptr() % 16 == off
        return view.view(torch.float8_e4m3fn if t.dim() == 3 else torch.float8_e5m2)

    A2 = moved(A.view(torch.uint8), M)
    B2 = moved(torch.stack([b.view(torch.uint8) for b, _, _ in Bs]), E, N)
    _, D = rows_of(M, N, "f32", fill=0x7F)
    assert plan.run_scaled(A2, SA, B2[2], Bs[2][1], D) == 0
    info = plan.last_config()
    assert info["launches"] == 3 and info["workspace_bytes"] == (M + N) * -(-K // 16) * 16
    near(D, *expect(a, Bs[2][2]), "f32")
    rows = 128 * E
    A3, SA3, a3 = operand(rng, rows, K, "e4m3", spread=1)
    starts, counts = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 128, 256], [5, 0, 100]))
    _, D = rows_of(rows, N, "f32", fill=0)
    assert plan.run_grouped(A3, SA3, B2, torch.stack([s for _, s, _ in Bs]), D, starts, counts) == 0
    assert plan.last_config()["launches"] == 2
    for s, n, e in ((0, 5, 0), (256, 100, 2)):
        near(D[s:s + n], *expect(a3[s:s + n], Bs[e][2]), "f32")
    assert plan.poll_error() == 0


def test_product_many_tiles_and_units(plan, monkeypatch):
    """Every kernel over several tiles a CTA (accumulators and scale columns reused), the slices' rows shared out."""
    import torch
    rng = np.random.default_rng(3)
    M, N, K = 1111, 5000, 1400
    A, SA, a = operand(rng, M, K, "e4m3", spread=1)
    B, SB, b = operand(rng, N, K, "e4m3", spread=1)
    want, off = expect(a, b)
    for kernel, slices in (("tile", 0), ("pair", 0), ("sliced", 1), ("sliced", 4)):
        monkeypatch.setenv("GEMM_SCALED_KERNEL", kernel)
        monkeypatch.setenv("GEMM_SCALED_SLICES", str(slices))
        _, D = rows_of(M, N, "f32", fill=0x7F)
        assert plan.run_scaled(A, SA, B, SB, D) == 0
        near(D, want, off, "f32")
        first = D.clone()
        assert plan.run_scaled(A, SA, B, SB, D) == 0
        assert torch.equal(first, D)  # the same bits every time
    assert plan.poll_error() == 0


def test_nan_stays_in_its_row_and_column(plan, g):
    import torch
    rng = np.random.default_rng(9)
    for M in (40, 300):
        A, SA, a = operand(rng, M, 512, "e4m3")
        B, SB, b = operand(rng, 700, 512, "e4m3")
        A.view(torch.uint8)[7, 300] = 0x7F
        SB[int(ref.scale_offset(130, 2, 512))] = 255
        _, D = rows_of(M, 700, "f32")
        assert plan.run_scaled(A, SA, B, SB, D) == 0
        got = torch.isnan(D).cpu().numpy()
        assert got[7].all() and got[:, 130].all()
        got[7] = got[:, 130] = False
        assert not got.any()
    assert plan.poll_error() == 0


def test_no_k_and_no_rows(plan, g):
    import torch
    D = torch.ones((40, 64), device="cuda")
    call = lambda **c: g.gemm_run_scaled(*{**dict(  # noqa: E731
        plan=plan.handle, M=40, N=64, K=0, A=None, lda=16, SA=None, a_type=4, B=None, ldb=16, SB=None, b_type=4,
        D=D.data_ptr(), ldd=64, d_type=2, alpha=1.0, beta=0.5, act=0, slope=0.0,
        stream=torch.cuda.current_stream().cuda_stream), **c}.values())
    assert call() == 0 and (D == 0.5).all()
    assert call(beta=0.0, M=39) == 0 and (D[:39] == 0).all() and (D[39] == 0.5).all()
    assert call(M=0, D=None) == 0 and plan.last_config()["path"] == "none"
    assert plan.poll_error() == 0


# ------------------------------------------------------------- experts' products

COUNTS = [[5], [0, 1, 0, 33, 128, 0], [129, 300, 2, 0, 64, 96, 127, 128], [0, 0], [1] * 40 + [700]]


def segments(counts):
    starts, at = [], 0
    for n in counts:
        starts.append(at)
        at += -(-n // 128) * 128
    return np.array(starts, np.int32), np.array(counts, np.int32), at


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "e%d" % len(c))
def test_grouped(plan, g, monkeypatch, kernel, counts):
    import torch
    rng = np.random.default_rng(len(counts))
    starts, n, rows = segments(counts)
    rows += 128  # rows in no group, at the end too
    for N, K, out, beta, slices in ((200, 300, "bf16", 0.0, 1), (256, 1024, "f32", 0.5, 3), (120, 130, "f16", 0.0, 8)):
        if kernel:
            monkeypatch.setenv("GEMM_SCALED_KERNEL", kernel)
        if kernel == "sliced":
            monkeypatch.setenv("GEMM_SCALED_SLICES", str(slices))
        A, SA, a = operand(rng, rows, K, "e4m3", spread=2)
        owner = np.full(rows, -1)
        for e, (s, c) in enumerate(zip(starts, n)):
            owner[s:s + c] = e
        none = torch.from_numpy(owner < 0).cuda()
        A.view(torch.uint8)[none] = 0x7F  # what rows between groups hold does not matter
        Bs = [operand(rng, N, K, "e4m3", spread=2) for _ in counts]
        B = torch.stack([v.view(torch.uint8) for v, _, _ in Bs])
        ld = -(-K // 16) * 16
        wide = torch.full((len(counts), N + 3, ld), 0x7F, dtype=torch.uint8, device="cuda")  # groups with a gap between them
        wide[:, :N, :K] = B
        SB = torch.stack([s for _, s, _ in Bs])
        buf, D = rows_of(rows, N, out, fill=0x11)
        c = rng.standard_normal((rows, N))
        live = torch.from_numpy(owner >= 0).cuda()
        D[live] = torch.from_numpy(c).cuda().to(D.dtype)[live]
        before = buf.clone()
        c = D.double().cpu().numpy()
        st = plan.run_grouped(A, SA, wide[:, :N, :K].view(torch.float8_e4m3fn), SB, D, torch.from_numpy(starts).cuda(),
                              torch.from_numpy(n).cuda(), alpha=0.25, beta=beta)
        assert st == 0
        for e, (s, m) in enumerate(zip(starts, n)):
            if m:
                want, off = expect(a[s:s + m], Bs[e][2], 0.25, beta, c[s:s + m])
                near(D[s:s + m], want, off, out)
        assert torch.equal(buf.view(torch.uint8).view(rows, -1)[none], before.view(torch.uint8).view(rows, -1)[none])
        assert torch.equal(buf[:, N:].contiguous().view(torch.uint8), before[:, N:].contiguous().view(torch.uint8))
    assert plan.poll_error() == 0


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("fa,fb", [("e5m2", "e4m3"), ("e5m2", "e5m2"), ("e4m3", "e5m2")])
def test_grouped_types(plan, monkeypatch, kernel, fa, fb):
    """The input gradient of experts: 8-bit gradients (e5m2) times transposed weights, in every kernel, with an activation or beta."""
    import torch
    if kernel:
        monkeypatch.setenv("GEMM_SCALED_KERNEL", kernel)
    rng = np.random.default_rng(16)
    starts, n, rows = segments([33, 0, 130, 64, 300])
    for N, K, out, beta, act in ((264, 520, "bf16", 0.0, 0), (136, 384, "f32", 0.5, 0), (200, 200, "bf16", 0.0, 4), (96, 130, "f16", 0.0, 3)):
        A, SA, a = operand(rng, rows, K, fa, spread=2)
        Bs = [operand(rng, N, K, fb, spread=2) for _ in n]
        B = torch.stack([v.view(torch.uint8) for v, _, _ in Bs]).view(dtype(fb))
        buf, D = rows_of(rows, N, out, fill=0x11)
        c = rng.standard_normal((rows, N))
        if beta:
            D.copy_(torch.from_numpy(c))
        before = buf.clone()
        c = D.double().cpu().numpy()
        assert plan.run_grouped(A, SA, B, torch.stack([s for _, s, _ in Bs]), D, torch.from_numpy(starts).cuda(), torch.from_numpy(n).cuda(),
                                alpha=2.0 ** -6, beta=beta, act=act) == 0
        none = np.ones(rows, bool)
        for e, (s, m) in enumerate(zip(starts, n)):
            none[s:s + m] = False
            if m:
                want, off = expect(a[s:s + m], Bs[e][2], 2.0 ** -6, beta, c[s:s + m], act)
                near(D[s:s + m], want, off, out)
        none = torch.from_numpy(none).cuda()
        assert torch.equal(buf.view(torch.uint8).view(rows, -1)[none], before.view(torch.uint8).view(rows, -1)[none])
    assert plan.poll_error() == 0


def test_grouped_takes_no_row_outside(plan, g):
    """Starts that are no multiple of 128 or outside, counts that are negative or reach past the end."""
    import torch
    rng = np.random.default_rng(2)
    rows, N, K = 512, 160, 256
    A, SA, a = operand(rng, rows, K, "e4m3", spread=1)
    Bs = [operand(rng, N, K, "e4m3", spread=1) for _ in range(6)]
    B = torch.stack([v.view(torch.uint8) for v, _, _ in Bs]).view(torch.float8_e4m3fn)
    SB = torch.stack([s for _, s, _ in Bs])
    starts = torch.tensor([64, -128, 512, 0, 128, 384], dtype=torch.int32, device="cuda")
    counts = torch.tensor([10, 10, 10, -5, 100, 1000], dtype=torch.int32, device="cuda")
    for _ in range(2):
        _, D = rows_of(rows, N, "f32", fill=0x11)
        before = D.clone()
        assert plan.run_grouped(A, SA, B, SB, D, starts, counts) == 0
        near(D[128:228], *expect(a[128:228], Bs[4][2]), "f32")
        near(D[384:], *expect(a[384:], Bs[5][2]), "f32")
        assert torch.equal(D[:128], before[:128]) and torch.equal(D[228:384], before[228:384])
    assert plan.poll_error() == 0


@pytest.mark.parametrize("kernel", KERNELS)
def test_groups_that_share_rows(plan, monkeypatch, kernel):
    """Segments over one another: as many tiles in all as they add up to, every one inside the matrices (the groups have
    equal B, so that it does not matter whose result stays)."""
    import torch
    if kernel:
        monkeypatch.setenv("GEMM_SCALED_KERNEL", kernel)
    rng = np.random.default_rng(14)
    rows, N, K, E = 400, 260, 200, 70
    A, SA, a = operand(rng, rows, K, "e4m3", spread=1)
    B, SB, b = operand(rng, N, K, "e4m3", spread=1)
    B = torch.stack([B.view(torch.uint8)] * E).view(torch.float8_e4m3fn)
    starts = torch.zeros(E, dtype=torch.int32, device="cuda")
    counts = torch.full((E,), rows, dtype=torch.int32, device="cuda")
    starts[1::3], counts[2::5] = 128, 0
    _, D = rows_of(rows, N, "f32", fill=0x7F)
    assert plan.run_grouped(A, SA, B, torch.cat([SB] * E), D, starts, counts) == 0
    near(D, *expect(a, b), "f32")
    assert plan.poll_error() == 0


@pytest.mark.parametrize("kernel", [None, "tile", "pair"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "e%d" % len(c))
def test_grouped_k(plan, g, monkeypatch, kernel, counts):
    import torch
    if kernel:
        monkeypatch.setenv("GEMM_SCALED_KERNEL", kernel)
    rng = np.random.default_rng(len(counts) + 50)
    starts, n, rows = segments(counts)
    rows = max(rows, 128) + 128
    owner = np.full(rows, -1)
    for e, (s, c) in enumerate(zip(starts, n)):
        owner[s:s + c] = e
    none = torch.from_numpy(owner < 0).cuda()
    for M, N, out, beta in ((100, 200, "f32", 0.0), (256, 136, "bf16", 0.5)):
        A, SA, a = operand(rng, M, rows, "e5m2", spread=2)
        B, SB, b = operand(rng, N, rows, "e4m3", spread=2)
        A.view(torch.uint8)[:, none] = 0
        B.view(torch.uint8)[:, none] = 0
        a[:, owner < 0] = b[:, owner < 0] = 0
        D = torch.full((len(counts), M + 1, N + 8), 7.0, device="cuda", dtype=dtype(out))
        view = D[:, :M, :N]
        c = rng.standard_normal((len(counts), M, N))
        view.copy_(torch.from_numpy(c))
        c = view.double().cpu().numpy()
        assert plan.run_grouped_k(A, SA, B, SB, view, torch.from_numpy(starts).cuda(), torch.from_numpy(n).cuda(), beta=beta) == 0
        for e in range(len(counts)):
            want, off = expect(a[:, owner == e], b[:, owner == e], 1.0, beta, c[e])
            near(view[e], want, off, out)
        assert (D[:, M:] == 7).all() and (D[:, :, N:] == 7).all()
    assert plan.poll_error() == 0


def test_results_between_the_groups(plan, g):
    """What lies between the matrices of a stack is not theirs: D in the gap between two B, A between two D."""
    import torch
    rng = np.random.default_rng(15)
    rows, N, K = 128, 32, 64
    A, SA, a = operand(rng, rows, K, "e4m3", spread=1)
    (B0, SB0, b0), (B1, SB1, b1) = (operand(rng, N, K, "e4m3", spread=1) for _ in range(2))
    d_bytes, b_bytes = rows * N * 4, N * K
    buf = torch.zeros(2 * b_bytes + d_bytes, dtype=torch.uint8, device="cuda")
    buf[:b_bytes], buf[b_bytes + d_bytes:] = B0.view(torch.uint8).reshape(-1), B1.view(torch.uint8).reshape(-1)
    D = buf[b_bytes:b_bytes + d_bytes].view(torch.float32).view(rows, N)
    SB = torch.cat([SB0, SB1])
    starts, counts = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    call = lambda **c: g.gemm_run_grouped(*{**dict(  # noqa: E731
        plan=plan.handle, groups=2, rows=rows, N=N, K=K, starts=starts.data_ptr(), counts=counts.data_ptr(), A=A.data_ptr(), lda=A.stride(0),
        SA=SA.data_ptr(), a_type=4, B=buf.data_ptr(), ldb=K, b_group=b_bytes + d_bytes, SB=SB.data_ptr(), b_type=4, D=D.data_ptr(), ldd=N,
        d_type=2, alpha=1.0, beta=0.0, act=0, slope=0.0, stream=torch.cuda.current_stream().cuda_stream), **c}.values())
    assert call() == g.GEMM_OK
    near(D[:100], *expect(a[:100], b1), "f32")
    assert (D[100:] == 0).all()
    assert call(D=D.data_ptr() - 16) == call(D=D.data_ptr() + 16) == g.GEMM_ERR_INVALID_ARG
    # columns of A and B times each other into two D with A's codes between them
    QA, SQ, qa = operand(rng, N, rows, "e4m3", spread=1)
    QA.view(torch.uint8)[:, 100:] = 0
    qa[:, 100:] = 0
    one = N * N * 4
    buf = torch.zeros(2 * one + N * rows, dtype=torch.uint8, device="cuda")
    buf[one:one + N * rows] = QA.view(torch.uint8).reshape(-1)
    call = lambda **c: g.gemm_run_grouped_k(*{**dict(  # noqa: E731
        plan=plan.handle, groups=2, M=N, N=N, rows=rows, starts=starts.data_ptr(), counts=counts.data_ptr(), A=buf.data_ptr() + one, lda=rows,
        SA=SQ.data_ptr(), a_type=4, B=QA.data_ptr(), ldb=QA.stride(0), SB=SQ.data_ptr(), b_type=4, D=buf.data_ptr(), ldd=N,
        d_group=(one + N * rows) // 4, d_type=2, alpha=1.0, beta=0.0, act=0, slope=0.0, stream=torch.cuda.current_stream().cuda_stream), **c}.values())
    assert call() == g.GEMM_OK
    near(buf[one + N * rows:].view(torch.float32).view(N, N), *expect(qa, qa), "f32")
    assert (buf[:one] == 0).all()  # an empty group
    assert call(A=buf.data_ptr() + one - 16) == call(A=buf.data_ptr() + one + 16) == g.GEMM_ERR_INVALID_ARG
    assert plan.poll_error() == 0


def test_grouped_refusals(plan, g):
    import torch
    A = torch.zeros((256, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    B = torch.zeros((2, 32, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.zeros(4096, dtype=torch.uint8, device="cuda")  # longer than it has to be, like D: moved ones stay apart
    D = torch.zeros((300, 32), device="cuda")
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    call = lambda **c: g.gemm_run_grouped(*{**dict(  # noqa: E731
        plan=plan.handle, groups=2, rows=256, N=32, K=64, starts=i.data_ptr(), counts=i.data_ptr(), A=A.data_ptr(), lda=64,
        SA=s.data_ptr(), a_type=4, B=B.data_ptr(), ldb=64, b_group=2048, SB=s.data_ptr(), b_type=4, D=D.data_ptr(), ldd=32,
        d_type=2, alpha=1.0, beta=0.0), **c}.values())
    assert call() == g.GEMM_OK and call(groups=0) == g.GEMM_OK and call(rows=0) == g.GEMM_OK
    for bad in ({"groups": -1}, {"starts": None}, {"counts": None}, {"b_group": 2032}, {"D": None}, {"A": None}, {"lda": 48},
                {"D": B.data_ptr() + 2048}):
        assert call(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    for bad in ({"SA": s.data_ptr() + 4}, {"D": D.data_ptr() + 4}, {"starts": i.data_ptr() + 2}):
        assert call(**bad) == g.GEMM_ERR_ALIGNMENT, bad
    assert call(groups=1025) == g.GEMM_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        plan.run_grouped(A, s, B, s, D[:256], i.long(), i)


# ------------------------------------------------ gradients, streams, graphs

def test_gradient_products(plan, g):
    """Forward, input and weight gradients of Y = X W^T on values that 8 bits hold exactly: against the
    formulas, and against central differences of <Y, dY>, which are exact for a linear map."""
    import torch
    rng = np.random.default_rng(4)
    T, I, O = 150, 200, 136
    # small integers: exact codes whatever the block's scale
    x, w, dy = (rng.integers(-8, 9, s).astype(np.float64) for s in ((T, I), (O, I), (T, O)))

    def both(m, fmt="e4m3", block=1):
        t = torch.from_numpy(m).to("cuda", torch.bfloat16)
        R, K = t.shape
        _, q = rows_of(R, K, fmt)
        _, qt = rows_of(K, R, fmt)
        s = torch.empty(g.gemm_scale_bytes(R, K), dtype=torch.uint8, device="cuda")
        st = torch.empty(g.gemm_scale_bytes(K, R), dtype=torch.uint8, device="cuda")
        buf, td = rows_of(R, K, "bf16")
        td.copy_(t)
        assert plan.quantize(td, q, s, qt, st, block_rows=block) == 0
        return (q, s), (qt, st)

    def product(a, b):
        _, D = rows_of(a[0].shape[0], b[0].shape[0], "f32")
        assert plan.run_scaled(*a, *b, D) == 0
        return D.double().cpu().numpy()

    (X, XT), (W, WT), (DY, DYT) = both(x), both(w, block=128), both(dy)
    y, dx, dw = product(X, W), product(DY, WT), product(DYT, XT)
    assert np.array_equal(y, x @ w.T) and np.array_equal(dx, dy @ w) and np.array_equal(dw, dy.T @ x)
    for _ in range(3):
        d = rng.integers(-1, 2, x.shape)
        lo, hi = ((product(both(x + s * d)[0], W) * dy).sum() for s in (-1, 1))
        assert (hi - lo) / 2 == (dx * d).sum()
        d = rng.integers(-1, 2, w.shape)
        lo, hi = ((product(X, both(w + s * d, block=128)[0]) * dy).sum() for s in (-1, 1))
        assert (hi - lo) / 2 == (dw * d).sum()


def test_on_a_stream_and_in_a_graph(plan, g):
    """Counts that change between replays of a captured graph."""
    import torch
    rng = np.random.default_rng(8)
    rows, N, K, E = 768, 192, 384, 3
    A, SA, a = operand(rng, rows, K, "e4m3", spread=1)
    Bs = [operand(rng, N, K, "e4m3", spread=1) for _ in range(E)]
    B = torch.stack([v.view(torch.uint8) for v, _, _ in Bs]).view(torch.float8_e4m3fn)
    SB = torch.stack([s for _, s, _ in Bs])
    starts = torch.tensor([0, 256, 512], dtype=torch.int32, device="cuda")
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    _, D = rows_of(rows, N, "f32")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        assert plan.run_grouped(A, SA, B, SB, D, starts, counts) == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            assert plan.run_grouped(A, SA, B, SB, D, starts, counts) == 0
    for new in ([0, 3, 0], [256, 1, 200]):
        torch.cuda.synchronize()
        D.zero_()
        counts.copy_(torch.tensor(new))
        graph.replay()
        torch.cuda.synchronize()
        for e, n in enumerate(new):
            if n:
                near(D[256 * e:256 * e + n], *expect(a[256 * e:256 * e + n], Bs[e][2]), "f32")
            assert (D[256 * e + n:256 * e + 256] == 0).all()
    assert plan.poll_error() == 0
