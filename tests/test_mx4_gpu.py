"""The 4-bit quantiser, the values of block-scaled matrices and the 4-bit products on the GPU against 64-bit numpy
(tests/more_ref.py).

Quantiser: codes' values and scale bytes are exact and have to be equal.  Values of codes are exact in bf16 and fp32.

Products, tolerance: the tensor core multiplies the values exactly and adds the 64 products of an MMA into an fp32
accumulator, K/64 times.  With S = sum |a b| (an upper bound of every partial sum), each of the K/64 additions, and the sum inside an
MMA, is off by at most two units of 2^-23 S: (K/64 + 1) * 2^-22 * S, to which the K slices of a cluster add eight more additions.
alpha, beta and the activation (slope at most 1.13, expf and erfcf to 2^-20) scale that and add 2^-20 of the result; the result's
rounding adds half a unit: 2^-24, 2^-11 (f16) or 2^-8 (bf16) of its size, and f16's least step.
"""
import numpy as np
import pytest

from tests import more_ref as ref
from tests import scaled_ref

pytestmark = pytest.mark.gpu

ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
KERNELS = [None, "tile", "pair", "sliced"]


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


def byte_rows(n, width, fill, extra=0):
    """n rows of `width` bytes, whole multiples of 16 (and `extra` bytes) apart, in a buffer of `fill`."""
    import torch
    ld = -(-max(width, 1) // 16) * 16 + extra
    buf = torch.full((n, ld), fill, dtype=torch.uint8, device="cuda")
    return buf, buf[:, :width]


def float_rows(n, width, name, extra=0, fill=float("nan")):
    import torch
    per = 16 // torch.empty((), dtype=dtype(name)).element_size()
    ld = -(-max(width, 1) // per) * per + extra
    buf = torch.full((n, ld), fill, dtype=dtype(name), device="cuda")
    return buf, buf[:, :width]


def scale_room(g, rows, cols, fill=0xEE):
    import torch
    return torch.full((g.gemm_mx_scale_bytes(rows, cols),), fill, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ quantiser

def values(rng, R, K, name, wild=True):
    import torch
    x = rng.standard_normal((R, K)) * 10.0 ** rng.integers(-4, 4, (R, 1))
    x[:, ::7] *= 30
    x.reshape(-1)[::41] = 6.0  # the rounding's edges: the largest code, ties, just past it
    if R > 5:
        x[5, : K // 2] = np.resize([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.0, -0.2, 6.001, 0.2501], K // 2)
    if R > 2:
        x[2] = 0
    if K > 40:
        x[R // 2, 32:64] = 1e-30 if name != "f16" else 6e-8  # a block of the smallest values
    if wild and R > 6 and K > 3:
        x[6, 1], x[6, K - 1] = np.inf, np.nan
    return torch.from_numpy(x).to(dtype(name))


def same(got, want):
    """The same codes' values, the sign of a zero apart."""
    assert np.array_equal(got, want), np.argwhere(got != want)[:4].tolist()


SHAPES = [(1, 1), (1, 32), (7, 31), (33, 2050), (127, 129), (128, 512), (129, 640), (300, 517)]


@pytest.mark.parametrize("R,K", SHAPES)
@pytest.mark.parametrize("name", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("odd", [0, 1, 2])
def test_quantize(plan, g, R, K, name, odd):
    import torch
    rng = np.random.default_rng(R * 1000 + K)
    x = values(rng, R, K, name)
    _, xd = float_rows(R, K, name, extra=odd)  # rows 1 value further apart: no wide loads; 2: words
    xd.copy_(x)
    x64 = x.double().numpy()
    want, byte = ref.quantize4(x64)
    want_t, byte_t = ref.quantize4(x64.T)
    for both in (0, 1, 2):  # as it stands, both, transposed
        qbuf, q = byte_rows(R, -(-K // 2), 0xA5)
        tbuf, qt = byte_rows(K, -(-R // 2), 0xA5)
        sq, sqt = scale_room(g, R, K), scale_room(g, K, R)
        assert plan.quantize_mx4(xd, *((q, sq) if both < 2 else (None, None)), *((qt, sqt) if both else (None, None))) == g.GEMM_OK
        if both < 2:
            same(ref.decode4(q.cpu().numpy(), K), want)
            assert np.array_equal(sq.cpu().numpy(), ref.pack_scales4(byte, K))
            assert (qbuf[:, -(-K // 2):] == 0xA5).all() and (K % 2 == 0 or (q[:, -1] >> 4 == 0).all())
        if both:
            same(ref.decode4(qt.cpu().numpy(), R), want_t)
            assert np.array_equal(sqt.cpu().numpy(), ref.pack_scales4(byte_t, R))
            assert (tbuf[:, -(-R // 2):] == 0xA5).all() and (R % 2 == 0 or (qt[:, -1] >> 4 == 0).all())
    assert plan.poll_error() == g.GEMM_OK


def test_quantize_every_exponent(plan, g):
    """Blocks whose largest magnitude has every exponent and the fractions round 1.5, subnormals too."""
    import torch
    bits = [(e << 23) | f for e in range(255) for f in (0, 1, 0x3FFFFF, 0x400000, 0x400001, 0x7FFFFF)]
    x = torch.zeros((len(bits), 32))
    x[:, 5] = torch.tensor(bits, dtype=torch.int32).view(torch.float32)
    x[:, 9] = -x[:, 5] / 3
    want, byte = ref.quantize4(x.double().numpy())
    _, q = byte_rows(len(bits), 16, 0)
    sq = scale_room(g, len(bits), 32)
    assert plan.quantize_mx4(x.cuda(), q, sq) == g.GEMM_OK
    assert np.array_equal(sq.cpu().numpy(), ref.pack_scales4(byte, 32))
    same(ref.decode4(q.cpu().numpy(), 32), want)


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_quantize_through_a_row_map(plan, g, name):
    import torch
    rng = np.random.default_rng(5)
    T, K, k, rows = 40, 200, 3, 260
    x = values(rng, T, K, name, wild=False)
    rowmap = np.full(rows, -1)
    at = rng.permutation(rows)[:100]
    rowmap[at] = rng.integers(0, T * k, 100)
    rowmap[at[:3]] = [-5, T * k, T * k - 1]  # none, past X, the last
    src = np.where((rowmap >= 0) & (rowmap // k < T), rowmap // k, -1)
    gathered = np.where(src[:, None] >= 0, x.double().numpy()[np.maximum(src, 0)], 0.0)
    want, byte = ref.quantize4(gathered)
    want_t, byte_t = ref.quantize4(gathered.T)
    qbuf, q = byte_rows(rows, K // 2, 0xA5)
    _, qt = byte_rows(K, rows // 2, 0xA5)
    sq, sqt = scale_room(g, rows, K), scale_room(g, K, rows)
    assert plan.quantize_mx4(x.cuda(), q, sq, qt, sqt, rowmap=torch.from_numpy(rowmap.astype(np.int32)).cuda(), map_div=k) == g.GEMM_OK
    got = ref.decode4(q.cpu().numpy(), K)
    same(got[src >= 0], want[src >= 0])
    assert (q.cpu().numpy()[src < 0] == 0xA5).all()  # a row without a source is left as it is
    assert np.array_equal(sq.cpu().numpy(), ref.pack_scales4(byte, K))
    same(ref.decode4(qt.cpu().numpy(), rows), want_t)
    assert np.array_equal(sqt.cpu().numpy(), ref.pack_scales4(byte_t, rows))


@pytest.mark.parametrize("R,K,gathered", [(2500, 2699, False), (2688, 2688, False), (2500, 2704, True), (130, 40100, False)])
@pytest.mark.parametrize("name", ["bf16", "f16", "f32"])
def test_quantize_more_tiles_than_ctas(plan, g, R, K, gathered, name):
    """Both orientations of more 128 x 128 tiles than CTAs run at once; a part of the rows and columns against 64 bits."""
    import torch
    rng = np.random.default_rng(R + K)
    x = torch.from_numpy(rng.standard_normal((R, K)) * 10.0 ** rng.integers(-3, 3, (R, 1))).to(dtype(name))
    _, xd = float_rows(R, K, name)
    xd.copy_(x)
    rowmap, source = None, np.arange(R)
    if gathered:
        source = np.where(rng.random(R) < 0.1, -1, rng.integers(0, R, R))
        rowmap = torch.from_numpy(source.astype(np.int32)).cuda()
    x64 = np.where(source[:, None] >= 0, x.double().numpy()[np.maximum(source, 0)], 0.0)
    _, q = byte_rows(R, -(-K // 2), 0xA5)
    _, qt = byte_rows(K, -(-R // 2), 0xA5)
    sq, sqt, one, tone = scale_room(g, R, K), scale_room(g, K, R), scale_room(g, R, K), scale_room(g, K, R)
    for _ in range(2):
        assert plan.quantize_mx4(xd, q, sq, qt, sqt, rowmap=rowmap) == g.GEMM_OK
    assert plan.quantize_mx4(xd, None, None, qt[:, :], tone, rowmap=rowmap) == g.GEMM_OK and torch.equal(tone, sqt)
    _, q1 = byte_rows(R, -(-K // 2), 0xA5)
    assert plan.quantize_mx4(xd, q1, one, rowmap=rowmap) == g.GEMM_OK
    assert torch.equal(one, sq) and torch.equal(q1, q)  # the rows' kernel says the same
    rows = np.unique(np.concatenate([rng.integers(0, R, 12), [0, R - 1]]))
    cols = np.unique(np.concatenate([rng.integers(0, K, 25), [0, K - 1]]))
    want, byte = ref.quantize4(x64[rows])
    live = source[rows] >= 0
    same(ref.decode4(q.cpu().numpy()[rows], K)[live], want[live])
    want_t, byte_t = ref.quantize4(x64.T[cols])
    same(ref.decode4(qt.cpu().numpy()[cols], R), want_t)
    for packed, at, want_b, width in ((sq, rows, byte, K), (sqt, cols, byte_t, R)):
        tiles, nb = -(-width // 128), np.arange(want_b.shape[1])
        where = ((at[:, None] // 128) * tiles + nb // 4) * 512 + at[:, None] % 32 * 16 + at[:, None] % 128 // 32 * 4 + nb % 4
        assert np.array_equal(packed.cpu().numpy()[where], want_b)


def test_sizes_past_the_indices(plan, g):
    import torch
    x = torch.zeros(64, device="cuda", dtype=torch.bfloat16)
    n, p = 2 ** 31 - 1, x.data_ptr()
    # (refused by its size before anything is read)
    assert g.gemm_quantize_mx(plan.handle, 1, n, p, n, 0, None, 1, 1, p + 32, n, p + 64, None, 0, None) == g.GEMM_ERR_UNSUPPORTED
    assert g.gemm_dequantize(plan.handle, 1, n, p, n, 6, p + 64, p + 32, n, 0) == g.GEMM_ERR_UNSUPPORTED
    assert g.gemm_dequantize(plan.handle, n, 1, p, n, 6, p + 64, p + 32, n, 0) == g.GEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("R,K", [(1, 1), (3, 33), (130, 515), (64, 1024)])
@pytest.mark.parametrize("out", ["bf16", "f32", "f16"])
def test_dequantize(plan, g, R, K, out):
    import torch
    rng = np.random.default_rng(R + K)
    for fmt, block in (("e2m1", 32), ("e4m3", 128), ("e5m2", 128)):
        byte = rng.integers(120, 134, (R, -(-K // block)))
        byte[0, 0] = 255  # a block of NaN
        if fmt == "e2m1":
            packed = ref.pack4(rng.integers(0, 16, (R, K)))
            _, q = byte_rows(R, -(-K // 2), 0xFF)
            q.copy_(torch.from_numpy(packed))
            want, s = ref.scaled4(ref.decode4(packed, K), byte), ref.pack_scales4(byte, K)
        else:
            code = rng.integers(0, 256, (R, K)).astype(np.uint8)
            _, q = byte_rows(R, K, 0)
            q.copy_(torch.from_numpy(code))
            q = q.view({"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt])
            value = scaled_ref.decode(code, fmt)
            by = np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))
            want, s = value * np.repeat(by, 128, axis=1)[:, :K], scaled_ref.pack(byte, K)
        for extra in (0, 1):
            buf, x = float_rows(R, K, out, extra=extra, fill=-3.0)
            assert plan.dequantize(q, torch.from_numpy(s).cuda(), x) == g.GEMM_OK
            expected = torch.from_numpy(want).to(dtype(out)).double().numpy()  # (exact but for f16's largest and least)
            assert np.array_equal(x.double().cpu().numpy(), expected, equal_nan=True)
            assert (buf[:, K:] == -3.0).all()


@pytest.mark.parametrize("off,ld_extra", [(0, 1), (4, 4), (1, 0), (3, 2), (8, 8)])
@pytest.mark.parametrize("R,K", [(40, 533), (130, 256)])
def test_quantize_to_any_address(plan, g, off, ld_extra, R, K):
    import torch
    x = torch.randn((R, K), device="cuda", dtype=torch.bfloat16)
    want, byte = ref.quantize4(x.double().cpu().numpy())
    want_t, byte_t = ref.quantize4(x.double().cpu().numpy().T)

    def room(rows, cols):
        width = (cols + 1) // 2
        buf = torch.full((rows * (width + ld_extra) + off,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, torch.as_strided(buf, (rows, width), (width + ld_extra, 1), off)

    for both in (False, True):
        buf, q = room(R, K)
        tbuf, qt = room(K, R)
        s, st = scale_room(g, R, K), scale_room(g, K, R)
        assert plan.quantize_mx4(x, q, s, *((qt, st) if both else (None, None))) == g.GEMM_OK
        same(ref.decode4(q.cpu().numpy(), K), want)
        assert np.array_equal(s.cpu().numpy(), ref.pack_scales4(byte, K))
        assert int((buf == 0xA5).sum()) >= R * ld_extra + off - ld_extra  # nothing between the rows is written
        if both:
            same(ref.decode4(qt.cpu().numpy(), R), want_t)
            assert np.array_equal(st.cpu().numpy(), ref.pack_scales4(byte_t, R))
        else:
            assert (tbuf == 0xA5).all()


@pytest.mark.parametrize("off,ld_extra", [(0, 1), (4, 4), (1, 0), (3, 2)])
def test_dequantize_at_any_address(plan, g, off, ld_extra):
    import torch
    rng = np.random.default_rng(off)
    R, K = 40, 533
    view, s, want = operand(rng, R, K, ld_extra=ld_extra, offset=off)
    x = torch.empty((R, K), device="cuda")
    assert plan.dequantize(view, s, x) == g.GEMM_OK
    assert np.array_equal(x.double().cpu().numpy(), want)
    code = rng.integers(0, 0x7F, (R, K)).astype(np.uint8)
    buf = torch.zeros(R * (K + ld_extra) + off, dtype=torch.uint8, device="cuda")
    q = torch.as_strided(buf, (R, K), (K + ld_extra, 1), off)
    q.copy_(torch.from_numpy(code))
    byte = rng.integers(120, 134, (R, -(-K // 128)))
    assert plan.dequantize(q.view(torch.float8_e4m3fn), torch.from_numpy(scaled_ref.pack(byte, K)).cuda(), x) == g.GEMM_OK
    assert np.array_equal(x.double().cpu().numpy(), scaled_ref.scaled(scaled_ref.decode(code, "e4m3"), byte))


def test_there_and_back(plan, g):
    """What a quantised matrix stands for quantises to itself."""
    import torch
    x = torch.randn((200, 300), device="cuda", dtype=torch.bfloat16)
    _, q = byte_rows(200, 150, 0)
    _, q2 = byte_rows(200, 150, 0)
    s, s2, v = scale_room(g, 200, 300), scale_room(g, 200, 300), torch.empty((200, 300), device="cuda", dtype=torch.bfloat16)
    assert plan.quantize_mx4(x, q, s) == g.GEMM_OK and plan.dequantize(q, s, v) == g.GEMM_OK
    assert ((v - x).abs() <= x.abs().float().view(200, -1).amax(1, keepdim=True) / 4).all()
    assert plan.quantize_mx4(v, q2, s2) == g.GEMM_OK
    v2 = torch.empty_like(v)
    assert plan.dequantize(q2, s2, v2) == g.GEMM_OK
    assert torch.equal(v, v2)


# ------------------------------------------------------------------- products

def operand(rng, rows, K, spread=4, ld_extra=0, offset=0):
    """Random codes (device view), packed scales, element values in 64 bits."""
    import torch
    code = rng.integers(0, 16, (rows, K))
    packed = ref.pack4(code)
    byte = rng.integers(127 - spread, 127 + spread, (rows, -(-K // 32)))
    width = packed.shape[1]
    ld = -(-width // 16) * 16 + ld_extra
    buf = torch.full((rows * ld + offset,), 0x77, dtype=torch.uint8, device="cuda")  # sixes beyond the rows' ends: not to be read as operands
    view = torch.as_strided(buf, (rows, width), (ld, 1), offset)
    view.copy_(torch.from_numpy(packed))
    return view, torch.from_numpy(ref.pack_scales4(byte, K)).cuda(), ref.scaled4(ref.decode4(packed, K), byte)


def expect(a, b, alpha=1.0, beta=0.0, c=None, act=0, slope=0.0):
    y = alpha * (a @ b.T)
    off = abs(alpha) * (np.abs(a) @ np.abs(b).T) * (a.shape[1] / 64 + 9) * 2.0 ** -22
    if beta:
        y = y + beta * c
        off = off + np.abs(beta * c) * 2.0 ** -22
    return scaled_ref.act(y, act, slope), off * 1.13


def near(got, want, off, out):
    got = got.double().cpu().numpy()
    tol = off + np.abs(want) * (2.0 ** -20 + ROUND[out]) + (2.0 ** -24 if out == "f16" else 1e-37)
    if out == "f16":  # past f16's largest value the result rounds to infinity
        got, want = (np.where(np.abs(v) >= 65520, np.sign(v) * 65520, v) for v in (got, want))
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


PRODUCTS = [(1, 8, 32), (1, 1, 1), (2, 130, 64), (33, 129, 257), (64, 256, 512), (129, 136, 1000), (200, 264, 1031),
            (513, 300, 2304), (130, 4096, 96), (40, 520, 4100)]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(plan, g, monkeypatch, kernel, M, N, K):
    if kernel:
        monkeypatch.setenv("GEMM_SCALED_KERNEL", kernel)
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    A, SA, a = operand(rng, M, K)
    B, SB, b = operand(rng, N, K)
    for out, alpha, beta, act in (("f32", 1.0, 0.0, 0), ("bf16", 0.5, 0.75, 4), ("f16", 0.125, 0.0, 3), ("bf16", 1.0, 0.0, 1)):
        buf, D = float_rows(M, N, out, fill=2.0)
        assert plan.run_mx4(A, SA, B, SB, D, K=K, alpha=alpha, beta=beta, act=act, slope=0.1) == g.GEMM_OK
        want, off = expect(a, b, alpha, beta, np.full((M, N), 2.0), act, 0.1)
        near(D, want, off, out)
        assert (buf[:, N:] == 2.0).all()
    assert plan.poll_error() == g.GEMM_OK
    cfg = plan.last_config()
    assert cfg["path"] == ("scaled_sliced" if kernel == "sliced" else "scaled") or kernel is None
    assert cfg["tile_k"] == 256


@pytest.mark.parametrize("M,N,K", [(300, 1030, 1300), (257, 33, 1537), (1, 257, 2048), (2100, 2090, 1281)])
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_six_stages(plan, g, monkeypatch, M, N, K, out):
    """Pairs into 16 bits with more than four k-blocks: a ring of six stages, boxes of 32 columns."""
    monkeypatch.setenv("GEMM_SCALED_KERNEL", "pair")
    rng = np.random.default_rng(M + N + K)
    A, SA, a = operand(rng, M, K, spread=2)
    B, SB, b = operand(rng, N, K, spread=2)
    a, b = a / 64, b / 64  # (alpha)
    for beta, act in ((0.0, 0), (0.0, 1), (0.0, 3), (0.0, 4), (0.5, 0), (-0.75, 3)):
        buf, D = float_rows(M, N, out, extra=8, fill=2.0)
        assert plan.run_mx4(A, SA, B, SB, D, K=K, alpha=2.0 ** -12, beta=beta, act=act, slope=0.1) == g.GEMM_OK
        assert plan.last_config()["stages"] == 6
        near(D, *expect(a, b, 1.0, beta, np.full((M, N), 2.0), act, 0.1), out)
        assert (buf[:, N:] == 2.0).all()
    _, D = float_rows(M, N, "f32")
    assert plan.run_mx4(A, SA, B, SB, D, K=K) == g.GEMM_OK and plan.last_config()["stages"] == 5
    assert plan.poll_error() == g.GEMM_OK


@pytest.mark.parametrize("E", [64, 65])
def test_groups_of_six_and_five_stages(plan, g, monkeypatch, E):
    import torch
    monkeypatch.setenv("GEMM_SCALED_KERNEL", "pair")
    rng = np.random.default_rng(E)
    N, K = 136, 1300
    counts = [int(c) for c in np.where(rng.random(E) < 0.2, 0, rng.integers(1, 200, E))]
    starts, at = [], 0
    for c in counts:
        starts.append(at)
        at += -(-c // 128) * 128
    A, SA, a = operand(rng, at + 128, K)
    B = [operand(rng, N, K) for _ in range(E)]
    Bq, SB = torch.stack([b[0] for b in B]), torch.cat([b[1] for b in B])
    _, D = float_rows(at + 128, N, "bf16", fill=7.0)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    assert plan.run_grouped_mx4(A, SA, Bq, SB, D, dev(starts), dev(counts), K=K) == g.GEMM_OK
    assert plan.last_config()["stages"] == (6 if E == 64 else 5)
    inside = np.zeros(at + 128, bool)
    for e, (s, c) in enumerate(zip(starts, counts)):
        if c:
            inside[s:s + c] = True
            near(D[s:s + c], *expect(a[s:s + c], B[e][2]), "bf16")
    assert (D[torch.from_numpy(~inside).cuda()] == 7.0).all()
    assert plan.poll_error() == g.GEMM_OK


@pytest.mark.parametrize("act", [3, 4])
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_activations_of_exact_products(plan, g, monkeypatch, act, out):
    """One product to each result, exact: the activation by itself, from small values to beyond where it ends, and NaN.

    Tolerance: the exponent's rounding -- SiLU's is one product by a constant that is 2^-26 off, 1.25 |x| 2^-24; GELU's two, of
    x^2 / 2, 1.125 x^2 2^-24; both below 2^-16 where the result is not 0 -- and 2^-20 for the rest, relative, and half a step."""
    import torch
    monkeypatch.setenv("GEMM_SCALED_KERNEL", "pair")
    K = 1312
    code, byte = np.zeros((256, K), int), np.full((256, K // 32), 127)
    code[:, 0] = np.arange(256) % 16  # x = value * value * 2^e, e = -14 to 1
    byte[:, 0] = 127 - 14 + np.arange(256) // 16
    w = np.zeros((24, K), int)
    w[:, 0] = 1 + np.arange(24) % 7
    wb = np.full((24, K // 32), 127)
    wb[8:, 0], wb[16:, 0] = 130, 127 + 120  # times 8; far out
    a, b = (ref.scaled4(ref.decode4(ref.pack4(c), K), s) for c, s in ((code, byte), (w, wb)))
    byte[255, 0] = 255
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    buf, D = float_rows(256, 24, out)
    A, B = (dev(np.ascontiguousarray(ref.pack4(c))) for c in (code, w))
    assert A.stride(0) % 16 == 0
    assert plan.run_mx4(A, dev(ref.pack_scales4(byte, K)), B, dev(ref.pack_scales4(wb, K)), D, K=K, act=act) == g.GEMM_OK
    assert plan.last_config()["stages"] == 6 and plan.poll_error() == g.GEMM_OK
    assert torch.isnan(D[255]).all()
    x = (a @ b.T)[:255]
    want = scaled_ref.act(x, act)
    most = 65520 if out == "f16" else 3.4e38
    got, want = (np.where(np.abs(v) >= most, np.sign(v) * most, v) for v in (D[:255].double().cpu().numpy(), want))
    part = np.minimum(1.25 * np.abs(x) * 2.0 ** -24 if act == 4 else 1.125 * x * x * 2.0 ** -24, 2.0 ** -16)
    # (1 / (1 + exp(-x)) and exp(-x^2 / 2) below the smallest normal number, 2^-126, may be 0)
    tol = np.abs(want) * (part + 2.0 ** -20 + ROUND[out]) + (2.0 ** -25 if out == "f16" else 2.0 ** -119)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (x[bad][:4], got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("slices", [1, 2, 3, 5, 8])
def test_product_slices(plan, g, monkeypatch, slices):
    monkeypatch.setenv("GEMM_SCALED_KERNEL", "sliced")
    monkeypatch.setenv("GEMM_SCALED_SLICES", str(slices))
    rng = np.random.default_rng(slices)
    for M, N, K in ((1, 300, 5000), (100, 140, 2600), (128, 128, 256)):
        A, SA, a = operand(rng, M, K)
        B, SB, b = operand(rng, N, K)
        import torch
        first = None
        for _ in range(2):
            _, D = float_rows(M, N, "f32")
            assert plan.run_mx4(A, SA, B, SB, D, K=K) == g.GEMM_OK
            near(D, *expect(a, b), "f32")
            assert first is None or torch.equal(first, D)  # the same bits every time
            first = D
    assert plan.poll_error() == g.GEMM_OK


@pytest.mark.parametrize("by,off", [(0, 8), (8, 0), (4, 4), (1, 3)])
@pytest.mark.parametrize("K", [41, 1000])
def test_operands_at_any_address(plan, g, by, off, K):
    rng = np.random.default_rng(by * 10 + off + K)
    A, SA, a = operand(rng, 70, K, ld_extra=by, offset=off)
    B, SB, b = operand(rng, 140, K, ld_extra=by, offset=off)
    _, D = float_rows(70, 140, "f32")
    assert plan.run_mx4(A, SA, B, SB, D, K=K) == g.GEMM_OK
    assert plan.last_config()["launches"] == 3  # both copied first
    near(D, *expect(a, b), "f32")


@pytest.mark.parametrize("kernel", KERNELS)
def test_nan_scales_stay_in_their_row_and_column(plan, g, monkeypatch, kernel):
    import torch
    if kernel:
        monkeypatch.setenv("GEMM_SCALED_KERNEL", kernel)
    x, w = torch.randn((70, 600), device="cuda"), torch.randn((300, 600), device="cuda")
    x[3, 100], w[200, 599] = float("nan"), float("inf")
    codes = []
    for t in (x, w):
        _, q = byte_rows(t.shape[0], 300, 0)
        s = scale_room(g, *t.shape)
        assert plan.quantize_mx4(t, q, s) == g.GEMM_OK
        codes += [q, s]
    _, D = float_rows(70, 300, "f32", fill=0.0)
    assert plan.run_mx4(*codes, D) == g.GEMM_OK
    nan = torch.isnan(D)
    want = torch.zeros_like(nan)
    want[3], want[:, 200] = True, True
    assert torch.equal(nan, want)


def test_no_k_and_no_rows(plan, g):
    import torch
    e = torch.empty((0, 0), dtype=torch.uint8, device="cuda")
    s = torch.zeros(512, dtype=torch.uint8, device="cuda")
    D = torch.full((4, 8), 2.0, device="cuda")
    A, B = torch.empty((4, 0), dtype=torch.uint8, device="cuda"), torch.empty((8, 0), dtype=torch.uint8, device="cuda")
    assert plan.run_mx4(A, s, B, s, D, beta=-1.0, act=g.GEMM_ACT_RELU) == g.GEMM_OK
    assert (D == 0).all()
    D.fill_(2.0)
    assert plan.run_mx4(A, s, B, s, D, beta=0.5) == g.GEMM_OK and (D == 1).all()
    assert plan.run_mx4(e, s, B, s, torch.empty((0, 8), device="cuda")) == g.GEMM_OK
    assert plan.last_config()["path"] == "none"


COUNTS = [[5], [0, 1, 0], [128, 1, 127, 129], [3, 0, 300, 64, 17, 0, 0, 200], [1] * 33, [700, 0, 260]]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "e%d" % len(c))
def test_grouped(plan, g, monkeypatch, kernel, counts):
    import torch
    if kernel:
        monkeypatch.setenv("GEMM_SCALED_KERNEL", kernel)
    rng = np.random.default_rng(sum(counts))
    E, N, K = len(counts), 140, 700
    starts, at = [], 0
    for c in counts:
        starts.append(at)
        at += -(-c // 128) * 128
    rows = at + 128
    A, SA, a = operand(rng, rows, K)
    B = [operand(rng, N, K) for _ in range(E)]
    Bq, SB = torch.stack([b[0] for b in B]), torch.cat([b[1] for b in B])
    _, D = float_rows(rows, N, "bf16", fill=7.0)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    assert plan.run_grouped_mx4(A, SA, Bq, SB, D, dev(starts), dev(counts), act=g.GEMM_ACT_SILU) == g.GEMM_OK
    inside = np.zeros(rows, bool)
    for e, (s, c) in enumerate(zip(starts, counts)):
        if c:
            inside[s:s + c] = True
            near(D[s:s + c], *expect(a[s:s + c], B[e][2], act=4), "bf16")
    assert (D[torch.from_numpy(~inside).cuda()] == 7.0).all()  # rows of no group are left as they are
    assert plan.poll_error() == g.GEMM_OK


def test_grouped_takes_no_row_outside(plan, g):
    """Starts and counts that lead out of the buffers: empty, or cut."""
    import torch
    rng = np.random.default_rng(3)
    A, SA, a = operand(rng, 256, 64)
    B = [operand(rng, 64, 64) for _ in range(5)]
    Bq, SB = torch.stack([b[0] for b in B]), torch.cat([b[1] for b in B])
    _, D = float_rows(256, 64, "f32", fill=7.0)
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    assert plan.run_grouped_mx4(A, SA, Bq, SB, D, dev([-128, 64, 256, 128, 0]), dev([128, 10, 4, 10 ** 9, -3])) == g.GEMM_OK
    near(D[128:], *expect(a[128:], B[3][2]), "f32")
    assert (D[:128] == 7.0).all()


def test_many_tiles(plan, g):
    """More tiles than CTAs: the pipeline's phases, both accumulators and every set of scale columns turn over."""
    rng = np.random.default_rng(9)
    A, SA, a = operand(rng, 2100, 1500)
    B, SB, b = operand(rng, 6150, 1500)
    _, D = float_rows(2100, 6150, "bf16")
    assert plan.run_mx4(A, SA, B, SB, D) == g.GEMM_OK
    near(D, *expect(a, b), "bf16")
    assert plan.poll_error() == g.GEMM_OK


def test_on_a_stream_and_in_a_graph(plan, g):
    import torch
    rng = np.random.default_rng(11)
    x = torch.from_numpy(rng.standard_normal((48, 520))).to(torch.bfloat16).cuda()
    B, SB, b = operand(rng, 264, 520)
    _, q = byte_rows(48, 260, 0)
    s = scale_room(g, 48, 520)
    _, D = float_rows(48, 264, "f32")
    v = torch.empty((48, 520), device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        assert plan.quantize_mx4(x, q, s) == g.GEMM_OK
        assert plan.run_mx4(q, s, B, SB, D) == g.GEMM_OK
        assert plan.dequantize(q, s, v) == g.GEMM_OK
    for _ in range(3):
        x.copy_(torch.from_numpy(rng.standard_normal((48, 520))))
        graph.replay()
        torch.cuda.synchronize()
        near(D, *expect(v.double().cpu().numpy(), b), "f32")


def test_refusals(plan, g):
    import torch
    x = torch.zeros((8, 64), device="cuda", dtype=torch.bfloat16)
    q, s = torch.zeros((8, 32), device="cuda", dtype=torch.uint8), torch.zeros(512, device="cuda", dtype=torch.uint8)
    call = lambda **c: g.gemm_quantize_mx(*{**dict(  # noqa: E731
        plan=plan.handle, rows=8, cols=64, X=x.data_ptr(), ldx=64, x_type=0, rowmap=None, map_div=1, src_rows=8, Q=q.data_ptr(), ldq=32,
        SQ=s.data_ptr(), QT=None, ldqt=0, SQT=None), **c}.values())
    assert call() == g.GEMM_OK and call(rows=0) == g.GEMM_OK and call(cols=0) == g.GEMM_OK
    for bad in ({"rows": -1}, {"x_type": 4}, {"Q": None}, {"SQ": None}, {"ldx": 63}, {"ldq": 16}, {"X": None}, {"Q": x.data_ptr()},
                {"SQ": q.data_ptr()}, {"QT": q.data_ptr()}, {"rowmap": s.data_ptr(), "map_div": 0}, {"plan": None}):
        assert call(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    for bad in ({"SQ": s.data_ptr() + 4}, {"X": x.data_ptr() + 1}):
        assert call(**bad) == g.GEMM_ERR_ALIGNMENT, bad
    assert call(rows=2 ** 24) == g.GEMM_ERR_UNSUPPORTED
    back = lambda **c: g.gemm_dequantize(*{**dict(plan=plan.handle, rows=8, cols=64, Q=q.data_ptr(), ldq=32, q_type=6, SQ=s.data_ptr(),  # noqa: E731
                                                  X=x.data_ptr(), ldx=64, x_type=0), **c}.values())
    assert back() == g.GEMM_OK and back(rows=0, Q=None, X=None) == g.GEMM_OK
    for bad in ({"q_type": 0}, {"q_type": 7}, {"x_type": 4}, {"Q": None}, {"SQ": None}, {"X": None}, {"ldq": 16}, {"ldx": 63},
                {"X": q.data_ptr()}, {"X": s.data_ptr()}, {"plan": None}, {"cols": -1}):
        assert back(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    for bad in ({"SQ": s.data_ptr() + 4}, {"X": x.data_ptr() + 1}):
        assert back(**bad) == g.GEMM_ERR_ALIGNMENT, bad
    with pytest.raises(ValueError):
        plan.quantize_mx4(x, q, s[:100])
    with pytest.raises(ValueError):
        plan.quantize_mx4(x, q[:, :31], s)
    with pytest.raises(ValueError):
        plan.run_mx4(q, s, q, s, torch.empty((8, 8), device="cuda"), K=62)
    with pytest.raises(ValueError):
        plan.run_mx4(x, s, q, s, torch.empty((8, 8), device="cuda"))
