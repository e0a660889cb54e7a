"""Routing, the order of the slots and the weighted sum on the GPU against 64-bit
numpy (tests/scaled_ref.py).

Indices, counts and positions are whole numbers and have to be equal: the logits lie on a grid
coarser than fp32's rounding of the scores, so the order of the keys does not hang on it.
Tolerances: a score is an fp32 exponential (2^-21 with its argument's rounding, times |x| at
most 30 for softmax's differences: 2^-19), a sum of at most 1024 terms (2^-19) and two
divisions; renormalising adds a sum of 32 and a division: 2^-17 of the value in all.  The logits'
gradient is a sum of at most 33 such products whose terms' magnitudes are added up: 2^-16 of
that.  The weighted sum and its gradients add k (or N) products in fp32: (n + 2) 2^-24 of the sum
of magnitudes, then half a unit of the result's type.
"""
import numpy as np
import pytest

from tests import scaled_ref as ref
from tests.test_scaled_gpu import ROUND, dtype, g, plan, rows_of  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def grid_logits(rng, T, E, name="f32", ties=False):
    """Every row a random order of E values 1/8 apart (1/4 and repeated, with ties)."""
    x = rng.permuted(np.tile(np.arange(E) / 8.0 - E / 16.0, (T, 1)), axis=1)
    if E > 64:
        x = x * (8.0 / E) * 4  # within the exponential's range: bf16 still tells neighbours apart or ties them
    if ties:
        x = np.round(x * 2) / 2
    return x


def run_route(plan, gm, x, k, name="f32", pad=0, **how):
    import torch
    T, E = x.shape
    buf = torch.full((T, E + pad), 77.0, device="cuda", dtype=dtype(name))
    buf[:, :E] = torch.from_numpy(x)
    w = torch.full((T, k), -5.0, device="cuda")
    i = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    bias = how.pop("bias", None)
    score = how.pop("score", "softmax")
    st = plan.route(buf[:, :E], w, i, bias=None if bias is None else torch.from_numpy(bias).float().cuda(),
                    score=gm.GEMM_SCORE_SIGMOID if score == "sigmoid" else gm.GEMM_SCORE_SOFTMAX, **how)
    assert st == 0
    return buf[:, :E].double().cpu().numpy(), w.double().cpu().numpy(), i.cpu().numpy()


ROUTES = [  # T, E, k, how
    (1, 1, 1, {}), (1, 8, 2, {"renormalize": True}), (3, 8, 8, {}), (33, 60, 6, {"renormalize": True, "scale": 2.5}),
    (5, 256, 8, {"score": "sigmoid", "groups": 8, "top_groups": 4, "group_top": 2, "renormalize": True, "bias": True}),
    (130, 160, 6, {"groups": 8, "top_groups": 3}), (7, 1024, 32, {"renormalize": True}), (64, 33, 1, {"score": "sigmoid"}),
    (9, 96, 5, {"score": "sigmoid", "groups": 32, "top_groups": 7, "group_top": 2, "bias": True}),
    (9, 32, 4, {"groups": 32, "top_groups": 5, "group_top": 2}), (2000, 64, 4, {"bias": True}),
]


@pytest.mark.parametrize("T,E,k,how", ROUTES)
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_route(plan, g, T, E, k, how, name):
    rng = np.random.default_rng(T + E + k)
    how = dict(how)
    if how.get("bias"):
        how["bias"] = rng.integers(-3, 4, E) / 64.0
    for ties in (False, True):
        x = grid_logits(rng, T, E, ties=ties)
        x, w, i = run_route(plan, g, x, k, name, pad=3, **how)
        want_i, want_w, s = ref.route(x, k, **how)
        if "bias" in how:  # equal sums may round apart: leave out rows whose order hangs on that
            key = s + how["bias"]
            near = np.abs(np.diff(np.sort(key, 1), axis=1)).min(1) < 1e-6 if E > 1 else np.zeros(T, bool)
            if how.get("groups", 1) > 1:
                two = np.sort(key.reshape(T, how["groups"], -1), 2)[..., -2:].sum(2)
                near |= np.abs(np.diff(np.sort(two, 1), axis=1)).min(1) < 1e-6
            x, w, i, want_i, want_w = (v[~near] for v in (x, w, i, want_i, want_w))
        elif how.get("group_top") == 2:  # keys are scores: equal logits tie exactly, sums of two may round apart
            two = np.sort(s.reshape(T, how["groups"], -1), 2)[..., -2:].sum(2)
            gap = np.abs(np.diff(np.sort(two, 1), axis=1))
            near = ((gap > 0) & (gap < 1e-6)).any(1)
            x, w, i, want_i, want_w = (v[~near] for v in (x, w, i, want_i, want_w))
        np.testing.assert_array_equal(i, want_i)
        assert (np.abs(w - want_w) <= 2.0 ** -17 * np.abs(want_w) + 1e-37).all()
    assert plan.poll_error() == 0


def test_route_masks(plan, g):
    inf = np.inf
    x = np.array([[-inf] * 8, [0, -inf, 1, -inf, -inf, -inf, -inf, -inf], [np.nan, 2, np.nan, 1, 3, 0, -1, -2],
                  [inf, 0, inf, 1, 2, 3, 4, 5], [-3.4e38] * 8, [3.4e38, -3.4e38, 0, 0, 0, 0, 0, 0], [0.0, -0.0] * 4,
                  [-inf, -inf, -inf, -inf, 1, 2, 3, 4]])
    for score in ("softmax", "sigmoid"):
        for how in ({}, {"renormalize": True}, {"bias": np.arange(8) / 4.0}, {"groups": 2, "top_groups": 1},
                    {"groups": 2, "top_groups": 1, "group_top": 2}):
            _, w, i = run_route(plan, g, x, 3, score=score, **how)
            want_i, want_w, _ = ref.route(x.astype(np.float32), 3, score=score, **how)
            np.testing.assert_array_equal(i, want_i)
            assert np.isfinite(w).all() and (np.abs(w - want_w) <= 2.0 ** -17 * want_w + 1e-37).all()


@pytest.mark.parametrize("T,E,k,how", [r for r in ROUTES if "bias" not in r[3] and "groups" not in r[3]])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_gradient(plan, g, T, E, k, how, score):
    import torch
    rng = np.random.default_rng(T * E + k)
    how = {n: v for n, v in how.items() if n != "score"}
    for name in ("f32", "bf16"):
        x, _, i = run_route(plan, g, grid_logits(rng, T, E), k, name, score=score, **how)
        i[0, 0] = -1  # takes no part
        if T > 1:
            i[1, k - 1] = E
        dw = rng.standard_normal((T, k)).astype(np.float32)
        xd = torch.full((T, E + 5), 3.0, device="cuda", dtype=dtype(name))
        xd[:, :E] = torch.from_numpy(x)
        dx = torch.full((T, E + 2), 9.0, device="cuda", dtype=dtype(name))
        st = plan.route_backward(xd[:, :E], torch.from_numpy(i).cuda(), torch.from_numpy(dw).cuda(), dx[:, :E],
                                 score=g.GEMM_SCORE_SIGMOID if score == "sigmoid" else g.GEMM_SCORE_SOFTMAX, **how)
        assert st == 0
        want = ref.route_backward(x, i, dw, score, **how)
        _, _, s = ref.route(x, 1, score)
        total = np.array([max(sum(s[t, e] for e in i[t] if 0 <= e < E), 1e-30) for t in range(T)])[:, None]
        terms = s * np.abs(dw).sum(1, keepdims=True) * how.get("scale", 1.0) * 2 / (total if how.get("renormalize") else 1.0)
        got = dx[:, :E].double().cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -16 * terms + ROUND[name] * np.abs(want) + 1e-37).all()
        assert (dx[:, E:] == 9).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 100, 256])
def test_route_gradient_of_constant_weights(plan, g, score, E):
    """A renormalised weight that is 1 whatever the logits (one choice, or one that is not masked) has no gradient, exactly."""
    import torch
    rng = np.random.default_rng(E)
    T = 152
    kind = g.GEMM_SCORE_SIGMOID if score == "sigmoid" else g.GEMM_SCORE_SOFTMAX
    for k in (1, 3):
        x = torch.from_numpy(grid_logits(rng, T, E)).float().cuda()
        if k > 1:
            keep = torch.from_numpy(rng.integers(0, E, T)).cuda()
            x[torch.arange(E, device="cuda") != keep[:, None]] = -float("inf")
        w, i = torch.empty((T, k), device="cuda"), torch.empty((T, k), dtype=torch.int32, device="cuda")
        assert plan.route(x, w, i, score=kind, renormalize=True) == 0
        assert torch.equal(w[:, 0], torch.ones_like(w[:, 0]))
        dw, dx = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda(), torch.full((T, E), 9.0, device="cuda")
        assert plan.route_backward(x, i, dw, dx, score=kind, renormalize=True) == 0
        assert (dx == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_against_differences(plan, g, score, renormalize):
    """The kernel's gradient along random directions against central differences of the 64-bit
    weights, choice held: the difference's own error is a third derivative (at most 10) times h^2."""
    import torch
    rng = np.random.default_rng(6)
    T, E, k, h = 16, 24, 4, 1e-4
    x, _, i = run_route(plan, g, grid_logits(rng, T, E), k, score=score, renormalize=renormalize)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dx = torch.empty((T, E), device="cuda")
    assert plan.route_backward(torch.from_numpy(x).float().cuda(), torch.from_numpy(i).cuda(), torch.from_numpy(dw).cuda(), dx,
                               score=g.GEMM_SCORE_SIGMOID if score == "sigmoid" else g.GEMM_SCORE_SOFTMAX,
                               renormalize=renormalize) == 0

    def weights(x):
        _, _, s = ref.route(x, 1, score)
        w = np.take_along_axis(s, i.astype(np.int64), 1)
        return w / w.sum(1, keepdims=True) if renormalize else w

    for _ in range(4):
        d = rng.standard_normal((T, E))
        slope = ((weights(x + h * d) - weights(x - h * d)) * dw).sum(1) / (2 * h)
        got = (dx.double().cpu().numpy() * d).sum(1)
        assert (np.abs(got - slope) <= 10 * h * h * np.abs(d).max() ** 3 * np.abs(dw).sum(1) + 2.0 ** -16 * np.abs(dw).sum(1) * np.abs(d).max() * 4).all()


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 64), (37, 4, 5), (1000, 2, 1024), (4096, 1, 3), (5000, 8, 128), (16384, 8, 256)])
def test_route_map(plan, g, T, k, E):
    import torch
    rng = np.random.default_rng(T + k + E)
    idx = rng.integers(0, E, (T, k))
    idx[rng.random((T, k)) < 0.02] = -1
    idx[rng.random((T, k)) < 0.01] = E + 3
    if E > 2 and T:
        idx[idx == 1] = 0  # an expert that nobody chose
    rows = g.gemm_route_rows(T, k, E) + 200
    ints = lambda *n: torch.full(n, -77, dtype=torch.int32, device="cuda")  # noqa: E731
    starts, counts, pos, rowmap = ints(E), ints(E), ints(T, k), ints(rows)
    for _ in range(2):
        assert plan.route_map(torch.from_numpy(idx.astype(np.int32)).cuda(), E, starts, counts, pos, rowmap) == 0
        for got, want in zip((starts, counts, pos, rowmap), ref.order(idx, E, rows)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)


COMBINES = [(1, 1, 1, 3), (1, 8, 64, 2048), (5, 3, 4, 517), (33, 9, 16, 40), (200, 4, 8, 1024), (20, 17, 32, 264),
            (24, 9, 8, 700), (300, 2, 4, 600), (1100, 2, 4, 262)]


def combine_case(rng, g, T, k, E, N, y, o, pad):
    import torch
    idx = rng.integers(0, E, (T, k))
    rows = g.gemm_route_rows(T, k, E)
    _, _, pos, rowmap = ref.order(idx, E, rows)
    drop = rng.random((T, k)) < 0.1
    rowmap[pos[drop]] = -1
    pos = np.where(drop, np.where(rng.random((T, k)) < 0.5, -1, rows + 5), pos)
    ybuf, Y = rows_of(rows, N, y, fill=0x7F, extra=pad)  # NaN in rows that nobody has
    vals = torch.from_numpy(rng.standard_normal((rows, N))).cuda().to(dtype(y))
    used = torch.from_numpy(rowmap >= 0).cuda()
    Y[used] = vals[used]
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    return pos, rowmap, Y, w, torch.from_numpy(pos.astype(np.int32)).cuda(), torch.from_numpy(rowmap.astype(np.int32)).cuda()


@pytest.mark.parametrize("T,k,E,N", COMBINES)
@pytest.mark.parametrize("y,o", [("bf16", "bf16"), ("f32", "f16"), ("f16", "f32")])
def test_combine(plan, g, T, k, E, N, y, o):
    import torch
    rng = np.random.default_rng(T + k + E + N)
    for pad in (0, 1):
        pos, rowmap, Y, w, pd, rd = combine_case(rng, g, T, k, E, N, y, o, pad)
        rows = len(rowmap)
        ok = (pos >= 0) & (pos < rows)
        y64 = np.nan_to_num(Y.double().cpu().numpy())[np.where(ok, pos, 0)] * ok[..., None]
        w64 = w.double().cpu().numpy()[..., None]
        obuf, out = rows_of(T, N, o, fill=0x11, extra=pad)
        assert plan.combine(Y, pd, w, out) == 0
        want, size = (w64 * y64).sum(1), np.abs(w64 * y64).sum(1)
        got = out.double().cpu().numpy()
        assert (np.abs(got - want) <= (k + 2) * 2.0 ** -24 * size + ROUND[o] * np.abs(want) + (2.0 ** -24 if o == "f16" else 1e-37)).all()
        assert (obuf.view(torch.uint8).view(T, -1)[:, N * obuf.element_size():] == 0x11).all()

        _, dout = rows_of(T, N, o, extra=pad)
        dout.copy_(torch.from_numpy(rng.standard_normal((T, N))))
        dbuf, dY = rows_of(rows, N, y, fill=0x11, extra=pad)
        before = dY.clone()
        dw = torch.full((T, k), 5.0, device="cuda")
        d64 = dout.double().cpu().numpy()
        for mapped in (False, True):
            assert plan.combine_backward(dout, Y, pd, w, dY, dw, rowmap=rd if mapped else None) == 0
            terms = d64[:, None] * y64
            assert (np.abs(dw.double().cpu().numpy() - terms.sum(2)) <= (N + 2) * 2.0 ** -24 * np.abs(terms).sum(2) + 1e-37).all()
            got = dY.double().cpu().numpy()
            t, j = np.nonzero(ok)
            want = w64[t, j] * d64[t]
            assert (np.abs(got[pos[t, j]] - want) <= (2.0 ** -23 + ROUND[y]) * np.abs(want) + (2.0 ** -24 if y == "f16" else 1e-37)).all()
            free = np.ones(rows, bool)
            free[pos[t, j]] = False
            if mapped:
                assert (got[free] == 0).all()
            else:
                assert torch.equal(dY[torch.from_numpy(free).cuda()], before[torch.from_numpy(free).cuda()])


def test_combine_gradient_against_differences(plan, g):
    """<out, dout> is linear in Y and in w: the kernels' differences along a direction are its
    gradients, up to the forward's fp32 sums."""
    import torch
    rng = np.random.default_rng(11)
    T, k, E, N = 12, 3, 4, 64
    idx = rng.integers(0, E, (T, k))
    rows = g.gemm_route_rows(T, k, E)
    _, _, pos, rowmap = ref.order(idx, E, rows)
    pd = torch.from_numpy(pos.astype(np.int32)).cuda()
    Y, w, dout = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda() for s in ((rows, N), (T, k), (T, N)))
    dY, dw = torch.empty_like(Y), torch.empty_like(w)
    assert plan.combine_backward(dout, Y, pd, w, dY, dw, rowmap=torch.from_numpy(rowmap.astype(np.int32)).cuda()) == 0

    def loss(Y, w):
        out = torch.empty((T, N), device="cuda")
        assert plan.combine(Y, pd, w, out) == 0
        return (out.double() * dout.double()).sum().item()

    for _ in range(3):
        eY, ew = (torch.from_numpy(rng.choice([-1.0, 1.0], s).astype(np.float32)).cuda() for s in (Y.shape, w.shape))
        got = (loss(Y + eY, w) - loss(Y - eY, w)) / 2
        assert abs(got - (dY.double() * eY.double()).sum().item()) < 1e-3  # 768 outputs of size 4, off by 2^-22 each
        got = (loss(Y, w + ew) - loss(Y, w - ew)) / 2
        assert abs(got - (dw.double() * ew.double()).sum().item()) < 1e-3


def test_refusals(plan, g):
    import torch
    t = torch.zeros(4096, device="cuda")
    p = t.data_ptr()
    r = lambda **c: g.gemm_route_t(*{**dict(score=0, top_k=2, groups=1, top_groups=1, group_top=1, renormalize=0, scale=1.0), **c}.values())  # noqa: E731
    call = lambda route=r(), **c: g.gemm_route(*{**dict(plan=plan.handle, tokens=4, experts=8, logits=p, ldl=8, l_type=2,  # noqa: E731
                                                       bias=None, route=route, weights=p + 4096, indices=p + 8192), **c}.values())
    assert call() == g.GEMM_OK and call(tokens=0, logits=None) == g.GEMM_OK
    for bad in ({"tokens": -1}, {"experts": 0}, {"l_type": 4}, {"ldl": 7}, {"logits": None}, {"weights": None}, {"indices": None},
                {"route": r(score=2)}, {"route": r(top_k=0)}, {"route": r(groups=3)}, {"route": r(groups=4, top_groups=5)},
                {"route": r(groups=8, top_groups=1)}, {"route": r(group_top=3)}, {"route": r(top_k=9)}):
        assert call(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    for bad in ({"experts": 1025, "ldl": 1025}, {"route": r(top_k=33), "experts": 64, "ldl": 64}, {"tokens": 2 ** 31}):
        assert call(**bad) == g.GEMM_ERR_UNSUPPORTED, bad
    assert call(logits=p + 2) == g.GEMM_ERR_ALIGNMENT
    m = lambda **c: g.gemm_route_map(*{**dict(plan=plan.handle, tokens=4, top_k=2, experts=8, indices=p, starts=p + 1024,  # noqa: E731
                                              counts=p + 2048, pos=p + 3200, rowmap=p + 4096, rows=1152), **c}.values())
    assert m(tokens=1, rows=256) == g.GEMM_OK
    for bad in ({"rows": 1023}, {"indices": None}, {"starts": None}, {"pos": None}, {"rowmap": None}, {"top_k": 0}):
        assert m(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    assert m(experts=2000) == g.GEMM_ERR_UNSUPPORTED
    c = lambda **k: g.gemm_combine(*{**dict(plan=plan.handle, tokens=2, top_k=1, cols=8, rows=4, Y=p, ldy=8, y_type=2, pos=p + 1024,  # noqa: E731
                                            weights=p + 2048, out=p + 3200, ldo=8, out_type=2), **k}.values())
    assert c() == g.GEMM_OK and c(tokens=0) == g.GEMM_OK
    for bad in ({"ldy": 7}, {"Y": None}, {"pos": None}, {"out": p + 16}, {"top_k": 0}, {"y_type": 5}):
        assert c(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    assert c(out=p + 3074) == g.GEMM_ERR_ALIGNMENT
    with pytest.raises(ValueError):
        plan.combine(t.view(64, 64), torch.zeros((4, 2), dtype=torch.int64, device="cuda"), t[:8].view(4, 2), t.view(64, 64)[:4])


def test_results_may_not_share_bytes(plan, g):
    """A result over an input or over another result is refused before anything is launched: most would be read
    after they were written."""
    import torch
    t = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = t.data_ptr()
    T, E, k = 8, 16, 2
    r = g.gemm_route_t(0, k, 1, 1, 1, 0, 1.0)
    # logits 8 x 16 f32 in rows of 20: 624 bytes from p
    route = lambda **c: g.gemm_route(*{**dict(plan=plan.handle, tokens=T, experts=E, logits=p, ldl=20, l_type=2, bias=p + 1024,  # noqa: E731
                                              route=r, weights=p + 2048, indices=p + 4096), **c}.values())
    assert route() == 0 and route(weights=p + 624) == 0 and route(indices=p + 2048 + 64) == 0 and route(bias=None) == 0
    for bad in ({"weights": p}, {"weights": p + 620}, {"indices": p + 560}, {"indices": p + 2048 + 60}, {"weights": p + 1024 + 60},
                {"indices": p + 1024 - 60}):
        assert route(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    back = lambda **c: g.gemm_route_backward(*{**dict(plan=plan.handle, tokens=T, experts=E, logits=p, ldl=20, l_type=2, route=r,  # noqa: E731
                                                      indices=p + 4096, dweights=p + 2048, dlogits=p + 8192, lddl=20), **c}.values())
    assert back() == 0 and back(dlogits=p) == 0 and back(dlogits=p + 640, lddl=16) == 0
    for bad in ({"dlogits": p, "lddl": 16}, {"dlogits": p + 4}, {"dlogits": p + 4096 - 64, "lddl": 16}, {"dlogits": p + 2048}):
        assert back(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    t.zero_()
    rows = g.gemm_route_rows(T, k, E)
    order = lambda **c: g.gemm_route_map(*{**dict(plan=plan.handle, tokens=T, top_k=k, experts=E, indices=p, starts=p + 1024,  # noqa: E731
                                                  counts=p + 2048, pos=p + 3072, rowmap=p + 4096, rows=rows), **c}.values())
    assert order() == 0
    for bad in ({"pos": p}, {"pos": p + 60}, {"starts": p + 2048 + 60}, {"counts": p + 3072 - 60}, {"rowmap": p + 4}, {"pos": p + 4096 + 4 * rows - 4}):
        assert order(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    t.zero_()
    summed = lambda **c: g.gemm_combine(*{**dict(plan=plan.handle, tokens=T, top_k=k, cols=E, rows=32, Y=p, ldy=16, y_type=2,  # noqa: E731
                                                 pos=p + 4096, weights=p + 5120, out=p + 8192, ldo=16, out_type=2), **c}.values())
    assert summed() == 0
    for bad in ({"out": p + 1024}, {"out": p + 4096 + 60}, {"out": p + 5120 - 480}):
        assert summed(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    grads = lambda **c: g.gemm_combine_backward(*{**dict(  # noqa: E731
        plan=plan.handle, tokens=T, top_k=k, cols=E, rows=32, dout=p + 8192, ldo=16, out_type=2, Y=p, ldy=16, y_type=2, pos=p + 4096,
        weights=p + 5120, rowmap=p + 6144, dY=p + 16384, lddy=16, dweights=p + 7168), **c}.values())
    assert grads() == 0 and grads(dweights=p + 5120) == 0 and grads(rowmap=None) == 0
    for bad in ({"dY": p}, {"dY": p + 8192 + 256}, {"dY": p + 4096 + 60}, {"dY": p + 5120 + 60}, {"dY": p + 6144}, {"dweights": p + 16384 + 64},
                {"dweights": p + 5120 + 4}, {"dweights": p + 4096}, {"dweights": p + 6144 + 124}, {"dweights": p + 2044}, {"dweights": p + 8192}):
        assert grads(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    c = lambda **k: g.gemm_run_grouped(*{**dict(  # noqa: E731
        plan=plan.handle, groups=2, rows=256, N=32, K=64, starts=p + 40960, counts=p + 41984, A=p + 49152, lda=64, SA=p, a_type=4,
        B=p + 45056, ldb=64, b_group=2048, SB=p + 1024, b_type=4, D=p + 4096, ldd=32, d_type=2, alpha=1.0, beta=0.0), **k}.values())
    assert c() == 0 and c(starts=p + 4096 + 256 * 128) == 0
    for bad in ({"starts": p + 4096 + 64}, {"counts": p + 4096 + 256 * 128 - 4}):
        assert c(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    assert plan.poll_error() == 0


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("E", [8, 60, 128])
def test_gradients_in_place(plan, g, name, E):
    """dlogits over the logits, dweights over the weights: the same bits as in places of their own."""
    import torch
    rng = np.random.default_rng(E)
    T, k = 70, 4
    for score, renormalize in (("softmax", False), ("sigmoid", True), ("softmax", True)):
        x, _, i = run_route(plan, g, grid_logits(rng, T, E), k, name, score=score)
        i[3, 1] = i[3, 0]  # two choices of one expert
        how = dict(score=g.GEMM_SCORE_SIGMOID if score == "sigmoid" else g.GEMM_SCORE_SOFTMAX, renormalize=renormalize)
        xd = torch.from_numpy(x).cuda().to(dtype(name))
        i, dw, dx = torch.from_numpy(i).cuda(), torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda(), torch.empty_like(xd)
        assert plan.route_backward(xd, i, dw, dx, **how) == 0
        assert plan.route_backward(xd, i, dw, xd, **how) == 0
        assert torch.equal(xd, dx)
    for T, k, N in ((20, 4, 512), (20, 19, 512), (1500, 3, 256), (30, 5, 90)):
        pos, rowmap, Y, w, pd, rd = combine_case(rng, g, T, k, E, N, name, name, 0)
        _, dout = rows_of(T, N, name)
        dout.copy_(torch.from_numpy(rng.standard_normal((T, N))))
        dY, dw, dY2 = torch.zeros_like(Y), torch.empty_like(w), torch.zeros_like(Y)
        assert plan.combine_backward(dout, Y, pd, w, dY, dw, rowmap=rd) == 0
        assert plan.combine_backward(dout, Y, pd, w, dY2, w, rowmap=rd) == 0
        assert torch.equal(dY, dY2) and torch.equal(dw, w)
    assert plan.poll_error() == 0


@pytest.mark.parametrize("E", [8, 100, 256])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_gradient_of_tiny_scores(plan, g, score, E):
    """Renormalised weights of experts whose scores are near fp32's least numbers (a bias or the groups chose
    them): their sum's reciprocal overflows, the gradient does not.  Tolerance: a score s in that range is off by 2^-150
    and a quotient of sums of k by k + 1 times that over the least chosen score, besides the 2^-16 of the others; a gradient is at most
    the weights' sum of |dw| times 2."""
    import torch
    rng = np.random.default_rng(E + 1)
    T, k = 40, 4
    x = rng.uniform(-95.0, -86.0, (T, E)) if score == "softmax" else rng.uniform(-88.5, -87.0, (T, E))
    i = np.argsort(rng.random((T, E - 1)), 1)[:, :k] + 1
    if score == "softmax":
        x[:, 0] = 0.0  # the score that is not tiny, which nobody chose
    x = x.astype(np.float32)
    dw = (rng.standard_normal((T, k)) * 100).astype(np.float32)
    dx = torch.full((T, E), 9.0, device="cuda")
    assert plan.route_backward(torch.from_numpy(x).cuda(), torch.from_numpy(i.astype(np.int32)).cuda(), torch.from_numpy(dw).cuda(), dx,
                               score=g.GEMM_SCORE_SIGMOID if score == "sigmoid" else g.GEMM_SCORE_SOFTMAX, renormalize=True, scale=1.5) == 0
    want = ref.route_backward(x, i, dw, score, renormalize=True, scale=1.5)
    _, _, s = ref.route(x, 1, score)
    least = np.take_along_axis(s, i, 1).min(1, keepdims=True)
    got = dx.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= (2.0 ** -16 + (k + 1) * 2.0 ** -149 / least) * 2 * 1.5 * np.abs(dw).sum(1, keepdims=True)).all()
    assert (np.abs(want).max(1) > 1).mean() > 0.8  # (of the oracle alone: most rows have a gradient worth the name)


@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_of_sure_sigmoids(plan, g, renormalize):
    """Sigmoid scores near 1, whose gradient is s (1 - s): 1 - s keeps the precision of exp(-x) where s has none left.  Tolerance:
    test_route_gradient's, with that factor in the terms."""
    import torch
    rng = np.random.default_rng(21)
    T, E, k = 64, 40, 6
    x = rng.uniform(-2.0, 20.0, (T, E)).astype(np.float32)
    i = np.argsort(rng.random((T, E)), 1)[:, :k]
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dx = torch.empty((T, E), device="cuda")
    assert plan.route_backward(torch.from_numpy(x).cuda(), torch.from_numpy(i.astype(np.int32)).cuda(), torch.from_numpy(dw).cuda(), dx,
                               score=g.GEMM_SCORE_SIGMOID, renormalize=renormalize) == 0
    x64 = x.astype(np.float64)
    s, rest = 1 / (1 + np.exp(-x64)), 1 / (1 + np.exp(x64))
    sj = np.take_along_axis(s, i, 1)
    w = sj / sj.sum(1, keepdims=True) if renormalize else sj
    d = dw - (dw * w).sum(1, keepdims=True) if renormalize else dw
    want, terms = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(want, i, w * d, 1)
    np.put_along_axis(terms, i, w * (np.abs(dw).sum(1, keepdims=True) if renormalize else np.abs(dw)) * 2, 1)
    got = dx.double().cpu().numpy()
    assert (np.abs(got - want * rest) <= 2.0 ** -16 * terms * rest).all()
    assert rest[got != 0].min() < 1e-7


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (33, 60, 6), (7, 1024, 32), (70, 128, 8)])
def test_route_gradient_f16(plan, g, score, T, E, k):
    """Logits and their gradient in f16: test_route_gradient's tolerance and f16's least step."""
    import torch
    rng = np.random.default_rng(T * E + k + 1)
    for renormalize in (False, True):
        x, _, i = run_route(plan, g, grid_logits(rng, T, E), k, "f16", score=score, renormalize=renormalize)
        dw = rng.standard_normal((T, k)).astype(np.float32)
        xd = torch.full((T, E + 3), 3.0, device="cuda", dtype=torch.float16)
        xd[:, :E] = torch.from_numpy(x)
        dx = torch.full((T, E + 5), 9.0, device="cuda", dtype=torch.float16)
        assert plan.route_backward(xd[:, :E], torch.from_numpy(i).cuda(), torch.from_numpy(dw).cuda(), dx[:, :E],
                                   score=g.GEMM_SCORE_SIGMOID if score == "sigmoid" else g.GEMM_SCORE_SOFTMAX, renormalize=renormalize) == 0
        want = ref.route_backward(x, i, dw, score, renormalize)
        _, _, s = ref.route(x, 1, score)
        total = np.take_along_axis(s, i.astype(np.int64), 1).sum(1, keepdims=True) if renormalize else 1.0
        terms = s * np.abs(dw).sum(1, keepdims=True) * 2 / total
        got = dx[:, :E].double().cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -16 * terms + ROUND["f16"] * np.abs(want) + 2.0 ** -25).all()
        assert (dx[:, E:] == 9).all()
