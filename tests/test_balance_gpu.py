"""The balance of a router's choice and its gradient on the GPU against 64-bit numpy (tests/more_ref.py).

Tolerance, with u = 2^-24: a difference of logits of size d is off by d u, which its exponential keeps as a relative error; expf
adds 4 u, a score's division 3 u; a token's sum of up to 1024 positive scores, 32 a lane and five exchanges, 40 u; its reciprocal 2 u: a share is off by
c = (60 + d) u, d the logits' spread.  The mean over T tokens adds their number a warp and the warps and CTAs behind one another, below T / 16 + 200
roundings, all terms positive.  Gradients: p (f - sum f p): three times c, and 40 u of the sum, of p (|f| + sum |f| p).
"""
import numpy as np
import pytest

from tests import more_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


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


class Call:
    def __init__(self, g, plan, logits, indices, score="softmax", scale=1.0):
        import torch
        E = logits.shape[1]
        self.counts = torch.full((E,), -7, dtype=torch.int32, device="cuda")
        self.shares, self.factor, self.loss = (torch.full((n,), float("nan"), device="cuda") for n in (E, E, 1))
        self.how = {"score": g.GEMM_SCORE_SIGMOID if score == "sigmoid" else g.GEMM_SCORE_SOFTMAX}
        assert plan.balance(logits, indices, self.counts, self.shares, self.factor, self.loss, scale=scale, **self.how) == g.GEMM_OK

    def all(self):
        return self.counts, self.shares, self.factor, self.loss


def near(got, want, tol):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], np.broadcast_to(want, got.shape)[bad][:4])


CASES = [(1, 1, 1), (1, 8, 2), (16, 256, 8), (33, 60, 6), (700, 5, 3), (5000, 128, 8), (300, 1000, 32), (1000, 1024, 4), (70, 300, 1), (4097, 64, 2)]


@pytest.mark.parametrize("T,E,k", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
def test_balance(plan, g, T, E, k, score, name):
    import torch
    rng = np.random.default_rng(T + E + k)
    x = torch.from_numpy(rng.standard_normal((T, E)) * 2).to(dtype(name))
    buf = torch.full((T, E + (T % 3)), 99.0, dtype=dtype(name), device="cuda")  # rows that are not together, not on 16-byte boundaries
    logits = buf[:, :E]
    logits.copy_(x)
    index = rng.integers(0, E, (T, k))  # the same expert twice among them
    index[rng.random(T) < 0.2] = -1
    index[rng.random((T, k)) < 0.05] = E + 3
    if T > 3:  # masks: an expert, all but one, all of them, NaN
        logits[1, 0] = float("-inf")
        logits[2, 1:] = float("-inf")
        logits[3] = float("-inf")
        logits[0, E // 2] = float("nan")
    x64 = logits.double().cpu().numpy()
    indices = torch.from_numpy(index.astype(np.int32)).cuda()
    scale = 0.01
    c = Call(g, plan, logits, indices, score, scale)
    counts, shares, factor, loss, p, live = ref.balance(x64, index, score, scale)
    assert np.array_equal(c.counts.cpu().numpy(), counts)
    finite = x64[np.isfinite(x64)]
    off = (60 + (finite.max() - finite.min() if finite.size else 0)) * U
    mean = off + (T / 16 + 200) * U
    near(c.shares, shares, shares * mean + 1e-37)
    near(c.factor, factor, factor * 8 * U)
    near(c.loss, loss, loss * (mean + 60 * U))
    again = Call(g, plan, logits, indices, score, scale)
    assert all(torch.equal(a, b) for a, b in zip(c.all(), again.all()))  # the same bits every time

    dloss = torch.tensor([1.5], device="cuda")
    dbuf = torch.full((T, E + (T % 2)), 5.0, dtype=dtype(name), device="cuda")
    dx = dbuf[:, :E]
    assert plan.balance_backward(logits, indices, c.factor, dx, dloss=dloss, **c.how) == g.GEMM_OK
    f = c.factor.double().cpu().numpy()
    want = ref.balance_backward(x64, index, f, 1.5, score)
    size = 1.5 * p * (np.abs(f) + (np.abs(f) * p).sum(1, keepdims=True)) * live[:, None]
    least = {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -24}[name]
    near(dx, want, size * (3 * off + 80 * U) + np.abs(want) * HALF[name] + least)
    assert (dbuf[:, E:] == 5.0).all()
    base = torch.from_numpy(rng.standard_normal((T, E)) * float(np.abs(want).max() or 1)).to(dtype(name)).cuda()
    both = base.clone()
    assert plan.balance_backward(logits, indices, c.factor, both, accumulate=True, **c.how) == g.GEMM_OK
    b64 = base.double().cpu().numpy()
    near(both, b64 + want / 1.5, size * (3 * off + 80 * U) + np.abs(b64 + want / 1.5) * (HALF[name] + U) + least)
    assert torch.equal(both[torch.from_numpy(~live).cuda()], base[torch.from_numpy(~live).cuda()])
    place = torch.nan_to_num(x.clone(), nan=0.0).cuda()  # the logits' own place
    apart = torch.empty_like(place)
    assert plan.balance_backward(place, indices, c.factor, apart, **c.how) == g.GEMM_OK
    assert plan.balance_backward(place, indices, c.factor, place, **c.how) == g.GEMM_OK
    assert torch.equal(place, apart)
    assert plan.poll_error() == g.GEMM_OK


@pytest.mark.parametrize("T", [0, 1, 100])
def test_no_token_has_a_choice(plan, g, T):
    import torch
    logits, indices = torch.randn((T, 12), device="cuda"), torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
    c = Call(g, plan, logits, indices)
    for t in c.all():
        assert (t == 0).all()
    dx = torch.full((T, 12), 3.0, device="cuda")
    assert plan.balance_backward(logits, indices, c.factor, dx) == g.GEMM_OK
    assert (dx == 0).all()


def test_even_and_uneven(plan, g):
    """An even router's loss is the scale; with every token sure of one expert it is the number of experts times that."""
    import torch
    T, E = 64, 16
    indices = (torch.arange(T, device="cuda") % E).to(torch.int32)[:, None]
    even = Call(g, plan, torch.zeros((T, E), device="cuda"), indices, scale=0.5)
    assert abs(float(even.loss) - 0.5) < 1e-6
    logits = torch.zeros((T, E), device="cuda")
    logits[:, 3] = 80.0
    sure = Call(g, plan, logits, torch.full((T, 1), 3, dtype=torch.int32, device="cuda"), scale=0.5)
    assert abs(float(sure.loss) - 0.5 * E) < 1e-5 and int(sure.counts[3]) == T


def test_sure_tokens_keep_their_gradient(plan, g):
    """p = 1 - 1e-6: the gradient of the surest expert is a difference of nearly equal numbers."""
    import torch
    T, E = 9, 40
    logits = torch.zeros((T, E), device="cuda")
    logits[:, 7] = 17.0
    index = torch.from_numpy(np.random.default_rng(1).integers(0, E, (T, 2)).astype(np.int32)).cuda()
    c = Call(g, plan, logits, index)
    dx = torch.empty_like(logits)
    assert plan.balance_backward(logits, index, c.factor, dx) == g.GEMM_OK
    want = ref.balance_backward(logits.double().cpu().numpy(), index.cpu().numpy(), c.factor.double().cpu().numpy(), 1.0)
    near(dx, want, np.abs(want) * 2.0 ** -17 + np.abs(want).max() * 2.0 ** -30)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(plan, g, score):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(4)
    T, E, k = 6, 12, 3
    x = torch.randn((T, E), generator=gen, device="cuda")
    index = x.topk(k, dim=1).indices.to(torch.int32)
    c = Call(g, plan, x, index, score)
    dx = torch.empty_like(x)
    assert plan.balance_backward(x, index, c.factor, dx, **c.how) == g.GEMM_OK
    step = 2.0 ** -6  # curvature ~ step^2 / 6 of a loss of 1: 4e-5; rounding: 70 u over two steps, 1.3e-4
    for _ in range(6):
        d = torch.randn((T, E), generator=gen, device="cuda")
        d = d / d.norm()
        diff = (float(Call(g, plan, x + step * d, index, score).loss) - float(Call(g, plan, x - step * d, index, score).loss)) / (2 * step)
        assert abs(diff - float((dx * d).sum())) < 1e-3


def test_on_a_stream_and_in_a_graph(g):
    """A plan's first calls, workspace and counters included, captured; replayed with new logits."""
    import torch
    plan = g.Plan(0)
    T, E, k = 3000, 64, 4
    logits, indices = torch.zeros((T, E), device="cuda"), torch.zeros((T, k), dtype=torch.int32, device="cuda")
    dx = torch.empty_like(logits)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c = Call(g, plan, logits, indices)
        assert plan.balance_backward(logits, indices, c.factor, dx) == g.GEMM_OK
    rng = np.random.default_rng(2)
    for _ in range(3):
        logits.copy_(torch.from_numpy(rng.standard_normal((T, E))))
        indices.copy_(torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        x64, index = logits.double().cpu().numpy(), indices.cpu().numpy()
        counts, shares, factor, loss, p, _ = ref.balance(x64, index)
        assert np.array_equal(c.counts.cpu().numpy(), counts)
        near(c.loss, loss, loss * 600 * U)
        near(dx, ref.balance_backward(x64, index, factor, 1.0), p * factor.max() * 600 * U)


def test_refusals(plan, g):
    import torch
    x, index = torch.zeros((8, 16), device="cuda"), torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    counts, shares, factor, loss = torch.zeros(16, dtype=torch.int32, device="cuda"), torch.zeros(16, device="cuda"), torch.zeros(16, device="cuda"), torch.zeros(1, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    call = lambda **c: g.gemm_balance(*{**dict(plan=plan.handle, tokens=8, experts=16, logits=p(x), ldl=16, l_type=2, score=0, top_k=2,  # noqa: E731
                                               indices=p(index), scale=1.0, counts=p(counts), shares=p(shares), factor=p(factor), loss=p(loss)), **c}.values())
    assert call() == g.GEMM_OK
    for bad in ({"plan": None}, {"tokens": -1}, {"experts": 0}, {"l_type": 4}, {"score": 2}, {"top_k": 0}, {"ldl": 15}, {"logits": None}, {"indices": None},
                {"counts": None}, {"shares": None}, {"factor": None}, {"loss": None}, {"counts": p(index)}, {"shares": p(x)}, {"factor": p(shares)},
                {"loss": p(shares) + 60}):
        assert call(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    for bad in ({"logits": p(x) + 2}, {"indices": p(index) + 2}, {"loss": p(loss) + 1}):
        assert call(**bad) == g.GEMM_ERR_ALIGNMENT, bad
    for bad in ({"experts": 1025, "ldl": 1025}, {"top_k": 33}, {"tokens": 2 ** 31}):
        assert call(**bad) == g.GEMM_ERR_UNSUPPORTED, bad
    dx, dloss = torch.zeros_like(x), torch.ones(1, device="cuda")
    back = lambda **c: g.gemm_balance_backward(*{**dict(plan=plan.handle, tokens=8, experts=16, logits=p(x), ldl=16, l_type=2, score=0, top_k=2,  # noqa: E731
                                                        indices=p(index), factor=p(factor), dloss=p(dloss), accumulate=0, dlogits=p(dx), lddl=16), **c}.values())
    assert back() == g.GEMM_OK and back(dloss=None) == g.GEMM_OK and back(dlogits=p(x)) == g.GEMM_OK
    for bad in ({"plan": None}, {"dlogits": None}, {"factor": None}, {"lddl": 15}, {"dlogits": p(x), "accumulate": 1}, {"dlogits": p(x) + 4},
                {"dlogits": p(factor)}, {"dlogits": p(x), "lddl": 20}):
        assert back(**bad) == g.GEMM_ERR_INVALID_ARG, bad
    with pytest.raises(ValueError):
        plan.balance(x, index[:4], counts, shares, factor, loss)
    with pytest.raises(ValueError):
        plan.balance(x, index, counts, shares[:10], factor, loss)
    with pytest.raises(ValueError):
        plan.balance_backward(x, index, factor, dx.bfloat16())
