"""Plan workspace and CUDA graphs: calls that need workspace may be captured as a plan's first calls, the graph may
be replayed any number of times, and it stays sound when later calls need more than the plan holds."""
import numpy as np
import pytest

from tests.test_scaled_gpu import g  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


class Work:
    """Calls that keep plan workspace: the order of many slots, a product of codes off the 16-byte grid, a product split along K,
    a product of one row."""

    def __init__(self, gm, scale):
        import torch
        T, k, E = 3000 * scale, 4, 64
        ints = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.gm, self.E = gm, E
        self.idx, self.rows = ints(T, k), gm.gemm_route_rows(T, k, E)
        self.order = lambda: (ints(E), ints(E), ints(T, k), ints(self.rows))
        M, N, K = 40 * scale, 132, 777
        self.A = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
        self.B = torch.zeros((N, K), dtype=torch.uint8, device="cuda")
        self.SA, self.SB = (torch.full((gm.gemm_scale_bytes(r, K),), 127, dtype=torch.uint8, device="cuda") for r in (M, N))
        self.P, self.Q = (torch.zeros((256 * scale, 65536), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.V, self.W = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((1, 8192), (8192, 1000 * scale)))
        self.new = lambda: (*self.order(), *(torch.zeros(s, device="cuda") for s in ((M, N), (256 * scale, 256 * scale), (1, 1000 * scale))))
        self.out = self.new()

    def fill(self, seed):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.idx.copy_(torch.randint(0, self.E, self.idx.shape, generator=gen, device="cuda"))
        for c in (self.A, self.B):
            c.copy_(torch.randint(0x28, 0x48, c.shape, generator=gen, device="cuda"))
        for x in (self.P, self.Q, self.V, self.W):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))

    def run(self, plan, out):
        """Runs them all into `out`; the workspace that they used."""
        import torch
        f8 = torch.float8_e4m3fn
        used = []
        assert plan.route_map(self.idx, self.E, *out[:4]) == 0
        for call in (lambda: plan.run_scaled(self.A.view(f8), self.SA, self.B.view(f8), self.SB, out[4]),
                     lambda: plan.run(self.P, self.Q, out[5], transB=True), lambda: plan.run(self.V, self.W, out[6])):
            assert call() == 0
            used.append(plan.last_config()["workspace_bytes"])
        return used


def test_first_calls_in_a_capture_and_growth_after_it(g):
    import torch
    plan, other = g.Plan(0), g.Plan(0)
    small, large = Work(g, 1), Work(g, 3)
    small.fill(0), large.fill(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        used = small.run(plan, small.out)  # the plan's first calls
    assert min(used) > 0, used
    held = []
    for n in range(6):
        if n == 3:  # larger calls outside the graph; what is freed by then is taken and filled by others
            assert min(a - b for a, b in zip(large.run(plan, large.out), used)) > 0
            torch.cuda.synchronize()
            held = [g.Plan(0) for _ in range(3)]
            for h in held:
                large.run(h, large.new())
        small.fill(10 + n)
        want = small.new()
        small.run(other, want)
        torch.cuda.synchronize()
        for t in small.out:
            t.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(small.out, want):
            assert torch.equal(a, b), n
    want = large.new()
    large.run(other, want)
    for a, b in zip(large.out, want):
        assert torch.equal(a, b)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):  # growth in a capture of what another graph holds
        large.run(plan, large.out)
    small.fill(99)
    small.run(other, want := small.new())
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(small.out, want):
        assert torch.equal(a, b)
    assert plan.poll_error() == 0


def test_growth_inside_a_capture(g):
    """A capture that needs more than the plan holds, after eager calls and after another graph."""
    import torch
    plan, other = g.Plan(0), g.Plan(0)
    small, large = Work(g, 1), Work(g, 2)
    small.fill(2), large.fill(3)
    small.run(plan, small.out)
    torch.cuda.synchronize()
    graphs = []
    for w in (small, large):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.run(plan, w.out)
        graphs.append(graph)
    for n in range(2):
        for w, graph in zip((small, large), graphs):
            w.fill(20 + n)
            w.run(other, want := w.new())
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(w.out, want):
                assert torch.equal(a, b)
    assert plan.poll_error() == 0 and np.isfinite(large.out[5].cpu().numpy()).all()
