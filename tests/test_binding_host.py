"""What the binding makes of a tensor's strides, without a device: a layout that the kernels cannot address is
refused with ValueError before any call; a stride is replaced only where no second row or matrix uses it."""
import pytest

from dense_gemm_mma_gb300 import gemm as g

torch = pytest.importorskip("torch")


@pytest.fixture
def plan(monkeypatch):
    """A plan whose every call into the library fails the test."""
    def load():
        raise AssertionError("called the library")
    monkeypatch.setattr(g, "load", load)
    p = g.Plan.__new__(g.Plan)
    p.handle, p.device, p._current = None, 0, lambda device: 0
    return p


def codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn)


def scales(rows, cols, groups=1):
    return torch.zeros(groups * max(1, -(-rows // 128)) * max(1, -(-cols // 512)) * 512, dtype=torch.uint8)


def test_strides_of_a_matrix():
    t = torch.zeros((6, 40))
    for view, want in ((t, 40), (t[:, :7], 40), (t[::2], 80), (t[:1], 40), (t[:1].expand(1, 40), 40),
                       (torch.zeros(40).expand(1, 40), 40), (torch.zeros((5, 0)), 1), (torch.zeros((0, 8)), 8),
                       (torch.zeros(1).expand(6, 1)[:1], 1), (t[:, :1], 40), (t.t()[:1, :1], 1)):
        p, rows, cols, ld = g._matrix(view)
        assert (p, rows, cols) == (view.data_ptr(), *view.shape) and ld == want, view.shape
    assert g._matrix(torch.zeros(3).expand(0, 3))[3] == 3 and g._matrix(torch.zeros((1, 0)).expand(4, 0))[3] == 1


@pytest.mark.parametrize("rows,cols", [(2, 1), (4, 8), (64, 32)])
def test_rows_that_share_memory_are_refused(rows, cols):
    for t in (torch.zeros(cols).expand(rows, cols), torch.zeros(1).expand(rows, cols),
              torch.zeros(rows * cols).as_strided((rows, cols), (cols - 1 if cols > 1 else 0, 1))):
        with pytest.raises(ValueError):
            g._matrix(t)
    with pytest.raises(ValueError):
        g._matrix(torch.zeros((8, 4)).t())  # rows that are not contiguous


def test_expanded_arguments_never_reach_a_kernel(plan):
    """Gradients of sums and means are expanded rows; so are broadcast inputs."""
    T, k, N, E, rows = 6, 2, 32, 4, 512
    wide = lambda r, c=N: torch.zeros(c).expand(r, c)  # noqa: E731
    w, i = torch.zeros((T, k)), torch.zeros((T, k), dtype=torch.int32)
    Y = torch.zeros((rows, N))
    calls = [
        lambda: plan.quantize(wide(T), codes(T, N), scales(T, N)),
        lambda: plan.quantize(torch.zeros((T, N)), codes(N).expand(T, N), scales(T, N)),
        lambda: plan.quantize(torch.zeros((T, N)), QT=codes(T).expand(N, T), SQT=scales(N, T)),
        lambda: plan.run_scaled(codes(N).expand(T, N), scales(T, N), codes(8, N), scales(8, N), torch.zeros((T, 8))),
        lambda: plan.run_scaled(codes(T, N), scales(T, N), codes(N).expand(8, N), scales(8, N), torch.zeros((T, 8))),
        lambda: plan.run_scaled(codes(T, N), scales(T, N), codes(8, N), scales(8, N), wide(T, 8)),
        lambda: plan.route(wide(T, E), w, i),
        lambda: plan.route_backward(wide(T, E), i, w, torch.zeros((T, E))),
        lambda: plan.route_backward(torch.zeros((T, E)), i, w, wide(T, E)),
        lambda: plan.combine(wide(rows), i, w, torch.zeros((T, N))),
        lambda: plan.combine(Y, i, w, wide(T)),
        lambda: plan.combine_backward(wide(T), Y, i, w, torch.zeros_like(Y), torch.zeros_like(w)),
        lambda: plan.combine_backward(torch.zeros((T, N)), wide(rows), i, w, torch.zeros_like(Y), torch.zeros_like(w)),
        lambda: plan.combine_backward(torch.zeros((T, N)), Y, i, w, wide(rows), torch.zeros_like(w)),
    ]
    for n, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d" % n)


def test_strides_of_a_stack():
    t = torch.zeros((3, 5, 8))
    close = torch.zeros(64).as_strided((3, 2, 6), (14, 8, 1))  # a matrix begins right after the one before ends
    for view, ld, group in ((t, 8, 40), (t[:, :2], 8, 40), (t[:, :, :3], 8, 40), (t[::2], 8, 80), (t[:1], 8, 40), (close, 8, 14),
                            (t.transpose(0, 1)[:1], 40, 120), (torch.zeros((2, 0, 8)), 8, 8), (torch.zeros((4, 1, 8)), 8, 8),
                            (torch.zeros((5, 8)).expand(1, 5, 8), 8, 40), (torch.zeros((4, 6)).unsqueeze(1)[:, :, :1], 6, 6)):
        p, n, rows, cols, *strides = g._matrices(view)
        assert (p, n, rows, cols) == (view.data_ptr(), *view.shape) and strides == [ld, group], (view.shape, strides)


def test_stacks_whose_matrices_share_or_interleave_are_refused(plan):
    E, N, K, rows = 4, 32, 128, 512
    A, SA, i = codes(rows, K), scales(rows, K), torch.zeros(E, dtype=torch.int32)
    D = torch.zeros((rows, N))
    stacks = lambda n, r, c, zero: (  # noqa: E731
        zero(r, n, c).transpose(0, 1), zero(r, c).expand(n, r, c), zero(n, 1, c).expand(n, r, c), zero(n * r * c + 1).as_strided((n, r, c), (r * c - 1, c, 1)))
    for B in stacks(E, N, K, codes):
        with pytest.raises(ValueError):
            g._matrices(B)
        with pytest.raises(ValueError):
            plan.run_grouped(A, SA, B, scales(N, K, E), D, i, i)
    QT, ST = codes(N, rows), scales(N, rows)
    for out in stacks(E, N, N, lambda *shape: torch.zeros(shape)):
        with pytest.raises(ValueError):
            plan.run_grouped_k(QT, ST, QT, ST, out, i, i)


def test_expanded_operands_of_the_dense_product_are_refused(plan):
    bf16 = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)  # noqa: E731
    whole = (bf16(16, 64), bf16(64, 32), bf16(16, 32))
    for at, t in enumerate(whole):
        bad = list(whole)
        bad[at] = bf16(t.shape[1]).expand(*t.shape)
        with pytest.raises(ValueError):
            plan.run(*bad)
    assert g._operand(bf16(64).expand(1, 64), False)[1] == 64
    assert g._operand(whole[0][::2, :5], False)[1] == 128
