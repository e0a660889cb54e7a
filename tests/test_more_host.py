"""Host side of the 4-bit products, the norm and the balance loss: sizes, every refusal of gemm_check_mx, calls without a
plan, and the references' own pins, without a device."""
import numpy as np
import pytest

from dense_gemm_mma_gb300 import gemm as g
from tests import more_ref as ref


@pytest.fixture(scope="module", autouse=True)
def built_library():
    import __graft_entry__
    __graft_entry__.build_library()
    g.load()


@pytest.mark.parametrize("rows,cols", [(1, 1), (0, 0), (128, 128), (129, 129), (1, 4096), (1000, 127)])
def test_scale_bytes(rows, cols):
    n = g.gemm_mx_scale_bytes(rows, cols)
    assert n == max(1, -(-rows // 128)) * max(1, -(-cols // 128)) * 512
    if cols:
        assert ref.pack_scales4(np.zeros((rows, -(-cols // 32)), np.int64), cols).size == n


def test_sizes_out_of_range():
    assert g.gemm_mx_scale_bytes(-1, 5) == -1 and g.gemm_mx_scale_bytes(5, 2 ** 31) == -1


OK = dict(M=64, N=96, K=201, A=0x100000, lda=112, SA=0x200000, B=0x300000, ldb=112, SB=0x400000, D=0x500000, ldd=96, d_type=0,
          alpha=1.0, beta=0.0, act=0)


def check(**change):
    return g.gemm_check_mx(**{**OK, **change})


def test_accepts():
    assert check() == g.GEMM_OK
    assert check(lda=101, ldb=101) == g.GEMM_OK  # (K + 1) / 2 bytes; copied before they are read
    assert check(d_type=2, beta=1.0, act=4) == g.GEMM_OK
    assert check(M=0, A=None, B=None, SA=None, SB=None, D=None) == g.GEMM_OK
    assert check(K=0, A=None, B=None, SA=None, SB=None) == g.GEMM_OK
    assert check(D=0x100000 + 64 * 112) == g.GEMM_OK  # behind A's last row


@pytest.mark.parametrize("change", [
    {"M": -1}, {"N": -1}, {"K": -1}, {"d_type": 3}, {"d_type": 4}, {"d_type": 6}, {"act": 5}, {"lda": 100}, {"ldb": 100}, {"ldd": 95},
    {"D": None}, {"A": None}, {"B": None}, {"SA": None}, {"SB": None}, {"D": 0x100000}, {"D": 0x300010}, {"D": 0x200000},
    {"D": 0x400000 + 1008},  # the last bytes of B's two scale tiles
])
def test_invalid(change):
    assert check(**change) == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [{"SA": 0x200004}, {"SB": 0x400008}, {"D": 0x500008}, {"ldd": 100}])
def test_misaligned(change):
    assert check(**change) == g.GEMM_ERR_ALIGNMENT


@pytest.mark.parametrize("change", [{"M": 2 ** 31}, {"N": 2 ** 31, "ldd": 2 ** 32}, {"K": 2 ** 31, "lda": 2 ** 32, "ldb": 2 ** 32}])
def test_unsupported(change):
    assert check(**change) == g.GEMM_ERR_UNSUPPORTED


def test_the_8_bit_product_takes_no_4_bit_type():
    assert g.gemm_check_scaled(64, 96, 200, 0x100000, 208, 0x200000, 6, 0x300000, 208, 0x400000, 6, 0x500000, 96, 0, 1.0, 0.0) == g.GEMM_ERR_INVALID_ARG


def test_calls_without_a_plan_are_refused():
    bad = g.GEMM_ERR_INVALID_ARG
    assert g.gemm_run_mx(None, *[OK[n] for n in ("M", "N", "K", "A", "lda", "SA", "B", "ldb", "SB", "D", "ldd", "d_type")], 1.0, 0.0) == bad
    assert g.gemm_run_grouped_mx(None, 1, 128, 8, 32, 16, 16, 16, 16, 16, 16, 16, 128, 16, 16, 8, 2, 1.0, 0.0) == bad
    assert g.gemm_quantize_mx(None, 1, 32, 16, 32, 2, None, 1, 1, 16, 16, 16, None, 0, None) == bad
    assert g.gemm_dequantize(None, 1, 32, 16, 16, 6, 16, 16, 32, 2) == bad
    assert g.gemm_norm(None, 1, 8, 16, 8, 2, None, 0, 2, None, 2, 1e-6, None, 0, 64, 8, 4, None, 0, None, None) == bad
    assert g.gemm_norm_backward(None, 1, 8, 16, 8, 2, 16, 8, 2, None, 2, 16, None, 0, 64, 8, None) == bad
    assert g.gemm_balance(None, 1, 4, 16, 4, 2, 0, 1, 16, 1.0, 16, 16, 16, 16) == bad
    assert g.gemm_balance_backward(None, 1, 4, 16, 4, 2, 0, 1, 16, 16, None, 0, 16, 4) == bad


def test_quantize_reference_is_the_nearest_code():
    """The reference's own pin: its values are codes, and no code lies nearer."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 100)) * 10.0 ** rng.integers(-6, 6, (4, 1))
    v, byte = ref.quantize4(x)
    y = x / np.repeat(2.0 ** (byte - 127.0), 32, axis=1)[:, :100]
    codes = np.concatenate([ref.E2M1, -ref.E2M1])
    assert np.isin(v, codes).all()
    assert np.allclose(np.abs(v - y), np.abs(codes[None, None] - y[..., None]).min(-1), rtol=0, atol=1e-12)
    for b in range(4):
        m = np.abs(y[:, 32 * b:32 * b + 32]).max(1)
        assert (m <= 6).all() and (m > 3).all()
    assert np.array_equal(ref.decode4(ref.pack4(np.arange(16)[None]), 16)[0], codes)


def test_references_gradients_against_differences():
    rng = np.random.default_rng(2)
    x, gain, w = rng.standard_normal((3, 9)), 1 + 0.2 * rng.standard_normal(9), rng.standard_normal((3, 9))
    _, rstd, _ = ref.norm(x, None, gain, 1e-3)
    dx, dgain, _, _ = ref.norm_backward(w, x, gain, rstd, None)
    d, dg, e = rng.standard_normal((3, 9)), rng.standard_normal(9), 1e-5
    f = lambda x, gain: (ref.norm(x, None, gain, 1e-3)[2] * w).sum()  # noqa: E731
    assert abs((f(x + e * d, gain) - f(x - e * d, gain)) / (2 * e) - (dx * d).sum()) < 1e-7
    assert abs((f(x, gain + e * dg) - f(x, gain - e * dg)) / (2 * e) - (dgain * dg).sum()) < 1e-7
    index = np.array([[0, 2], [2, 2], [-1, -1], [1, 9]])
    x, d = rng.standard_normal((4, 5)), rng.standard_normal((4, 5))
    for score in ("softmax", "sigmoid"):
        dx = ref.balance_backward(x, index, ref.balance(x, index, score)[2], 1.0, score)
        f = lambda x: ref.balance(x, index, score)[3]  # noqa: E731
        assert abs((f(x + e * d) - f(x - e * d)) / (2 * e) - (dx * d).sum()) < 1e-8
