"""Host side of the block-scaled products: the packed scale order, sizes and every
refusal of gemm_check_scaled, without a device."""
import numpy as np
import pytest

from dense_gemm_mma_gb300 import gemm as g
from tests import scaled_ref as ref


@pytest.fixture(scope="module", autouse=True)
def built_library():
    import __graft_entry__
    __graft_entry__.build_library()
    g.load()


@pytest.mark.parametrize("rows,cols", [(1, 1), (0, 0), (128, 512), (129, 513), (1, 4096), (1000, 127), (127, 1025)])
def test_scale_bytes_and_packed_order(rows, cols):
    torch = pytest.importorskip("torch")
    n = g.gemm_scale_bytes(rows, cols)
    assert n == max(1, -(-rows // 128)) * max(1, -(-cols // 512)) * 512
    byte = np.random.default_rng(rows + cols).integers(1, 255, (rows, -(-cols // 128)))
    packed = g.pack_scales(torch.from_numpy(byte.astype(np.uint8)))
    if cols > 0:
        assert packed.numel() == n
        assert np.array_equal(packed.numpy(), ref.pack(byte, cols))
        assert np.array_equal(g.unpack_scales(packed, rows, cols).numpy(), byte)


def test_sizes_out_of_range():
    assert g.gemm_scale_bytes(-1, 5) == -1 and g.gemm_scale_bytes(5, 2 ** 31) == -1
    assert g.gemm_route_rows(0, 4, 8) == 0
    assert g.gemm_route_rows(1, 4, 8) == 512  # four experts with one row each: 4 + 4 * 127
    assert g.gemm_route_rows(1000, 2, 8) == -(-(2000 + 8 * 127) // 128) * 128
    assert g.gemm_route_rows(-1, 1, 1) == -1 and g.gemm_route_rows(2 ** 30, 4, 8) == -1 and g.gemm_route_rows(1, 0, 1) == -1


OK = dict(M=64, N=96, K=200, A=0x100000, lda=208, SA=0x200000, a_type=4, B=0x300000, ldb=208, SB=0x400000, b_type=5,
          D=0x500000, ldd=96, d_type=0, alpha=1.0, beta=0.0, act=0)


def check(**change):
    return g.gemm_check_scaled(**{**OK, **change})


def test_accepts():
    assert check() == g.GEMM_OK
    assert check(d_type=2, beta=1.0, act=4, a_type=5, b_type=4) == g.GEMM_OK
    assert check(M=0, A=None, B=None, SA=None, SB=None, D=None) == g.GEMM_OK
    assert check(K=0, A=None, B=None, SA=None, SB=None) == g.GEMM_OK
    assert check(M=1, N=1, K=1, lda=16, ldb=16, ldd=8) == g.GEMM_OK
    assert check(A=0x100001, lda=201, B=0x300008, ldb=216) == g.GEMM_OK  # copied before they are read


@pytest.mark.parametrize("change", [
    {"M": -1}, {"N": -1}, {"K": -1}, {"a_type": 0}, {"b_type": 2}, {"a_type": 6}, {"d_type": 3}, {"d_type": 4}, {"act": 5},
    {"act": -1}, {"lda": 199}, {"ldb": 192}, {"ldd": 95}, {"D": None}, {"A": None}, {"B": None}, {"SA": None}, {"SB": None},
    {"D": 0x100000}, {"D": 0x300010}, {"D": 0x200000}, {"D": 0x400000 + 256},
    {"D": 0x100000 - 63 * 192 - 16},  # D's last row ends inside A
])
def test_invalid(change):
    assert check(**change) == g.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    {"D": 0x200000}, {"D": 0x200000 + 496}, {"D": 0x200000 - 16}, {"D": 0x400000}, {"D": 0x400000 + 496, "N": 8, "ldd": 8},
    {"D": 0x100000 + 192}, {"N": 1, "D": 0x400000 + 496}, {"N": 1, "D": 0x300000 + 192}, {"N": 1, "D": 0x100000}])
def test_one_row_over_an_operand(change):
    """One row of D against one run of bytes (scales, one row of an operand): neither has a pitch that means anything."""
    assert check(M=1, **change) == g.GEMM_ERR_INVALID_ARG


def test_one_row_beside_the_operands():
    for d in (0x200000 - 192, 0x200000 + 512, 0x400000 - 192, 0x400000 + 512, 0x100000 + 208):
        assert check(M=1, D=d) == g.GEMM_OK


@pytest.mark.parametrize("change", [{"SA": 0x200004}, {"SB": 0x400008}, {"D": 0x500008}, {"ldd": 100}])
def test_misaligned(change):
    assert check(**change) == g.GEMM_ERR_ALIGNMENT


@pytest.mark.parametrize("change", [{"M": 2 ** 31}, {"N": 2 ** 31, "ldd": 2 ** 32}, {"K": 2 ** 31, "lda": 2 ** 32, "ldb": 2 ** 32}])
def test_unsupported(change):
    assert check(**change) == g.GEMM_ERR_UNSUPPORTED


def test_calls_without_a_plan_are_refused():
    assert g.gemm_run_scaled(None, *[OK[n] for n in ("M", "N", "K", "A", "lda", "SA", "a_type", "B", "ldb", "SB", "b_type",
                                                     "D", "ldd", "d_type")], 1.0, 0.0) == g.GEMM_ERR_INVALID_ARG
    r = g.gemm_route_t(0, 2, 1, 1, 1, 0, 1.0)
    assert g.gemm_route(None, 1, 4, 16, 4, 2, None, r, 16, 16) == g.GEMM_ERR_INVALID_ARG
    assert g.gemm_route_map(None, 1, 2, 4, 16, 16, 16, 16, 16, 256) == g.GEMM_ERR_INVALID_ARG


def test_quantize_reference_is_the_nearest_code():
    """The reference's own pin: its values are codes, and no code lies nearer."""
    rng = np.random.default_rng(1)
    for fmt in ("e4m3", "e5m2"):
        codes = ref.decode(np.arange(256), fmt)
        codes = codes[np.isfinite(codes)]
        x = rng.standard_normal((3, 300)) * 10.0 ** rng.integers(-6, 6, (3, 1))
        v, byte = ref.quantize(x, fmt)
        y = x / np.repeat(2.0 ** (byte - 127.0), 128, axis=1)[:, :300]
        assert np.isin(np.abs(v), np.abs(codes)).all()
        assert np.allclose(np.abs(v - y), np.abs(codes[None, None] - y[..., None]).min(-1), rtol=0, atol=1e-12)
        top = ref.FORMATS[fmt][0]
        for b in range(3):
            m = np.abs(y[:, 128 * b:128 * b + 128]).max(1)
            assert (m <= top).all() and (m > top / 2).all()
