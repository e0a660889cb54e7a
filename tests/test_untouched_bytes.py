"""What lies between and around the rows of the 4-bit quantiser's results, of the values of codes and of the norm's results keeps
every byte: buffers are compared outside the rows, byte by byte, after calls at any address and row distance."""
import numpy as np
import pytest

from tests import more_ref as ref
from tests.test_mx4_gpu import g, plan, same, scale_room  # noqa: F401  (g, plan: fixtures)

pytestmark = pytest.mark.gpu


def room(rows, width, gap, off, dtype):
    """(buffer, rows x width view `off` values into it with rows `gap` values apart, which bytes of the buffer are none of the
    view's); the buffer has a gap behind its last row too."""
    import torch
    size = torch.empty((), dtype=dtype).element_size()
    buf = torch.full(((off + rows * (width + gap) + 64) * size,), 0xA5, dtype=torch.uint8, device="cuda")
    outside = torch.ones(buf.numel() // size, dtype=torch.bool, device="cuda")
    outside.as_strided((rows, width), (width + gap, 1), off).fill_(False)
    return buf, buf.view(dtype).as_strided((rows, width), (width + gap, 1), off), outside.repeat_interleave(size)


def test_the_check_sees_a_stray_byte():
    """A code byte that is 0xA5 by chance hides nothing; a changed byte outside the rows shows."""
    import torch
    buf, view, outside = room(5, 7, 3, 2, torch.uint8)
    view.fill_(0x11)
    assert (buf[outside] == 0xA5).all() and int(outside.sum()) == buf.numel() - 35
    for at in (1, 2 + 7, 2 + 4 * 10 + 7, buf.numel() - 1):
        hurt = buf.clone()
        hurt[at] = 0
        assert not (hurt[outside] == 0xA5).all()


@pytest.mark.parametrize("off,gap", [(0, 1), (4, 4), (1, 0), (3, 2), (8, 8), (5, 11), (0, 0)])
@pytest.mark.parametrize("R,K", [(40, 533), (130, 256), (33, 31), (129, 2050), (2500, 2699)])
@pytest.mark.parametrize("name", ["bfloat16", "float32"])
def test_quantizer(plan, g, off, gap, R, K, name):  # noqa: F811
    import torch
    x = torch.randn((R, K), device="cuda").to(getattr(torch, name))
    rowmap = torch.randperm(R, device="cuda").to(torch.int32)
    rowmap[:: 9] = -1
    for both in (0, 1, 2):  # as it stands, both, transposed
        for by in (None, rowmap):
            buf, q, out = room(R, (K + 1) // 2, gap, off, torch.uint8)
            tbuf, qt, tout = room(K, (R + 1) // 2, gap, off, torch.uint8)
            sbuf, stbuf = (torch.full((g.gemm_mx_scale_bytes(*n) + 256,), 0xA5, dtype=torch.uint8, device="cuda") for n in ((R, K), (K, R)))
            args = [(q, sbuf[128:-128]) if both < 2 else (None, None), (qt, stbuf[128:-128]) if both else (None, None)]
            assert plan.quantize_mx4(x, *args[0], *args[1], rowmap=by) == g.GEMM_OK
            if both == 2:
                assert (buf == 0xA5).all() and (sbuf == 0xA5).all()
            if both == 0:
                assert (tbuf == 0xA5).all() and (stbuf == 0xA5).all()
            assert (buf[out] == 0xA5).all() and (tbuf[tout] == 0xA5).all()
            for s in (sbuf, stbuf):
                assert (s[:128] == 0xA5).all() and (s[-128:] == 0xA5).all()
            if by is not None and both < 2:
                assert (q[by < 0] == 0xA5).all()  # rows without a source
    assert plan.poll_error() == g.GEMM_OK


@pytest.mark.parametrize("off,gap", [(0, 1), (4, 4), (1, 0), (3, 2), (8, 8)])
@pytest.mark.parametrize("R,K", [(40, 533), (5, 31), (3, 2050)])
@pytest.mark.parametrize("name", ["bfloat16", "float16", "float32"])
def test_values(plan, g, off, gap, R, K, name):  # noqa: F811
    import torch
    codes = torch.randint(0, 256, (R, (K + 1) // 2), dtype=torch.uint8, device="cuda")
    codes8 = torch.randint(0, 127, (R, K), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    for q, n in ((codes, g.gemm_mx_scale_bytes(R, K)), (codes8, g.gemm_scale_bytes(R, K))):
        s = torch.full((n,), 127, dtype=torch.uint8, device="cuda")
        buf, x, out = room(R, K, gap, off, getattr(torch, name))
        assert plan.dequantize(q, s, x) == g.GEMM_OK
        assert (buf[out] == 0xA5).all()
        want = torch.empty((R, K), device="cuda")
        assert plan.dequantize(q, s, want) == g.GEMM_OK
        assert torch.equal(x.float(), want)  # (scales of 1: every value is one of each type's)
    assert plan.poll_error() == g.GEMM_OK


@pytest.mark.parametrize("off,gap", [(0, 1), (4, 4), (1, 0), (3, 2), (8, 8)])
@pytest.mark.parametrize("R,N", [(1, 7), (5, 513), (33, 2050), (3, 9001)])
@pytest.mark.parametrize("x_name,h_name", [("bfloat16", "bfloat16"), ("float16", "float32"), ("float32", "float32")])
def test_norm(plan, g, off, gap, R, N, x_name, h_name):  # noqa: F811
    import torch
    xt, ht = getattr(torch, x_name), getattr(torch, h_name)
    _, x, _ = room(R, N, gap, off, xt)
    _, r, _ = room(R, N, gap, off, ht)
    x.normal_(), r.normal_()
    ybuf, y, yout = room(R, N, gap, off, xt)
    hbuf, h, hout = room(R, N, gap, off, ht)
    rbuf, rstd, rout = room(1, R, 0, 1, torch.float32)
    assert plan.norm(x, Y=y, residual=r, H=h, rstd=rstd[0]) == g.GEMM_OK
    dbuf, dx, dout = room(R, N, gap, off, ht)
    gbuf, dgain, gout = room(1, N, 0, 1, torch.float32)
    assert plan.norm_backward(y, h, None, rstd[0], dx, dgain=dgain[0], dH=r) == g.GEMM_OK
    for buf, out in ((ybuf, yout), (hbuf, hout), (rbuf, rout), (dbuf, dout), (gbuf, gout)):
        assert (buf[out] == 0xA5).all()
    assert plan.poll_error() == g.GEMM_OK


@pytest.mark.parametrize("R,N", [(1, 16), (5, 513), (130, 2050)])
def test_norm_into_codes(plan, g, R, N):  # noqa: F811
    import torch
    x = torch.randn((R, N), device="cuda", dtype=torch.bfloat16)
    ld = -(-N // 16) * 16
    for gap in (ld - N, ld - N + 32):  # (rows of codes are on 16-byte boundaries)
        buf, q, out = room(R, N, gap, 16, torch.uint8)
        sbuf = torch.full((g.gemm_scale_bytes(R, N) + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        assert plan.norm(x, Q=q.view(torch.float8_e4m3fn), SQ=sbuf[128:-128]) == g.GEMM_OK
        assert (buf[out] == 0xA5).all() and (sbuf[:128] == 0xA5).all() and (sbuf[-128:] == 0xA5).all()


def test_codes_at_any_address_are_the_nearest(plan, g):  # noqa: F811
    """The rows themselves, at the same addresses: against 64 bits."""
    import torch
    R, K = 33, 531
    x = torch.randn((R, K), device="cuda", dtype=torch.bfloat16)
    want, byte = ref.quantize4(x.double().cpu().numpy())
    want_t, byte_t = ref.quantize4(x.double().cpu().numpy().T)
    for off, gap in ((5, 11), (2, 0), (3, 3)):
        _, q, _ = room(R, (K + 1) // 2, gap, off, torch.uint8)
        _, qt, _ = room(K, (R + 1) // 2, gap, off, torch.uint8)
        s, st = scale_room(g, R, K), scale_room(g, K, R)
        assert plan.quantize_mx4(x, q, s, qt, st) == g.GEMM_OK
        same(ref.decode4(q.cpu().numpy(), K), want)
        same(ref.decode4(qt.cpu().numpy(), R), want_t)
        assert np.array_equal(s.cpu().numpy(), ref.pack_scales4(byte, K)) and np.array_equal(st.cpu().numpy(), ref.pack_scales4(byte_t, R))
