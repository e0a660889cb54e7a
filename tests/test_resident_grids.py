"""Launches of kernels that walk over rows are as large as what the device holds at once: a captured call's kernel nodes against
what the driver says of the same kernels (CTAs that fit an SM, with the node's threads and shared memory)."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    from dense_gemm_mma_gb300 import gemm
    return gemm


class KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS (cuda.h)
    _fields_ = [("func", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in ("gx", "gy", "gz", "bx", "by", "bz", "shared")] + [
        (n, ctypes.c_void_p) for n in ("params", "extra", "kern", "ctx")]


def launches(call):
    """[(CTAs, CTAs that fit an SM)] of the kernels that call(stream handle) launches, found by capturing it."""
    import torch
    cu = ctypes.CDLL("libcuda.so.1")
    ok = lambda status: status == 0 or pytest.fail(f"driver status {status}")  # noqa: E731
    stream, graph = torch.cuda.Stream(), ctypes.c_void_p()
    handle = ctypes.c_void_p(stream.cuda_stream)
    ok(cu.cuStreamBeginCapture_v2(handle, 1))  # 1: of this thread
    try:
        call(stream.cuda_stream)
    finally:
        ok(cu.cuStreamEndCapture(handle, ctypes.byref(graph)))
    n, out = ctypes.c_size_t(), []
    ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
    nodes = (ctypes.c_void_p * n.value)()
    ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
    for node in nodes:
        kind = ctypes.c_int()
        ok(cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)))
        if kind.value != 0:  # not a kernel
            continue
        p, func, fit = KernelNode(), ctypes.c_void_p(), ctypes.c_int()
        ok(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)))
        func.value = p.func
        if not func.value:
            ok(cu.cuKernelGetFunction(ctypes.byref(func), ctypes.c_void_p(p.kern)))
        ok(cu.cuOccupancyMaxActiveBlocksPerMultiprocessor(ctypes.byref(fit), func, p.bx * p.by * p.bz, ctypes.c_size_t(p.shared)))
        out.append((p.gx * p.gy * p.gz, fit.value))
    ok(cu.cuGraphDestroy(graph))
    return out


@pytest.mark.parametrize("x_name,h_name", [("float32", "float32"), ("bfloat16", "float32"), ("float16", "float16"), ("bfloat16", "bfloat16")])
@pytest.mark.parametrize("cols", [2050, 8192, 8193, 10001, 16384, 20000, 32768])
def test_norm_gradients(g, cols, x_name, h_name):
    import torch
    plan = g.Plan(0)
    rows, sms = 2000, torch.cuda.get_device_properties(0).multi_processor_count
    x, h = (torch.zeros((rows, cols), dtype=getattr(torch, n), device="cuda") for n in (x_name, h_name))
    rstd, dx, dgain = torch.zeros(rows, device="cuda"), torch.empty_like(h), torch.empty(cols, device="cuda")
    torch.cuda.synchronize()
    statuses = []
    got = launches(lambda s: statuses.append(plan.norm_backward(x, h, None, rstd, dx, dgain=dgain, stream=s)))
    assert statuses == [g.GEMM_OK]
    (ctas, fit), _ = got  # the rows' kernel, and the one that adds the gain's parts
    assert ctas == min(rows, sms * fit), (ctas, fit)
