"""A feed-forward block of experts with 8-bit products, forward and backward, on one GB300:

    python examples/experts_block.py [--tokens 4096] [--experts 32] [--top-k 4] [--hidden 1024] [--inner 2048]

    logits = x Wg^T          gemm_run (bf16 operands, fp32 result)
    choice, weights          gemm_route, order of the rows by expert: gemm_route_map
    x in expert order        gemm_quantize through the map
    p_e = x_e W1_e^T         gemm_run_grouped        h = SiLU(p), gemm_quantize
    y_e = h_e W2_e^T         gemm_run_grouped        out = sum of w y: gemm_combine

and back: gemm_combine_backward, gemm_run_grouped on the transposed weights, gemm_run_grouped_k
for the weights' gradients, gemm_combine for dx and gemm_route_backward for the logits.
What the backward pass needs of the activations is kept in 8 bits (the transposed copies that
gemm_quantize writes beside the forward's).  No row count leaves the device.

Prints how far each result is from the same block in 32 bits, and the time of a forward and of a
forward and backward pass.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dense_gemm_mma_gb300 import gemm  # noqa: E402

E4M3 = torch.float8_e4m3fn


def ok(status: int) -> None:
    if status != gemm.GEMM_OK:
        raise RuntimeError(gemm.gemm_status_string(status))


def padded(rows: int, cols: int, dtype) -> torch.Tensor:
    """rows x cols whose rows are whole multiples of 128 bytes apart (any multiple of 16 would do; these are read fastest)."""
    per = 128 // torch.empty((), dtype=dtype).element_size()
    return torch.zeros((rows, -(-cols // per) * per), dtype=dtype, device="cuda")[:, :cols]


class Codes:
    """A block-scaled 8-bit matrix (and, if asked for, its transpose)."""

    def __init__(self, plan, x, *, block_rows=1, transposed=False, rowmap=None, map_div=1):
        rows, cols = (x.shape[0] if rowmap is None else rowmap.numel()), x.shape[1]
        self.q, self.s = padded(rows, cols, E4M3), torch.empty(gemm.gemm_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        self.qt = self.st = None
        if transposed:
            self.qt, self.st = padded(cols, rows, E4M3), torch.empty(gemm.gemm_scale_bytes(cols, rows), dtype=torch.uint8, device="cuda")
        ok(plan.quantize(x, self.q, self.s, self.qt, self.st, block_rows=block_rows, rowmap=rowmap, map_div=map_div))


class Weights:
    """Experts' weights (experts x out x in) in 8 bits, 128 x 128 scales, as they stand and transposed."""

    def __init__(self, plan, w):
        both = [Codes(plan, e, block_rows=128, transposed=True) for e in w]
        self.q, self.s = torch.stack([c.q for c in both]), torch.stack([c.s for c in both])
        self.qt, self.st = torch.stack([c.qt for c in both]), torch.stack([c.st for c in both])


class Block:
    def __init__(self, plan, gate, w1, w2, top_k):
        self.plan, self.gate, self.top_k = plan, gate, top_k
        self.experts = w1.shape[0]
        self.w1, self.w2 = Weights(plan, w1), Weights(plan, w2)

    def forward(self, x, train=False):
        plan, E, k = self.plan, self.experts, self.top_k
        T, hidden = x.shape
        inner = self.w1.q.shape[1]
        rows = gemm.gemm_route_rows(T, k, E)
        ints = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        s = {"x": x, "logits": padded(T, E, torch.float32), "weights": torch.empty((T, k), device="cuda"),
             "indices": ints(T, k), "starts": ints(E), "counts": ints(E), "pos": ints(T, k), "rowmap": ints(rows)}
        ok(plan.run(x, self.gate, s["logits"], transB=True))
        ok(plan.route(s["logits"], s["weights"], s["indices"], renormalize=True))
        ok(plan.route_map(s["indices"], E, s["starts"], s["counts"], s["pos"], s["rowmap"]))
        s["xq"] = Codes(plan, x, rowmap=s["rowmap"], map_div=k, transposed=train)
        s["p"] = padded(rows, inner, torch.bfloat16)
        act = gemm.GEMM_ACT_NONE if train else gemm.GEMM_ACT_SILU  # the backward pass needs p itself
        ok(plan.run_grouped(s["xq"].q, s["xq"].s, self.w1.q, self.w1.s, s["p"], s["starts"], s["counts"], act=act))
        s["hq"] = Codes(plan, torch.nn.functional.silu(s["p"]) if train else s["p"], transposed=train)
        s["y"] = padded(rows, hidden, torch.bfloat16)
        ok(plan.run_grouped(s["hq"].q, s["hq"].s, self.w2.q, self.w2.s, s["y"], s["starts"], s["counts"]))
        out = torch.empty_like(x)
        ok(plan.combine(s["y"], s["pos"], s["weights"], out))
        return out, s

    def backward(self, s, dout):
        """Gradients of x (through the experts and the gate), W1, W2 and the logits."""
        plan, at = self.plan, (s["starts"], s["counts"])
        rows, hidden = s["y"].shape
        inner, E = s["p"].shape[1], self.experts
        dy, dweights = padded(rows, hidden, torch.bfloat16), torch.empty_like(s["weights"])
        ok(plan.combine_backward(dout, s["y"], s["pos"], s["weights"], dy, dweights, rowmap=s["rowmap"]))
        dyq = Codes(plan, dy, transposed=True)
        dw2 = torch.empty((E, hidden, inner), device="cuda")
        ok(plan.run_grouped_k(dyq.qt, dyq.st, s["hq"].qt, s["hq"].st, dw2, *at))
        dh = padded(rows, inner, torch.bfloat16)
        ok(plan.run_grouped(dyq.q, dyq.s, self.w2.qt, self.w2.st, dh, *at))
        sig = torch.sigmoid(s["p"].float())
        dpq = Codes(plan, (dh * (sig * (1 + s["p"] * (1 - sig)))).to(torch.bfloat16), transposed=True)
        dw1 = torch.empty((E, inner, hidden), device="cuda")
        ok(plan.run_grouped_k(dpq.qt, dpq.st, s["xq"].qt, s["xq"].st, dw1, *at))
        dxrows = padded(rows, hidden, torch.bfloat16)
        ok(plan.run_grouped(dpq.q, dpq.s, self.w1.qt, self.w1.st, dxrows, *at))
        dx = torch.empty_like(s["x"])
        ok(plan.combine(dxrows, s["pos"], torch.ones_like(s["weights"]), dx))
        dlogits = padded(*s["logits"].shape, torch.float32)
        ok(plan.route_backward(s["logits"], s["indices"], dweights, dlogits, renormalize=True))
        dx.add_((dlogits @ self.gate.float()).to(dx.dtype))
        return {"x": dx, "w1": dw1, "w2": dw2, "logits": dlogits}


def reference(x, gate, w1, w2, top_k, dout, choice):
    """The same block in 32 bits with autograd, the choice of experts given."""
    x, w1, w2 = (t.float().requires_grad_() for t in (x, w1, w2))
    logits = x @ gate.float().t()
    logits.retain_grad()
    w = torch.softmax(logits, 1).gather(1, choice)
    w = w / w.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, j = (choice == e).nonzero(as_tuple=True)
        y = torch.nn.functional.silu(x[t] @ w1[e].t()) @ w2[e].t()
        out = out.index_add(0, t, w[t, j, None] * y)
    out.backward(dout.float())
    return out.detach(), {"x": x.grad, "w1": w1.grad, "w2": w2.grad, "logits": logits.grad}


def off(got, want) -> float:
    return float((got.double() - want.double()).norm() / want.double().norm())


def compare(tokens=512, experts=8, top_k=2, hidden=256, inner=512, seed=0):
    """{name: relative error} of the block's results and gradients."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *n, by=1.0: (torch.randn(n, generator=g, device="cuda") * by).to(torch.bfloat16)  # noqa: E731
    x, gate = rand(tokens, hidden), rand(experts, hidden, by=hidden ** -0.5)
    w1, w2 = rand(experts, inner, hidden, by=hidden ** -0.5), rand(experts, hidden, inner, by=inner ** -0.5)
    dout = rand(tokens, hidden)
    plan = gemm.Plan(0)
    block = Block(plan, gate, w1, w2, top_k)
    out, s = block.forward(x, train=True)
    grads = block.backward(s, dout)
    serve, _ = block.forward(x)
    want, want_grads = reference(x, gate, w1, w2, top_k, dout, s["indices"].long())
    errors = {"out": off(out, want), "out (serving)": off(serve, want)}
    errors.update({"d" + n: off(grads[n], want_grads[n]) for n in grads})
    ok(plan.poll_error())
    return errors


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("experts", 32), ("top-k", 4), ("hidden", 1024), ("inner", 2048)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    for name, e in compare(a.tokens, a.experts, a.top_k, a.hidden, a.inner).items():
        print(f"{name:14s} off by {e:.3f} of its norm")
    plan = gemm.Plan(0)
    r = lambda *n: torch.randn(n, device="cuda", dtype=torch.bfloat16) * n[-1] ** -0.5  # noqa: E731
    block = Block(plan, r(a.experts, a.hidden), r(a.experts, a.inner, a.hidden), r(a.experts, a.hidden, a.inner), a.top_k)
    x = torch.randn((a.tokens, a.hidden), device="cuda", dtype=torch.bfloat16)
    steps = {"forward": lambda: block.forward(x), "forward + backward": lambda: block.backward(block.forward(x, train=True)[1], x)}
    for name, step in steps.items():
        for _ in range(3):
            step()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(10):
            step()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {start.elapsed_time(end) / 10:.3f} ms for {a.tokens} tokens")


if __name__ == "__main__":
    main()
