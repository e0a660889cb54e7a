"""A layer of experts behind a norm, on one GB300: training with 8-bit products, serving with 4-bit ones.

    python examples/experts_layer.py [--tokens 4096] [--experts 32] [--top-k 4] [--hidden 1024] [--inner 2048]

    h = x + residual, y = norm(h)     gemm_norm: one pass, h kept for the next layer and for the backward pass
    out = experts(y)                  the block of experts_block.py
    balance loss of the choice        gemm_balance

and back: gemm_balance_backward adds the loss's part to the logits' gradient, gemm_norm_backward takes the experts' gradient and
the one that reaches h past the norm.  Serving: the experts' weights in 4 bits (gemm_quantize_mx), the tokens quantised
through the router's map, gemm_run_grouped_mx twice; a projection behind it reads the norm's own 8-bit codes.

Prints how far each result is from the same layer in 32 bits (serving: from one with the same 4-bit weights), and times.
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
from dense_gemm_mma_gb300 import gemm  # noqa: E402

_spec = importlib.util.spec_from_file_location("experts_block", os.path.join(ROOT, "examples", "experts_block.py"))
block = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(block)
ok, padded, off = block.ok, block.padded, block.off
EPS = 1e-6


class Codes4:
    """A block-scaled 4-bit matrix."""

    def __init__(self, plan, x, *, rowmap=None, map_div=1):
        rows, cols = (x.shape[0] if rowmap is None else rowmap.numel()), x.shape[1]
        self.q = padded(rows, (cols + 1) // 2, torch.uint8)
        self.s = torch.empty(gemm.gemm_mx_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        ok(plan.quantize_mx4(x, self.q, self.s, rowmap=rowmap, map_div=map_div))


class Weights4:
    """Experts' weights (experts x out x in) in 4 bits."""

    def __init__(self, plan, w):
        each = [Codes4(plan, e) for e in w]
        self.q, self.s = torch.stack([c.q for c in each]), torch.stack([c.s for c in each])
        self.cols = w.shape[2]

    def values(self, plan):
        """What they stand for (experts x out x in, bf16): operands for gemm_run."""
        out = torch.empty((*self.q.shape[:2], self.cols), dtype=torch.bfloat16, device="cuda")
        for q, s, v in zip(self.q, self.s, out):
            ok(plan.dequantize(q, s, v))
        return out


class Layer:
    def __init__(self, plan, gain, gate, w1, w2, top_k, balance=0.01):
        self.plan, self.gain, self.balance = plan, gain, balance
        self.experts = block.Block(plan, gate, w1, w2, top_k)
        self.w1, self.w2 = Weights4(plan, w1), Weights4(plan, w2)

    def norm(self, x, residual):
        s = {"h": torch.empty_like(x), "y": torch.empty_like(x), "rstd": torch.empty(x.shape[0], device="cuda")}
        ok(self.plan.norm(x, self.gain, Y=s["y"], residual=residual, H=s["h"], rstd=s["rstd"], eps=EPS))
        return s

    def forward(self, x, residual):
        """(out, balance loss, what the backward pass needs)."""
        E = self.experts.experts
        s = self.norm(x, residual)
        out, s["block"] = self.experts.forward(s["y"], train=True)
        s["loss"], s["factor"], s["shares"] = (torch.empty(n, device="cuda") for n in (1, E, E))
        s["load"] = torch.empty(E, dtype=torch.int32, device="cuda")
        ok(self.plan.balance(s["block"]["logits"], s["block"]["indices"], s["load"], s["shares"], s["factor"], s["loss"],
                             scale=self.balance))
        return out, s["loss"], s

    def backward(self, s, dout, dh):
        """Gradients of x (and of the residual: the same), the gain, W1, W2 and the logits, from those of out, of h past the norm
        (dh) and of the balance loss (1)."""
        b = s["block"]
        grads = self.experts.backward(b, dout)
        dbalance = padded(*b["logits"].shape, torch.float32)
        ok(self.plan.balance_backward(b["logits"], b["indices"], s["factor"], dbalance))
        dy = grads["x"].add_((dbalance @ self.experts.gate.float()).to(dout.dtype))
        dlogits = grads["logits"].clone()
        ok(self.plan.balance_backward(b["logits"], b["indices"], s["factor"], dlogits, accumulate=True))
        dx, dgain = torch.empty_like(dout), torch.empty(dout.shape[1], device="cuda")
        ok(self.plan.norm_backward(dy, s["h"], self.gain, s["rstd"], dx, dgain=dgain, dH=dh))
        return {"x": dx, "gain": dgain, "w1": grads["w1"], "w2": grads["w2"], "logits": dlogits}

    def serve(self, x, residual):
        """(out, h) with 4-bit products."""
        plan, E, k = self.plan, self.experts.experts, self.experts.top_k
        s = self.norm(x, residual)
        T, hidden = x.shape
        rows, inner = gemm.gemm_route_rows(T, k, E), self.w1.q.shape[1]
        ints = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        logits, weights = padded(T, E, torch.float32), torch.empty((T, k), device="cuda")
        indices, starts, counts, pos, rowmap = ints(T, k), ints(E), ints(E), ints(T, k), ints(rows)
        ok(plan.run(s["y"], self.experts.gate, logits, transB=True))
        ok(plan.route(logits, weights, indices, renormalize=True))
        ok(plan.route_map(indices, E, starts, counts, pos, rowmap))
        xq = Codes4(plan, s["y"], rowmap=rowmap, map_div=k)
        p, y, out = padded(rows, inner, torch.bfloat16), padded(rows, hidden, torch.bfloat16), torch.empty_like(x)
        ok(plan.run_grouped_mx4(xq.q, xq.s, self.w1.q, self.w1.s, p, starts, counts, K=hidden, act=gemm.GEMM_ACT_SILU))
        hq = Codes4(plan, p)
        ok(plan.run_grouped_mx4(hq.q, hq.s, self.w2.q, self.w2.s, y, starts, counts, K=inner))
        ok(plan.combine(y, pos, weights, out))
        return out, s["h"], indices

    def project(self, x, residual, w):
        """W norm(x + residual) from the norm's own 8-bit codes, h kept."""
        (T, hidden), n = x.shape, w.shape[0]
        q, s = padded(T, hidden, block.E4M3), torch.empty(gemm.gemm_scale_bytes(T, hidden), dtype=torch.uint8, device="cuda")
        h, out = torch.empty_like(x), padded(T, n, torch.bfloat16)
        wq = block.Codes(self.plan, w, block_rows=128)
        ok(self.plan.norm(x, self.gain, Q=q, SQ=s, residual=residual, H=h, eps=EPS))
        ok(self.plan.run_scaled(q, s, wq.q, wq.s, out))
        return out, h


def normed(h, gain):
    return h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * gain


def loss_of(logits, choice, scale):
    E = logits.shape[1]
    load = torch.bincount(choice.reshape(-1), minlength=E).float() / choice.numel()
    return scale * E * (load * torch.softmax(logits, 1).mean(0)).sum()


def experts_of(y, gate, w1, w2, choice):
    """(out, logits) of the experts in 32 bits, the choice given."""
    logits = y @ gate.float().t()
    w = torch.softmax(logits, 1).gather(1, choice)
    w = w / w.sum(1, keepdim=True)
    out = torch.zeros_like(y)
    for e in range(w1.shape[0]):
        t, j = (choice == e).nonzero(as_tuple=True)
        out = out.index_add(0, t, w[t, j, None] * (torch.nn.functional.silu(y[t] @ w1[e].t()) @ w2[e].t()))
    return out, logits


def make(tokens, experts, top_k, hidden, inner, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *n, by=1.0: (torch.randn(n, generator=g, device="cuda") * by).to(torch.bfloat16)  # noqa: E731
    gain = (1 + 0.2 * rand(hidden)).to(torch.bfloat16)
    gate, w1, w2 = rand(experts, hidden, by=hidden ** -0.5), rand(experts, inner, hidden, by=hidden ** -0.5), rand(experts, hidden, inner, by=inner ** -0.5)
    plan = gemm.Plan(0)
    return Layer(plan, gain, gate, w1, w2, top_k), w1, w2, rand


def compare(tokens=512, experts=8, top_k=2, hidden=256, inner=512, seed=0):
    """{name: relative error} of the layer's results and gradients."""
    layer, w1, w2, rand = make(tokens, experts, top_k, hidden, inner, seed)
    plan, gate = layer.plan, layer.experts.gate
    x, residual, dout, dh, proj = rand(tokens, hidden), rand(tokens, hidden), rand(tokens, hidden), rand(tokens, hidden), rand(264, hidden, by=hidden ** -0.5)
    out, loss, s = layer.forward(x, residual)
    grads = layer.backward(s, dout, dh)
    choice = s["block"]["indices"].long()
    fx, fgain, fw1, fw2 = (t.float().requires_grad_() for t in (x, layer.gain, w1, w2))
    h = fx + residual.float()
    want, logits = experts_of(normed(h, fgain), gate, fw1, fw2, choice)
    logits.retain_grad()
    want_loss = loss_of(logits, choice, layer.balance)
    ((want * dout.float()).sum() + (h * dh.float()).sum() + want_loss).backward()
    errors = {"h": off(s["h"], h.detach()), "y": off(s["y"], normed(h, fgain).detach()), "out": off(out, want.detach()), "loss": off(loss, want_loss.detach()[None]),
              "dx": off(grads["x"], fx.grad), "dgain": off(grads["gain"], fgain.grad), "dw1": off(grads["w1"], fw1.grad),
              "dw2": off(grads["w2"], fw2.grad), "dlogits": off(grads["logits"], logits.grad)}
    with torch.no_grad():
        served, hs, chosen = layer.serve(x, residual)
        same, _ = experts_of(normed(h, fgain), gate, layer.w1.values(plan).float(), layer.w2.values(plan).float(), chosen.long())
        projected, hp = layer.project(x, residual, proj)
        errors.update({"out (4 bits)": off(served, same), "projection": off(projected, normed(h, fgain) @ proj.float().t())})
        if not (torch.equal(hs, s["h"]) and torch.equal(hp, s["h"])):
            raise RuntimeError("the sums differ")
    ok(plan.poll_error())
    return errors


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("experts", 32), ("top-k", 4), ("hidden", 1024), ("inner", 2048)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    for name, e in compare(a.tokens, a.experts, a.top_k, a.hidden, a.inner).items():
        print(f"{name:14s} off by {e:.4f} of its norm")
    layer, _, _, rand = make(a.tokens, a.experts, a.top_k, a.hidden, a.inner)
    x, r = rand(a.tokens, a.hidden), rand(a.tokens, a.hidden)
    steps = {"forward + backward": lambda: layer.backward(layer.forward(x, r)[2], x, r), "serving, 4 bits": lambda: layer.serve(x, r)}
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
