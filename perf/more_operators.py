"""What the norm with the residual's addition, the balance loss of a router and the 4-bit products are measured on.

Five operators (include/gemm.h):

  norm       root-mean-square norm of x + residual, into 16 or 32 bits or into 8-bit codes with scales; with its gradients
  balance    how evenly a router spreads its tokens: counts, shares, loss; with the gradient of the logits
  quantize4  matrix -> 4-bit values (E2M1) with a power-of-two scale for each block of 32, and its transpose
  product4   D = A @ B^T of two such matrices
  experts4   the same product for each expert's rows

Codes are returned as the values that they stand for. `run` computes everything with elementary torch operations in 32 bits,
or, where `own` is true, with this package.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes by code; bit 3 is the sign


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token between two layers: the residual's addition and the norm, latency
        {"name": "norm_one_token", "op": "norm", "R": 1, "N": 4096, "x": "bf16", "form": "plain"},
        # a prompt's activations on their way into an 8-bit product
        {"name": "norm_prompt_codes", "op": "norm", "R": 8192, "N": 4096, "x": "bf16", "form": "codes"},
        # a training batch: the norm and its gradients (activations, residual and gain), ragged
        {"name": "norm_train", "op": "norm", "R": 6912, "N": 2050, "x": "bf16", "form": "train"},
        # the loads of one decoded batch, looked at by a server that places experts
        {"name": "balance_decode", "op": "balance", "T": 16, "E": 256, "k": 8, "score": "sigmoid", "grad": False},
        # a training batch's balance loss and what it adds to the logits' gradient; a tenth of the tokens is padding
        {"name": "balance_train", "op": "balance", "T": 16384, "E": 128, "k": 8, "score": "softmax", "grad": True},
        # a decoded batch on its way into a 4-bit product
        {"name": "quantize4_decode", "op": "quantize4", "R": 33, "K": 2050, "x": "bf16", "both": False},
        # a layer's activations, kept in 4 bits for the product and, transposed, for the backward pass
        {"name": "quantize4_activations", "op": "quantize4", "R": 8192, "K": 4096, "x": "bf16", "both": True},
        # one token through a square projection: latency and the weights' bytes
        {"name": "product4_one_token", "op": "product4", "M": 1, "N": 4096, "K": 4096, "out": "bf16", "act": "none"},
        # a long prompt through a large projection: the benchmark's square size
        {"name": "product4_prompt", "op": "product4", "M": 8192, "N": 8192, "K": 8192, "out": "bf16", "act": "none"},
        # a ragged batch through an up-projection with its activation, odd K
        {"name": "product4_ragged", "op": "product4", "M": 2304, "N": 6920, "K": 2051, "out": "f16", "act": "silu"},
        # single tokens through experts: every chosen expert's weights are read for a few rows
        {"name": "experts4_decode", "op": "experts4", "T": 48, "k": 4, "E": 64, "N": 2048, "K": 2048, "out": "bf16"},
        # a prompt through experts, uneven loads
        {"name": "experts4_prompt", "op": "experts4", "T": 8192, "k": 4, "E": 32, "N": 4096, "K": 2048, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "balance", "quantize4", "product4", "product4", "experts4"])
    if op == "norm":
        return {"op": op, "R": _log(rng, 1, 8192), "N": _log(rng, 512, 8192), "x": rng.choice(["bf16", "bf16", "f16", "f32"]), "form": rng.choice(["plain", "codes", "train"])}
    if op == "balance":
        return {"op": op, "T": _log(rng, 1, 16384), "E": rng.choice([8, 16, 60, 64, 128, 160, 256]), "k": rng.randint(1, 8), "score": rng.choice(["softmax", "sigmoid"]), "grad": rng.random() < 0.5}
    if op == "quantize4":
        return {"op": op, "R": _log(rng, 1, 8192), "K": _log(rng, 512, 8192), "x": rng.choice(["bf16", "f16", "f32"]), "both": rng.random() < 0.5}
    if op == "product4":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 512, 8192), "K": _log(rng, 512, 8192), "out": rng.choice(["bf16", "f16", "f32"]), "act": rng.choice(["none", "silu"])}
    return {"op": op, "T": _log(rng, 1, 8192), "k": rng.choice([1, 2, 4]), "E": rng.choice([8, 16, 32, 48, 64]), "N": 8 * _log(rng, 64, 256), "K": 8 * _log(rng, 64, 256), "out": "bf16"}


# ------------------------------------------------------------------ inputs

def _up(n, to):
    return -(-n // to) * to


def _rows(n, width, dtype, like=torch.empty):
    """n rows of `width` values, each row on a 16-byte boundary."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return like((n, _up(max(width, 1), per)), dtype=dtype, device="cuda")[:, :width]


def _normal(g, n, width, dtype):
    """Activations: normal, with a few channels a hundred times larger than the others."""
    x = torch.randn((n, width), generator=g, device="cuda")
    loud = 1 + 99 * (torch.rand((1, width), generator=g, device="cuda") < 0.002)
    out = _rows(n, width, dtype)
    out.copy_(x * loud * 0.5)
    return out


def _bytes(n):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _scale_room(rows, cols, block):
    """Packed scale bytes: tiles of 128 rows x 4 blocks."""
    return _bytes(512 * max(1, -(-rows // 128)) * max(1, -(-cols // (4 * block))))


def _pack(b):
    """Scale bytes, one for each row and block, in the packed order: tiles of 128 rows x 4 blocks, each as 32 lines of 16 bytes; row
    r, block c of a tile is byte (r % 32) * 16 + (r // 32) * 4 + c. What is beyond the matrix is 0."""
    rows, blocks = b.shape
    R, C = _up(max(rows, 1), 128), _up(max(blocks, 1), 4)
    full = torch.zeros((R, C), dtype=torch.uint8, device=b.device)
    full[:rows, :blocks] = b
    return full.view(R // 128, 4, 32, C // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _codes4(g, rows, K):
    """A 4-bit matrix and its scales, as a quantiser leaves them: values up to the largest, scales around 2^-3; two codes to a byte,
    the even column's in the low four bits."""
    v = torch.randn((rows, _up(K, 2)), generator=g, device="cuda") * 2
    v[:, K:] = 0
    edges = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device="cuda")
    code = torch.bucketize(v.abs(), edges).to(torch.uint8) | (v < 0).to(torch.uint8) << 3
    q = _rows(rows, _up(K, 2) // 2, torch.uint8)
    q.copy_(code[:, ::2] | code[:, 1::2] << 4)
    spread = torch.randint(-5, 0, (rows, -(-K // 32)), generator=g, device="cuda")
    return q, _pack((spread + 127).to(torch.uint8))


def _segments(g, T, k, E):
    """An uneven choice of k different experts for each token, and the order of its rows: expert e has `counts[e]` rows from
    `starts[e]`, a multiple of 128."""
    liking = torch.randn((1, E), generator=g, device="cuda") * 0.5
    chosen = torch.topk(liking + torch.randn((T, E), generator=g, device="cuda"), min(k, E), dim=1).indices
    counts = torch.bincount(chosen.reshape(-1), minlength=E)
    padded = (counts + 127) // 128 * 128
    return (padded.cumsum(0) - padded).to(torch.int32), counts.to(torch.int32), _up(T * k + 127 * min(E, T * k), 128)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 6151 + 29)
    s, op = {"case": case}, case["op"]
    if op == "norm":
        R, N, t = case["R"], case["N"], TYPES[case["x"]]
        s["X"], s["residual"] = _normal(g, R, N, t), _normal(g, R, N, t)
        s["gain"] = (1 + 0.2 * torch.randn(N, generator=g, device="cuda")).to(t)
        s["H"], s["rstd"] = _rows(R, N, t), torch.empty(R, device="cuda")
        if case["form"] == "codes":
            s["Q"], s["SQ"] = _rows(R, N, torch.float8_e4m3fn), _scale_room(R, N, 128)
            s["V"] = _rows(R, N, torch.bfloat16)
        else:
            s["Y"] = _rows(R, N, t)
        if case["form"] == "train":
            s["dY"], s["dH"] = _normal(g, R, N, t), _normal(g, R, N, t)
            s["dX"], s["dgain"] = _rows(R, N, t), torch.empty(N, device="cuda")
    elif op == "balance":
        T, E, k = case["T"], case["E"], min(case["k"], case["E"])
        s["logits"] = torch.randn((T, E), generator=g, device="cuda") * 1.5 + torch.randn((1, E), generator=g, device="cuda") * 0.5
        chosen = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
        padding = torch.rand((T, 1), generator=g, device="cuda") < (0.1 if T > 1 else 0.0)
        s["indices"] = torch.where(padding, -1, chosen)
        s["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        s["shares"], s["factor"], s["loss"] = (torch.empty(n, device="cuda") for n in (E, E, 1))
        if case["grad"]:
            s["dloss"], s["dlogits"] = torch.rand(1, generator=g, device="cuda") + 0.5, torch.empty((T, E), device="cuda")
    elif op == "quantize4":
        R, K = case["R"], case["K"]
        s["X"] = _normal(g, R, K, TYPES[case["x"]])
        s["Q"], s["SQ"], s["V"] = _rows(R, -(-K // 2), torch.uint8), _scale_room(R, K, 32), _rows(R, K, torch.bfloat16)
        if case["both"]:
            s["QT"], s["SQT"], s["VT"] = _rows(K, -(-R // 2), torch.uint8), _scale_room(K, R, 32), _rows(K, R, torch.bfloat16)
    elif op == "product4":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["SA"] = _codes4(g, M, K)
        s["B"], s["SB"] = _codes4(g, N, K)
        s["D"] = _rows(M, N, TYPES[case["out"]])
    else:
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        s["starts"], s["counts"], rows = _segments(g, T, k, E)
        s["A"], s["SA"] = _codes4(g, rows, K)
        B = [_codes4(g, N, K) for _ in range(E)]
        s["B"], s["SB"] = torch.stack([b for b, _ in B]), torch.stack([c for _, c in B])
        s["D"] = _rows(rows, N, TYPES[case["out"]], torch.zeros)
        s["most"] = int(s["counts"].max())  # rows of the fullest expert, for the plain form's batch
    return s


# -------------------------------------------------------------- plain forms

def _scales(packed, rows, cols, block):
    """Scales of a rows x cols matrix, one for each value, in 32 bits."""
    R, C = _up(max(rows, 1), 128), _up(max(-(-cols // block), 1), 4)
    b = packed.view(R // 128, C // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R, C)[:rows].int()
    two = torch.where(b == 0, 1 << 22, b << 23).view(torch.float32)  # 2^(b - 127)
    return two.repeat_interleave(block, 1)[:, :cols]


def _values4(q, packed, K):
    """Values of a 4-bit matrix of K columns in 32 bits."""
    code = torch.stack((q & 15, q >> 4), 2).flatten(1)[:, :K].long()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    return table[code] * _scales(packed, q.shape[0], K, 32)


def _up_scale(most, top):
    """The least e, -127 at least, with most <= 1.5 or 1.75 (by the fraction of `top`) * 2^(e + the exponent of `top`)."""
    m, e = torch.frexp(most)
    half, exponent = math.frexp(top)
    return torch.where(most > 0, (e - exponent + (m > half)).clamp(min=-127), -127).to(torch.int32)


def _blocks(x, block):
    """Largest magnitude of each row's blocks."""
    R, K = x.shape
    return torch.nn.functional.pad(x.abs(), (0, -K % block)).view(R, -1, block).amax(2)


def _down(e, block, K):
    return ((127 - e) << 23).view(torch.float32).repeat_interleave(block, 1)[:, :K]  # 2^-e


def _two_to(e, block, K):
    return torch.where(e == -127, 1 << 22, (e + 127) << 23).view(torch.float32).repeat_interleave(block, 1)[:, :K]


def _quantized8(x):
    """The values that x has in 8 bits (E4M3, blocks of 128)."""
    e = _up_scale(_blocks(x, 128), 448.0)
    return ((x * _down(e, 128, x.shape[1])).to(torch.float8_e4m3fn).float() * _two_to(e, 128, x.shape[1])).to(torch.bfloat16)


def _quantized4(x):
    """The values that x has in 4 bits (E2M1, blocks of 32), and its packed scales."""
    K = x.shape[1]
    e = _up_scale(_blocks(x, 32), 6.0)
    v = x * _down(e, 32, K)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    near = torch.copysign(torch.round(a / step) * step, v)  # (ties to the even multiple of the step: the even code)
    return (near * _two_to(e, 32, K)).to(torch.bfloat16), _pack((e + 127).to(torch.uint8))


def _plain_norm(s):
    case = s["case"]
    t, gain = TYPES[case["x"]], s["gain"].float()
    h = s["X"].float() + s["residual"].float()
    rstd = 1 / torch.sqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * gain
    got = {"H": h.to(t)}
    if case["form"] == "codes":
        return {**got, "V": _quantized8(y)}
    got["Y"] = y.to(t)
    if case["form"] == "train":
        xhat, dy = got["H"].float() * rstd[:, None], s["dY"].float()
        g = dy * gain
        got["dX"] = (rstd[:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True)) + s["dH"].float()).to(t)
        got["dgain"], got["rstd"] = (dy * xhat).sum(0), rstd
    return got


def _plain_balance(s):
    case, x, index = s["case"], s["logits"], s["indices"].long()
    E = case["E"]
    valid = (index >= 0) & (index < E)
    live = valid.any(1, keepdim=True)
    counts = (torch.where(valid, index, E).reshape(-1)[:, None] == torch.arange(E, device=x.device)).sum(0)
    s1 = 1 / (1 + torch.exp(-x)) if case["score"] == "sigmoid" else torch.exp(x - x.amax(1, keepdim=True))
    p = s1 / s1.sum(1, keepdim=True)
    m, n = live.sum().clamp(min=1), counts.sum().clamp(min=1)
    shares = torch.where(live, p, 0).sum(0) / m
    factor = E * counts.float() / n / m
    got = {"counts": counts.to(torch.int32), "shares": shares, "factor": factor, "loss": (E * counts.float() / n * shares).sum()[None]}
    if case["grad"]:
        d = p * (factor - (factor * p).sum(1, keepdim=True))
        if case["score"] == "sigmoid":
            d = d * (1 - s1)
        got["dlogits"] = torch.where(live, s["dloss"] * d, 0)
    return got


def _plain_quantize4(s):
    x = s["X"].float()
    got = dict(zip(("V", "SQ"), _quantized4(x)))
    if s["case"]["both"]:
        got.update(zip(("VT", "SQT"), _quantized4(x.t())))
    return got


def _plain_product4(s):
    K = s["case"]["K"]
    y = _values4(s["A"], s["SA"], K) @ _values4(s["B"], s["SB"], K).t()
    return (y / (1 + torch.exp(-y)) if s["case"]["act"] == "silu" else y).to(s["D"].dtype)


def _plain_experts4(s):
    case = s["case"]
    E, N, K = case["E"], case["N"], case["K"]
    at = torch.arange(s["most"], device="cuda")
    held = at < s["counts"][:, None]
    rows = torch.where(held, s["starts"][:, None] + at, 0).long()
    x = _values4(s["A"], s["SA"], K)[rows]
    R, C = _up(N, 128), _up(-(-K // 32), 4)  # each expert's scales are whole tiles
    scale = _scales(s["SB"].reshape(-1), E * R, 32 * C, 32).view(E, R, 32 * C)[:, :N, :K]
    code = torch.stack((s["B"] & 15, s["B"] >> 4), 3).flatten(2)[..., :K].long()
    w = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")[code] * scale
    out = torch.zeros((s["A"].shape[0], N), device="cuda")
    out[rows[held]] = torch.bmm(x, w.transpose(1, 2))[held]
    return out.to(s["D"].dtype)


# ---------------------------------------------------------------- this package

_plans = []


def _plan():
    if not _plans:
        from dense_gemm_mma_gb300 import gemm
        _plans.extend([gemm.Plan(0), gemm])
    return _plans


def _done(status):
    if status:
        raise RuntimeError("status %d" % status)


def _own(s):
    case, op = s["case"], s["case"]["op"]
    plan, gemm = _plan()
    if op == "norm":
        _done(plan.norm(s["X"], s["gain"], Y=s.get("Y"), Q=s.get("Q"), SQ=s.get("SQ"), residual=s["residual"], H=s["H"], rstd=s["rstd"], eps=EPS))
        if case["form"] == "codes":
            _done(plan.dequantize(s["Q"], s["SQ"], s["V"]))
            return {"H": s["H"], "V": s["V"]}
        if case["form"] == "train":
            _done(plan.norm_backward(s["dY"], s["H"], s["gain"], s["rstd"], s["dX"], dgain=s["dgain"], dH=s["dH"]))
        return {n: s[n] for n in (("H", "Y", "dX", "dgain", "rstd") if case["form"] == "train" else ("H", "Y"))}
    if op == "balance":
        score = gemm.GEMM_SCORE_SIGMOID if case["score"] == "sigmoid" else gemm.GEMM_SCORE_SOFTMAX
        _done(plan.balance(s["logits"], s["indices"], s["counts"], s["shares"], s["factor"], s["loss"], score=score))
        if case["grad"]:
            _done(plan.balance_backward(s["logits"], s["indices"], s["factor"], s["dlogits"], dloss=s["dloss"], score=score))
        return {n: s[n] for n in ("counts", "shares", "factor", "loss", "dlogits") if n in s}
    if op == "quantize4":
        _done(plan.quantize_mx4(s["X"], s["Q"], s["SQ"], s.get("QT"), s.get("SQT")))
        _done(plan.dequantize(s["Q"], s["SQ"], s["V"]))
        if case["both"]:
            _done(plan.dequantize(s["QT"], s["SQT"], s["VT"]))
        return {n: s[n] for n in ("V", "SQ", "VT", "SQT") if n in s}
    act = gemm.GEMM_ACT_SILU if case.get("act") == "silu" else gemm.GEMM_ACT_NONE
    if op == "product4":
        _done(plan.run_mx4(s["A"], s["SA"], s["B"], s["SB"], s["D"], K=case["K"], act=act))
    else:
        _done(plan.run_grouped_mx4(s["A"], s["SA"], s["B"], s["SB"], s["D"], s["starts"], s["counts"], K=case["K"], act=act))
    return s["D"]


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "balance": _plain_balance, "quantize4": _plain_quantize4, "product4": _plain_product4, "experts4": _plain_experts4}[state["case"]["op"]](state)


# ----------------------------------------------------------- in 64 bits

def _wide4(q, packed, K):
    """The numbers a 4-bit matrix stands for."""
    r, c = torch.arange(q.shape[0], device="cuda")[:, None], torch.arange(K, device="cuda")[None]
    code = (q[:, (c // 2)[0]].int() >> (4 * (c % 2))) & 15
    e, f = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e == 0, f / 2, torch.ldexp(1 + f / 2, e - 1)) * torch.where(code > 7, -1.0, 1.0)
    b = c // 32
    at = ((r // 128) * max(1, -(-K // 128)) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    return torch.ldexp(v, packed[at].to(torch.int32) - 127)


def _nearest(x, block, top, bits, least):
    """The values nearest to x (64 bits) that the codes and scales of its rows' blocks can have."""
    R, K = x.shape
    part = torch.nn.functional.pad(x, (0, -K % block)).view(R, -1, block)
    most = part.abs().amax(2, keepdim=True)
    up = torch.where(most == 0, -127.0, torch.ceil(torch.log2(most / top)).clamp(-127, 127))  # off by one at most, mended here
    up = torch.where(most > top * torch.exp2(up), up + 1, up)
    up = torch.where((most <= top * torch.exp2(up - 1)) & (up > -127), up - 1, up)
    v = part / torch.exp2(up)
    unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** (least - 1)))).clamp(min=least) - (bits - 1))
    return (torch.round(v / unit) * unit * torch.exp2(up)).view(R, -1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        t, gain = TYPES[case["x"]], s["gain"].double()
        h = s["X"].double() + s["residual"].double()
        y = h / (h.square().sum(1, keepdim=True) / case["N"] + EPS).sqrt()
        got = {"H": h}
        if case["form"] == "codes":
            return {**got, "V": _nearest(y * gain, 128, 448.0, 4, -6)}
        got["Y"] = y * gain
        if case["form"] == "train":  # the gradients are those at the sum as it was kept, with the factor of the sum itself
            r = (h.square().sum(1) / case["N"] + EPS).rsqrt()
            kept, dy = h.to(t).double(), s["dY"].double()
            inner = torch.einsum("rn,rn,n->r", dy, kept, gain) / case["N"]
            got["dX"] = dy * gain * r[:, None] - kept * (inner * r ** 3)[:, None] + s["dH"].double()
            got["dgain"], got["rstd"] = torch.einsum("rn,rn,r->n", dy, kept, r), r
        return got
    if op == "balance":
        T, E = case["T"], case["E"]
        x, index = s["logits"].double().requires_grad_(case["grad"]), s["indices"]
        on = index[(index >= 0) & (index < E)]
        counts = torch.bincount(on.long(), minlength=E).double()
        rows = (index >= 0).any(1).nonzero()[:, 0]
        p = torch.special.expit(x[rows]) if case["score"] == "sigmoid" else torch.softmax(x[rows], 1)
        shares = (p / p.sum(1, keepdim=True)).mean(0) if len(rows) else torch.zeros(E, dtype=torch.float64, device="cuda")
        f = counts / max(1, on.numel())
        loss = E * (f * shares).sum()
        got = {"counts": None, "shares": shares.detach(), "factor": E * f / max(1, len(rows)), "loss": loss.detach()[None]}
        if case["grad"]:
            d = torch.autograd.grad(loss, x)[0] if len(rows) else torch.zeros_like(x)
            got["dlogits"] = d * s["dloss"].double()
        return got
    if op == "quantize4":
        x = s["X"].double()
        got = {"V": _nearest(x, 32, 6.0, 2, 0), "SQ": None}
        return {**got, "VT": _nearest(x.t(), 32, 6.0, 2, 0), "SQT": None} if case["both"] else got
    if op == "product4":
        y = _wide4(s["A"], s["SA"], case["K"]) @ _wide4(s["B"], s["SB"], case["K"]).t()
        return y * torch.special.expit(y) if case["act"] == "silu" else y
    x, out = _wide4(s["A"], s["SA"], case["K"]), torch.zeros(s["D"].shape, dtype=torch.float64, device="cuda")
    for e, (start, n) in enumerate(zip(s["starts"].tolist(), s["counts"].tolist())):
        if n:
            out[start:start + n] = x[start:start + n] @ _wide4(s["B"][e], s["SB"][e], case["K"]).t()
    return out


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    size = lambda t: {"f32": 4}.get(t, 2)  # noqa: E731
    if op == "norm":
        R, N, b = case["R"], case["N"], size(case["x"])
        if case["form"] == "codes":  # x, residual in; sum, codes and their values out
            return {"bytes": R * N * (3 * b + 1 + 1 / 128 + 2), "flops": 6 * R * N}
        train = case["form"] == "train"  # also: dY and dH in, dX out (the sum is at hand)
        return {"bytes": R * N * (4 + 3 * train) * b + N * b, "flops": (5 + 10 * train) * R * N}
    if op == "balance":
        T, E, k = case["T"], case["E"], min(case["k"], case["E"])
        return {"bytes": T * E * 4 * (1 + case["grad"]) + T * k * 4, "flops": T * E * (4 + 5 * case["grad"])}
    if op == "quantize4":
        R, K, ways = case["R"], case["K"], 1 + case["both"]
        return {"bytes": R * K * size(case["x"]) + ways * R * K * (0.5 + 1 / 32 + 2), "flops": 2 * ways * R * K}
    if op == "product4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * (0.5 + 1 / 32) + M * N * size(case["out"]), "flops": 2 * M * N * K}
    T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
    read = E * (1 - (1 - k / E) ** T)  # experts that no token chose are not read: as for even choices
    return {"bytes": read * N * K * (0.5 + 1 / 32) + T * k * (K * (0.5 + 1 / 32) + N * 2), "flops": 2 * T * k * N * K}
