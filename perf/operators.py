"""What the 8-bit product, the experts' products and the routing around them are measured on.

Five operators (include/gemm.h):

  quantize   matrix -> 8-bit values with a power-of-two scale for each block of 128, and its transpose
  product    D = A @ B^T of two such matrices
  experts    the same product for each expert's rows ("rows": y = x @ W_e^T; "grad": dW_e = dy_e^T @ x_e)
  route      scores -> the chosen experts, their weights and the order of the rows; with the gradient of the scores
  combine    the weighted sum of the experts' rows back into tokens; with its gradients

`run` computes them with elementary torch operations in 32 bits, or, where `own` is true, with this package.
"""
import math

import torch

own = False

LOWEST, BLOCK = -127, 128  # the least exponent of a scale byte; values that share a scale
FORMATS = {"e4m3": (torch.float8_e4m3fn, 9, 4, -6), "e5m2": (torch.float8_e5m2, 16, 3, -14)}  # type, frexp of the largest value (0.875 x 2^), significant bits, least exponent
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token through a square projection: latency and the weights' bytes
        {"name": "product_one_token", "op": "product", "M": 1, "N": 4096, "K": 4096, "a": "e4m3", "out": "bf16", "act": "none"},
        # a long prompt through a large projection: the benchmark's square size
        {"name": "product_prompt", "op": "product", "M": 8192, "N": 8192, "K": 8192, "a": "e4m3", "out": "bf16", "act": "none"},
        # a weight's gradient over a ragged number of tokens: gradients in e5m2, 32-bit result
        {"name": "product_weight_grad", "op": "product", "M": 6912, "N": 2048, "K": 4099, "a": "e5m2", "out": "f32", "act": "none"},
        # a layer's activations, kept in 8 bits for the product and, transposed, for the backward pass
        {"name": "quantize_activations", "op": "quantize", "R": 8192, "K": 4096, "a": "e4m3", "x": "bf16", "both": True, "rows": 1},
        # a decoded batch on its way into an 8-bit product
        {"name": "quantize_decode", "op": "quantize", "R": 33, "K": 2050, "a": "e4m3", "x": "bf16", "both": False, "rows": 1},
        # single tokens through experts: every chosen expert's weights are read for a few rows
        {"name": "experts_decode", "op": "experts", "form": "rows", "T": 48, "k": 4, "E": 64, "N": 2048, "K": 2048, "out": "bf16"},
        # a prompt through experts, uneven loads
        {"name": "experts_prompt", "op": "experts", "form": "rows", "T": 8192, "k": 4, "E": 32, "N": 4096, "K": 2048, "out": "bf16"},
        # the experts' weight gradients of a training step
        {"name": "experts_grad", "op": "experts", "form": "grad", "T": 4096, "k": 4, "E": 16, "N": 2048, "K": 2048, "out": "f32"},
        # routing one decoded batch: sigmoid scores, balance bias, groups of experts
        {"name": "route_decode", "op": "route", "T": 16, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "grad": False},
        # routing a training batch, with the gradient of the scores
        {"name": "route_train", "op": "route", "T": 16384, "E": 128, "k": 8, "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "grad": True},
        # the experts' rows of a decoded batch summed into tokens
        {"name": "combine_decode", "op": "combine", "T": 24, "k": 8, "E": 64, "N": 2048, "grad": False},
        # the experts' rows of a training batch summed into tokens, and the gradients of rows and weights
        {"name": "combine_train", "op": "combine", "T": 8192, "k": 4, "E": 32, "N": 2048, "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product", "quantize", "experts", "experts", "route", "combine"])
    if op == "product":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 512, 8192), "K": _log(rng, 512, 8192),
                "a": rng.choice(["e4m3", "e4m3", "e5m2"]), "out": rng.choice(["bf16", "f16", "f32"]), "act": rng.choice(["none", "silu"])}
    if op == "quantize":
        return {"op": op, "R": _log(rng, 1, 8192), "K": _log(rng, 512, 8192), "a": rng.choice(["e4m3", "e5m2"]),
                "x": rng.choice(["bf16", "f16", "f32"]), "both": rng.random() < 0.5, "rows": rng.choice([1, 1, 128])}
    if op == "experts":
        form, E = rng.choice(["rows", "grad"]), rng.choice([8, 16, 32, 48, 64])
        return {"op": op, "form": form, "T": _log(rng, 1 if form == "rows" else 256, 8192 if form == "rows" else 4096), "k": rng.choice([1, 2, 4]), "E": E,
                "N": 8 * _log(rng, 64, 256), "K": 8 * _log(rng, 64, 256), "out": "bf16" if form == "rows" else "f32"}
    if op == "route":
        score = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 4, 8]) if score == "sigmoid" else 1
        return {"op": op, "T": _log(rng, 1, 16384), "E": rng.choice([8, 16, 64, 128, 160, 256]) if groups == 1 else rng.choice([64, 128, 160, 256]), "k": rng.randint(1, 8),
                "score": score, "bias": score == "sigmoid", "groups": groups, "top_groups": max(1, groups // 2), "grad": rng.random() < 0.5}
    return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, 8), "E": rng.choice([8, 32, 64]), "N": 2 * _log(rng, 256, 1024), "grad": rng.random() < 0.5}


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


def _codes(g, rows, K, kind):
    """An 8-bit matrix and its scales, as a quantiser leaves them: values up to the type's largest, scales around 2^-8."""
    dtype = FORMATS[kind][0]
    top = 448.0 if kind == "e4m3" else 57344.0
    q = _rows(rows, K, dtype)
    blocks = -(-K // BLOCK)
    grain = torch.randn((rows, K), generator=g, device="cuda").mul_(top / 5).clamp_(-top, top)
    q.copy_(grain.to(dtype))
    spread = torch.randint(-10 if kind == "e4m3" else -17, -6 if kind == "e4m3" else -13, (rows, blocks), generator=g, device="cuda")
    return q, _pack((spread + 127).to(torch.uint8))


def _pack(b):
    """Scale bytes, one for each row and block of 128 columns, in the packed order: tiles of 128 rows x 4 blocks, each as 32 lines
    of 16 bytes; row r, block c of a tile is byte (r % 32) * 16 + (r // 32) * 4 + c. What is beyond the matrix is 0."""
    rows, blocks = b.shape
    R, C = _up(max(rows, 1), 128), _up(max(blocks, 1), 4)
    full = torch.zeros((R, C), dtype=torch.uint8, device=b.device)
    full[:rows, :blocks] = b
    return full.view(R // 128, 4, 32, C // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _segments(g, T, k, E):
    """An uneven choice of k different experts for each token, and the order of its rows: expert e has `counts[e]` rows from
    `starts[e]`, a multiple of 128; row r holds choice `rowmap[r]` (token * k + j), or none (-1)."""
    liking = torch.randn((1, E), generator=g, device="cuda") * 0.5
    chosen = torch.topk(liking + torch.randn((T, E), generator=g, device="cuda"), min(k, E), dim=1).indices.to(torch.int32)
    return chosen, *_order(chosen, E, _capacity(T * k, E))


def _capacity(slots, E):
    return _up(slots + 127 * min(E, slots), 128)


def _order(chosen, E, cap):
    flat = chosen.reshape(-1).long()
    counts = (flat[:, None] == torch.arange(E, device=flat.device)).sum(0)
    padded = (counts + 127) // 128 * 128
    starts = padded.cumsum(0) - padded
    by = torch.sort(flat, stable=True).indices
    first = counts.cumsum(0) - counts
    pos = torch.empty_like(flat)
    pos[by] = starts[flat[by]] + torch.arange(flat.numel(), device=flat.device) - first[flat[by]]
    rowmap = torch.full((cap,), -1, dtype=torch.int32, device=flat.device)
    rowmap[pos] = torch.arange(flat.numel(), dtype=torch.int32, device=flat.device)
    return starts.to(torch.int32), counts.to(torch.int32), pos.to(torch.int32).view(chosen.shape), rowmap


def _clear(logits, bias, case):
    """Whether no choice of a row hangs on the last bits: the sorted keys (and groups' keys) are apart."""
    key = torch.sigmoid(logits.double()) if case["score"] == "sigmoid" else torch.softmax(logits.double(), 1)
    if bias is not None:
        key = key + bias.double()
    near = lambda v: (v.sort(1).values.diff(dim=1) < 2e-6).any(1)  # noqa: E731
    bad = near(key)
    if case["groups"] > 1:
        bad |= near(key.view(len(key), case["groups"], -1).topk(2, dim=2).values.sum(2))
    return ~bad


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    s, op = {"case": case}, case["op"]
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["SA"] = _codes(g, M, K, case["a"])
        s["B"], s["SB"] = _codes(g, N, K, "e4m3")
        s["D"] = _rows(M, N, TYPES[case["out"]])
    elif op == "quantize":
        R, K, kind = case["R"], case["K"], FORMATS[case["a"]][0]
        s["X"] = _normal(g, R, K, TYPES[case["x"]])
        s["Q"], s["SQ"] = _rows(R, K, kind), _pack(torch.zeros((R, -(-K // BLOCK)), dtype=torch.uint8, device="cuda"))
        if case["both"]:
            s["QT"], s["SQT"] = _rows(K, R, kind), _pack(torch.zeros((K, -(-R // BLOCK)), dtype=torch.uint8, device="cuda"))
    elif op == "experts":
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        s["chosen"], s["starts"], s["counts"], s["pos"], s["rowmap"] = _segments(g, T, k, E)
        cap = s["rowmap"].numel()
        if case["form"] == "rows":
            s["A"], s["SA"] = _codes(g, cap, K, "e4m3")
            B = [_codes(g, N, K, "e4m3") for _ in range(E)]
            s["B"], s["SB"] = torch.stack([b for b, _ in B]), torch.stack([c for _, c in B])
            s["D"] = _rows(cap, N, TYPES[case["out"]], torch.zeros)
        else:  # rows that hold no choice are zero, as the quantiser leaves them
            s["A"], s["SA"] = _codes(g, N, cap, "e5m2")
            s["B"], s["SB"] = _codes(g, K, cap, "e4m3")
            for n in "AB":
                s[n].view(torch.uint8)[:, s["rowmap"] < 0] = 0
            s["D"] = torch.empty((E, N, K), device="cuda")
        s["most"] = int(s["counts"].max())  # rows of the fullest expert, for the plain form's batch
    elif op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        draw_logits = lambda: torch.randn((T, E), generator=g, device="cuda") * 1.5  # noqa: E731
        s["bias"] = torch.rand((E,), generator=g, device="cuda") * 0.2 - 0.1 if case["bias"] else None
        s["logits"] = draw_logits()
        for _ in range(12 if case["bias"] else 0):
            s["logits"] = torch.where(_clear(s["logits"], s["bias"], case)[:, None], s["logits"], draw_logits())
        whole = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        s["weights"], s["indices"], s["pos"] = torch.empty((T, k), device="cuda"), whole(T, k), whole(T, k)
        s["starts"], s["counts"], s["rowmap"] = whole(E), whole(E), whole(_capacity(T * k, E))
        if case["grad"]:
            s["dweights"], s["dlogits"] = torch.randn((T, k), generator=g, device="cuda"), torch.empty((T, E), device="cuda")
    else:
        T, k, E, N = case["T"], case["k"], case["E"], case["N"]
        s["chosen"], s["starts"], s["counts"], s["pos"], s["rowmap"] = _segments(g, T, k, E)
        s["Y"] = _normal(g, s["rowmap"].numel(), N, torch.bfloat16)
        s["weights"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1)
        s["out"] = _rows(T, N, torch.bfloat16)
        if case["grad"]:
            s["dout"] = _normal(g, T, N, torch.bfloat16)
            s["dY"], s["dweights"] = _rows(s["rowmap"].numel(), N, torch.bfloat16), torch.empty((T, k), device="cuda")
    return s


# -------------------------------------------------------------- plain forms

def _scales(packed, rows, cols):
    """Scales of a rows x cols matrix, one for each value, in 32 bits."""
    R, C = _up(max(rows, 1), 128), _up(max(-(-cols // BLOCK), 1), 4)
    b = packed.view(R // 128, C // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R, C)[:rows].int()
    two = torch.where(b == 0, 1 << 22, b << 23).view(torch.float32)  # 2^(b - 127)
    return two.repeat_interleave(BLOCK, 1)[:, :cols]


def _values(q, packed):
    return q.float() * _scales(packed, *q.shape)


def _act(x, act):
    return x / (1 + torch.exp(-x)) if act == "silu" else x


def _quantized(x, kind, rows):
    """Codes and packed scales of x in 32 bits, one scale for `rows` x 128 values."""
    dtype, top, _, _ = FORMATS[kind]
    R, K = x.shape
    fine = torch.isfinite(x)
    full = torch.zeros((_up(R, rows), _up(K, BLOCK)), device=x.device)
    full[:R, :K] = torch.where(fine, x, 0).abs()
    most = full.view(-1, rows, full.shape[1] // BLOCK, BLOCK).amax((1, 3))
    m, e = torch.frexp(most)
    e = torch.where(most > 0, (e - top + (m > 0.875)).clamp(min=LOWEST), LOWEST).to(torch.int32)
    e = e.repeat_interleave(rows, 0)[:R]
    down = ((127 - e) << 23).view(torch.float32).repeat_interleave(BLOCK, 1)[:, :K]  # 2^-e
    return torch.where(fine, x * down, math.nan).to(dtype), _pack((e + 127).to(torch.uint8))


def _plain_quantize(s):
    case, x = s["case"], s["X"].float()
    got = dict(zip(("Q", "SQ"), _quantized(x, case["a"], case["rows"])))
    if case["both"]:
        got.update(zip(("QT", "SQT"), _quantized(x.t(), case["a"], case["rows"])))
    return got


def _plain_product(s):
    y = _values(s["A"], s["SA"]) @ _values(s["B"], s["SB"]).t()
    return _act(y, s["case"]["act"]).to(s["D"].dtype)


def _batch(s):
    """[E, most] rows of the experts, and whether an expert has that many."""
    at = torch.arange(s["most"], device="cuda")
    held = at < s["counts"][:, None]
    return torch.where(held, s["starts"][:, None] + at, 0).long(), held


def _plain_experts(s):
    case = s["case"]
    E, N, K = case["E"], case["N"], case["K"]
    rows, held = _batch(s)
    if case["form"] == "rows":
        x = _values(s["A"], s["SA"])[rows]
        C, R = _up(-(-K // BLOCK), 4), _up(N, 128)
        packed = s["SB"].view(E * R // 128, -1).reshape(-1)
        w = s["B"].float() * _scales(packed, E * R, C * BLOCK).view(E, R, C * BLOCK)[:, :N, :K]
        y = torch.bmm(x, w.transpose(1, 2))
        out = torch.zeros((s["A"].shape[0], N), device="cuda")
        out[rows[held]] = y[held]
        return out.to(s["D"].dtype)
    dy = torch.where(held[..., None], _values(s["A"], s["SA"]).t()[rows], 0)
    x = torch.where(held[..., None], _values(s["B"], s["SB"]).t()[rows], 0)
    return torch.bmm(dy.transpose(1, 2), x)


def _score(logits, kind):
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    case = s["case"]
    E, k, groups = case["E"], case["k"], case["groups"]
    score = _score(s["logits"], case["score"])
    key = s["logits"] if s["bias"] is None and groups == 1 else score if s["bias"] is None else score + s["bias"]
    if groups > 1:  # experts of the groups whose two highest keys have the highest sums
        per = key.view(-1, groups, E // groups)
        best = per.sort(2, descending=True).values[..., :2].sum(2)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        on = torch.zeros_like(best, dtype=torch.bool).scatter_(1, keep, True)
        key = torch.where(on[..., None], per, -math.inf).view(-1, E)
    indices = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, indices)
    total = w.sum(1, keepdim=True)
    weights = w / total
    starts, counts, pos, rowmap = _order(indices, E, s["rowmap"].numel())
    got = {"weights": weights, "indices": indices.to(torch.int32), "starts": starts, "counts": counts, "pos": pos, "rowmap": rowmap}
    if case["grad"]:
        dw = s["dweights"]
        dchosen = (dw - (dw * weights).sum(1, keepdim=True)) / total
        ds = torch.zeros_like(score).scatter_(1, indices, dchosen)
        got["dlogits"] = ds * score * (1 - score) if case["score"] == "sigmoid" else score * (ds - (ds * score).sum(1, keepdim=True))
    return got


def _plain_combine(s):
    case, w = s["case"], s["weights"]
    rows = s["Y"].float()[s["pos"].long()]  # [T, k, N]
    got = {"out": (w[..., None] * rows).sum(1).to(torch.bfloat16)}
    if case["grad"]:
        dout = s["dout"].float()
        dY = torch.zeros_like(s["dY"], dtype=torch.float32)
        dY[s["pos"].long()] = w[..., None] * dout[:, None]
        got["dY"], got["dweights"] = dY.to(torch.bfloat16), (rows * dout[:, None]).sum(2)
    return got


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
    case = s["case"]
    plan, gemm = _plan()
    if case["op"] == "product":
        _done(plan.run_scaled(s["A"], s["SA"], s["B"], s["SB"], s["D"], act=gemm.GEMM_ACT_SILU if case["act"] == "silu" else gemm.GEMM_ACT_NONE))
        return s["D"]
    if case["op"] == "quantize":
        _done(plan.quantize(s["X"], s["Q"], s["SQ"], s.get("QT"), s.get("SQT"), block_rows=case["rows"]))
        return {n: s[n] for n in ("Q", "SQ", "QT", "SQT") if n in s}
    if case["op"] == "experts":
        call = plan.run_grouped if case["form"] == "rows" else plan.run_grouped_k
        _done(call(s["A"], s["SA"], s["B"], s["SB"], s["D"], s["starts"], s["counts"]))
        return s["D"]
    if case["op"] == "route":
        how = {"score": gemm.GEMM_SCORE_SIGMOID if case["score"] == "sigmoid" else gemm.GEMM_SCORE_SOFTMAX, "renormalize": True}
        _done(plan.route(s["logits"], s["weights"], s["indices"], bias=s["bias"], groups=case["groups"], top_groups=case["top_groups"],
                         group_top=2 if case["groups"] > 1 else 1, **how))
        _done(plan.route_map(s["indices"], case["E"], s["starts"], s["counts"], s["pos"], s["rowmap"]))
        names = ("weights", "indices", "starts", "counts", "pos", "rowmap")
        if case["grad"]:
            _done(plan.route_backward(s["logits"], s["indices"], s["dweights"], s["dlogits"], **how))
            names += ("dlogits",)
        return {n: s[n] for n in names}
    _done(plan.combine(s["Y"], s["pos"], s["weights"], s["out"]))
    if case["grad"]:
        _done(plan.combine_backward(s["dout"], s["Y"], s["pos"], s["weights"], s["dY"], s["dweights"], rowmap=s["rowmap"]))
    return {n: s[n] for n in ("out", "dY", "dweights") if n in s}


def run(state):
    if own:
        return _own(state)
    return {"product": _plain_product, "quantize": _plain_quantize, "experts": _plain_experts, "route": _plain_route, "combine": _plain_combine}[state["case"]["op"]](state)


# ----------------------------------------------------------- in 64 bits

def _wide(q, packed):
    """The numbers an 8-bit matrix stands for."""
    rows, cols = q.shape
    r, c = torch.arange(rows, device="cuda")[:, None], torch.arange(cols, device="cuda")[None] // BLOCK
    tiles = max(1, -(-cols // (4 * BLOCK)))
    at = ((r // 128) * tiles + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
    return torch.ldexp(q.to(torch.float64), packed[at].to(torch.int32) - 127)


def _nearest(x, kind, rows):
    """The codes' values for x (64 bits) in blocks of 128 along its last axis, the scale shared by `rows` lines."""
    dtype, _, bits, least = FORMATS[kind]
    top = 448.0 if kind == "e4m3" else 57344.0
    R, K = x.shape
    full = torch.nn.functional.pad(x, (0, -K % BLOCK, 0, -R % rows))
    part = full.view(full.shape[0] // rows, rows, full.shape[1] // BLOCK, BLOCK)
    most = part.abs().amax((1, 3), keepdim=True)
    up = torch.where(most == 0, -127.0, torch.ceil(torch.log2(most / top)).clamp(-127, 127))  # off by one at most, mended here
    up = torch.where(most > top * torch.exp2(up), up + 1, up)
    up = torch.where((most <= top * torch.exp2(up - 1)) & (up > -127), up - 1, up)
    v = part / torch.exp2(up)
    unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** (least - 1)))).clamp(min=least) - (bits - 1))
    return (torch.round(v / unit) * unit).view(full.shape)[:R, :K]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        y = _wide(s["A"], s["SA"]) @ _wide(s["B"], s["SB"]).t()
        return y * torch.special.expit(y) if case["act"] == "silu" else y
    if op == "quantize":
        x = s["X"].double()
        got = {"Q": _nearest(x, case["a"], case["rows"]), "SQ": None}
        return {**got, "QT": _nearest(x.t(), case["a"], case["rows"]), "SQT": None} if case["both"] else got
    if op == "experts":
        E, k = case["E"], case["k"]
        if case["form"] == "rows":
            x, out = _wide(s["A"], s["SA"]), torch.zeros(s["D"].shape, dtype=torch.float64, device="cuda")
            for e in range(E):
                mine = (s["chosen"] == e).nonzero()
                rows = s["pos"][mine[:, 0], mine[:, 1]].long()
                out[rows] = x[rows] @ _wide(s["B"][e], s["SB"][e]).t()
            return out
        dy, x = _wide(s["A"], s["SA"]), _wide(s["B"], s["SB"])
        owner = torch.where(s["rowmap"] >= 0, s["chosen"].reshape(-1)[s["rowmap"].clamp(min=0).long()], -1)
        return torch.stack([dy[:, owner == e] @ x[:, owner == e].t() for e in range(E)])
    if op == "route":
        x = s["logits"].double().requires_grad_(case["grad"])
        score = torch.special.expit(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
        key = (score if s["bias"] is None else score + s["bias"].double()).detach().cpu().numpy().copy()
        T, E, k, groups = case["T"], case["E"], case["k"], case["groups"]
        if groups > 1:
            import numpy as np
            per = key.reshape(T, groups, -1)
            two = np.sort(per, 2)[..., -2:].sum(2)
            drop = np.argsort(-two, 1, kind="stable")[:, case["top_groups"]:]
            np.put_along_axis(per, drop[..., None], -np.inf, 1)
        chosen = torch.from_numpy((-key).argsort(1, kind="stable")[:, :k].copy()).cuda()
        w = score.gather(1, chosen)
        w = w / w.sum(1, keepdim=True)
        got = {n: None for n in ("indices", "starts", "counts", "pos", "rowmap")}
        got["weights"] = w.detach()
        if case["grad"]:
            got["dlogits"], = torch.autograd.grad(w, x, s["dweights"].double())
        return got
    T, k, N = case["T"], case["k"], case["N"]
    w, out = s["weights"].double(), torch.zeros((T, N), dtype=torch.float64, device="cuda")
    for j in range(k):
        out += w[:, j, None] * s["Y"][s["pos"][:, j].long()].double()
    got = {"out": out}
    if case["grad"]:
        dout, dY, dw = s["dout"].double(), torch.zeros(s["dY"].shape, dtype=torch.float64, device="cuda"), torch.zeros((T, k), dtype=torch.float64, device="cuda")
        for j in range(k):
            at = s["pos"][:, j].long()
            dY[at] = w[:, j, None] * dout
            dw[:, j] = (dout * s["Y"][at].double()).sum(1)
        got["dY"], got["dweights"] = dY, dw
    return got


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    size = lambda t: {"f32": 4}.get(t, 2)  # noqa: E731
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K + -(-K // BLOCK)) + M * N * size(case["out"]), "flops": 2 * M * N * K}
    if op == "quantize":
        R, K = case["R"], case["K"]
        return {"bytes": R * K * size(case["x"]) + (1 + case["both"]) * R * K * (1 + 1 / BLOCK), "flops": 2 * R * K}
    if op == "experts":
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        slots = T * k
        if case["form"] == "rows":  # experts that no token chose are not read: as for even choices
            read = E * (1 - (1 - k / E) ** T)
            return {"bytes": read * N * K + slots * (K + N * size(case["out"])), "flops": 2 * slots * N * K}
        return {"bytes": slots * (N + K) + E * N * K * 4, "flops": 2 * slots * N * K}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * 4 + 4 * T * k * 4 + case["grad"] * (2 * T * E * 4 + 2 * T * k * 4), "flops": T * E * (k + 4)}
    T, k, N = case["T"], case["k"], case["N"]
    return {"bytes": T * N * 2 * (k + 1) + T * k * 8 + case["grad"] * (T * N * 2 * (2 * k + 1) + 2 * T * k * 4), "flops": 2 * T * k * N * (1 + 2 * case["grad"])}
