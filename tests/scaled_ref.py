"""Plain 64-bit implementations of the block-scaled products, the quantiser, routing and
the weighted sum (include/gemm.h), written from their formulas in numpy; what the
GPU and host tests compare with."""
from __future__ import annotations

import numpy as np

# largest value, bits of the significand (with the leading one), least exponent of a normal value
FORMATS = {"e4m3": (448.0, 4, -6), "e5m2": (57344.0, 3, -14)}


def decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    """What 8-bit codes stand for, in 64 bits."""
    c = np.arange(256)
    sign = np.where(c & 128, -1.0, 1.0)
    if fmt == "e4m3":
        e, f = (c >> 3) & 15, c & 7
        v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7.0))
        v = np.where((c & 127) == 127, np.nan, v)
    else:
        e, f = (c >> 2) & 31, c & 3
        v = np.where(e == 0, f * 2.0 ** -16, (1 + f / 4) * 2.0 ** (e - 15.0))
        v = np.where(e == 31, np.where(f == 0, np.inf, np.nan), v)
    return (sign * v)[codes]


def quantize(x: np.ndarray, fmt: str, block_rows: int = 1):
    """Values of the codes (before the scale) and scale bytes (rows x blocks) of x."""
    top, bits, least = FORMATS[fmt]
    x = np.asarray(x, np.float64)
    R, K = x.shape
    nb = -(-K // 128)
    byte = np.zeros((R, nb), np.int64)
    v = np.full(x.shape, np.nan)
    for r0 in range(0, R, block_rows):
        for b in range(nb):
            at = (slice(r0, r0 + block_rows), slice(128 * b, 128 * b + 128))
            part = x[at]
            fine = np.isfinite(part)
            m = np.abs(part[fine]).max() if fine.any() else 0.0
            e = -127
            while m > top * 2.0 ** e:
                e += 1
            byte[r0:r0 + block_rows, b] = e + 127
            y = np.where(fine, part, 0.0) / 2.0 ** e
            unit = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 1e-300))), least) - (bits - 1))
            v[at] = np.where(fine, np.round(y / unit) * unit, np.nan)  # (numpy rounds ties to even)
    return v, byte


def scale_offset(r, c, cols: int):
    """Byte of row r, block c in the packed scales of a matrix of `cols` columns."""
    groups = max(1, -(-cols // 512))
    return ((r // 128) * groups + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4


def pack(byte: np.ndarray, cols: int) -> np.ndarray:
    R, nb = byte.shape
    out = np.zeros(max(1, -(-R // 128)) * max(1, -(-cols // 512)) * 512, np.uint8)
    r, c = np.meshgrid(np.arange(R), np.arange(nb), indexing="ij")
    out[scale_offset(r, c, cols)] = byte
    return out


def scaled(values: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """Element values of a block-scaled matrix."""
    return values * np.repeat(2.0 ** (byte - 127.0), 128, axis=1)[:, :values.shape[1]]


def act(y: np.ndarray, kind: int, slope: float = 0.0) -> np.ndarray:
    from math import erfc
    if kind == 1:
        return np.where(y < 0, slope * y, y)
    if kind == 2:
        return np.where(y < 0, 0.0, y)
    if kind == 3:
        return 0.5 * y * np.vectorize(erfc)(-y / np.sqrt(2.0))
    if kind == 4:
        with np.errstate(over="ignore"):
            return y / (1 + np.exp(-y))
    return y


def route(x, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=False, scale=1.0):
    """(indices, weights, scores) of logits x; keys as gemm_route's, in 64 bits."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))
    T, E = x.shape
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-x))
        else:
            top = x.max(1, keepdims=True)
            e = np.where(np.isneginf(x), 0.0, np.where(x == top, 1.0, np.exp(x - top)))
            s = np.where(e.sum(1, keepdims=True) > 0, e / np.maximum(e.sum(1, keepdims=True), 1e-300), 0.0)
    key = x.copy() if bias is None and group_top == 1 else s + (0.0 if bias is None else np.asarray(bias, np.float64))
    key[np.isneginf(x) | np.isnan(key)] = -np.inf
    out = np.zeros((T, k), np.int64)
    w = np.zeros((T, k))
    per = E // groups
    for t in range(T):
        g = key[t].reshape(groups, per)
        best = np.sort(g, 1)[:, ::-1]
        gk = best[:, 0] if group_top == 1 or per == 1 else best[:, 0] + best[:, 1]
        chosen = sorted(range(groups), key=lambda i: (-gk[i], i))[:top_groups]
        experts = [e for c in sorted(chosen) for e in range(c * per, (c + 1) * per)]
        out[t] = sorted(experts, key=lambda e: (-key[t, e], e))[:k]
        w[t] = s[t, out[t]]
    if renormalize:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1), 0.0)
    return out, w * scale, s


def route_backward(x, indices, dw, score="softmax", renormalize=False, scale=1.0):
    """Gradient of the weights' sum with dw with respect to x, from the formula."""
    _, _, s = route(x, 1, score)
    T, E = s.shape
    dx = np.zeros((T, E))
    for t in range(T):
        on = [j for j, e in enumerate(indices[t]) if 0 <= e < E]
        sj = np.array([s[t, indices[t][j]] for j in on])
        d = np.array([dw[t][j] for j in on], np.float64)
        if renormalize:
            total = sj.sum()
            d = (d - (d * sj).sum() / total) / total if total > 0 else np.zeros_like(d)
        ds = np.zeros(E)
        for j, v in zip(on, scale * d):
            ds[indices[t][j]] += v
        dx[t] = s[t] * (1 - s[t]) * ds if score == "sigmoid" else s[t] * (ds - (ds * s[t]).sum())
    return dx


def order(indices: np.ndarray, experts: int, rows: int):
    """(starts, counts, pos, rowmap) of the slots in expert order."""
    flat = indices.reshape(-1)
    starts, counts, at = [], [], 0
    pos = np.full(flat.shape, -1, np.int64)
    rowmap = np.full(rows, -1, np.int64)
    for e in range(experts):
        mine = np.nonzero(flat == e)[0]
        starts.append(at)
        counts.append(len(mine))
        pos[mine] = at + np.arange(len(mine))
        rowmap[at:at + len(mine)] = mine
        at += -(-len(mine) // 128) * 128
    return np.array(starts), np.array(counts), pos.reshape(indices.shape), rowmap
