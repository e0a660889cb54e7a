"""Plain 64-bit implementations of the 4-bit quantiser and codes, the norm and the balance loss
(include/gemm.h), written from their formulas in numpy; what the GPU and host tests compare with."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def decode4(packed: np.ndarray, cols: int) -> np.ndarray:
    """What rows of 4-bit codes, two to a byte, stand for."""
    code = np.stack([packed & 15, packed >> 4], 2).reshape(packed.shape[0], -1)[:, :cols]
    return np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]


def pack4(code: np.ndarray) -> np.ndarray:
    """Rows of codes (0 .. 15) as bytes of two, the even column's in the low four bits."""
    code = np.pad(code, ((0, 0), (0, code.shape[1] % 2))).astype(np.uint8)
    return code[:, ::2] | code[:, 1::2] << 4


def quantize4(x: np.ndarray):
    """Values of the codes (before the scale) and scale bytes (rows x blocks of 32) of x; 255 and codes of 0 for a block that is not
    finite."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    nb = -(-K // 32)
    byte, v = np.zeros((R, nb), np.int64), np.zeros(x.shape)
    for r in range(R):
        for b in range(nb):
            part = x[r, 32 * b:32 * b + 32]
            if not np.isfinite(part).all():
                byte[r, b] = 255
                continue
            m, e = np.abs(part).max(), -127
            if m > 0:
                e = max(-127, int(np.floor(np.log2(m))) - 4)
                while m > 6 * 2.0 ** e:
                    e += 1
            byte[r, b] = e + 127
            y = np.abs(part) / 2.0 ** e
            unit = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(y, 1e-300))), 0) - 1)
            v[r, 32 * b:32 * b + 32] = np.copysign(np.round(y / unit) * unit, part)  # (numpy rounds ties to even)
    return v, byte


def pack_scales4(byte: np.ndarray, cols: int) -> np.ndarray:
    R, nb = byte.shape
    tiles = max(1, -(-cols // 128))
    out = np.zeros(max(1, -(-R // 128)) * tiles * 512, np.uint8)
    r, c = np.meshgrid(np.arange(R), np.arange(nb), indexing="ij")
    out[((r // 128) * tiles + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4] = byte
    return out


def scaled4(values: np.ndarray, byte: np.ndarray) -> np.ndarray:
    by = np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))
    return values * np.repeat(by, 32, axis=1)[:, :values.shape[1]]


def norm(x, r, gain, eps):
    """(h, rstd, y)."""
    h = x.astype(np.float64) + (0.0 if r is None else r.astype(np.float64))
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1 / np.sqrt((h * h).mean(1) + eps)
        y = h * rstd[:, None] * (1.0 if gain is None else gain.astype(np.float64))
    return h, rstd, y


def norm_backward(dy, h, gain, rstd, dh):
    """(dx, dgain, what dx's and dgain's terms add up to in size)."""
    gain = np.ones(h.shape[1]) if gain is None else gain
    xhat, g = h * rstd[:, None], dy * gain
    mean = (g * xhat).mean(1, keepdims=True)
    size = rstd[:, None] * (np.abs(g) + np.abs(xhat) * np.abs(g * xhat).mean(1, keepdims=True))
    extra = 0.0 if dh is None else dh
    return rstd[:, None] * (g - xhat * mean) + extra, (dy * xhat).sum(0), size + np.abs(extra), np.abs(dy * xhat).sum(0)


def balance(x, indices, score="softmax", scale=1.0):
    """(counts, shares, factor, loss, p, which tokens take part)."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))
    T, E = x.shape
    valid = (indices >= 0) & (indices < E)
    live = valid.any(1)
    counts = np.bincount(indices[valid], minlength=E).astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1 / (1 + np.exp(-x))
        else:
            top = x.max(1, keepdims=True) if E else x
            s = np.where(np.isneginf(x), 0.0, np.where(x == top, 1.0, np.exp(x - top)))
    total = s.sum(1, keepdims=True)
    p = np.where(total > 0, s / np.where(total > 0, total, 1), 0.0)
    m, n = max(1, live.sum()), max(1, counts.sum())
    shares = p[live].sum(0) / m
    factor = scale * E * counts / n / m
    return counts.astype(np.int64), shares, factor, (scale * E * counts / n * shares).sum(), p, live


def balance_backward(x, indices, factor, dloss, score="softmax"):
    _, _, _, _, p, live = balance(x, indices, score)
    d = dloss * p * (factor - (factor * p).sum(1, keepdims=True))
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            d = d / (1 + np.exp(np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))))
    return np.where(live[:, None], d, 0.0)
