"""Plain definitions of the backward pass (numpy, fp64): what the gradient
calls of include/q4.h are checked against.  Loops over blocks, experts and
choices as the definitions are written; nothing is shared with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np

MX8_TOP = {"mxint8": 127.0, "mxfp8": 448.0}
MX8_LEAST = -111


def _e4m3_values() -> np.ndarray:
    """Magnitudes of the E4M3 codes 0..126 in order."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(v[:127])


E4M3 = _e4m3_values()


def _e4m3_code(t: float) -> int:
    """Nearest E4M3 magnitude code of t in [0, 448], ties to the even code."""
    d = np.abs(E4M3 - t)
    best = np.flatnonzero(d == d.min())
    return int(best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1])


def mx8_quantize(fmt: str, x: np.ndarray):
    """(codes uint8 [rows, cols], scales uint8 [rows, cols/32]) of fp32 x that
    holds bf16 values."""
    top = MX8_TOP[fmt]
    rows, cols = x.shape
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, cols // 32), np.uint8)
    for r in range(rows):
        for b in range(cols // 32):
            v = x[r, 32 * b:32 * b + 32].astype(np.float64)
            if not np.all(np.isfinite(v)):
                scales[r, b] = 255
                codes[r, 32 * b:32 * b + 32] = 0 if fmt == "mxint8" else 0x7F
                continue
            e, amax = MX8_LEAST, float(np.max(np.abs(v)))
            while amax > top * 2.0 ** e:
                e += 1
            scales[r, b] = e + 127
            for i, w in enumerate(v):
                y = float(w) * 2.0 ** -e
                if fmt == "mxint8":
                    q = int(np.rint(y))
                    while abs(q) * 2.0 ** e >= 2.0 ** 128:
                        q -= 1 if q > 0 else -1
                    codes[r, 32 * b + i] = q & 0xFF
                else:
                    c = _e4m3_code(abs(y))
                    while E4M3[c] * 2.0 ** e >= 2.0 ** 128:
                        c -= 1
                    codes[r, 32 * b + i] = c | (0x80 if math.copysign(1.0, y) < 0 else 0)
    return codes, scales


def mx8_dequant(fmt: str, codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values (fp64) that codes and scales stand for."""
    if fmt == "mxint8":
        v = codes.view(np.int8).astype(np.float64)
    else:
        m = np.append(E4M3, np.nan)[codes & 0x7F]
        v = np.where(codes & 0x80, -m, m)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=1)


def moe_sort(ids: np.ndarray, E: int):
    """(offsets [E+1], gather of the kept rows, inv [T, k])."""
    T, k = ids.shape
    rows = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                rows[ids[t, j]].append((t, j))
    offsets = np.zeros(E + 1, np.int32)
    gather, inv = [], np.full((T, k), -1, np.int32)
    for e in range(E):
        for t, j in rows[e]:
            inv[t, j] = len(gather)
            gather.append(t)
        offsets[e + 1] = len(gather)
    return offsets, np.array(gather, np.int32), inv


def permute(x, inv, xs) -> np.ndarray:
    xs = xs.copy()
    for t in range(inv.shape[0]):
        for p in inv[t]:
            if 0 <= p < xs.shape[0]:
                xs[p] = x[t]
    return xs


def permute_backward(dxs, inv) -> np.ndarray:
    dx = np.zeros((inv.shape[0], dxs.shape[1]))
    for t in range(inv.shape[0]):
        for p in inv[t]:
            if 0 <= p < dxs.shape[0]:
                dx[t] += dxs[p]
    return dx


def combine_backward(dout, y, inv, weights, dy):
    """(dy with the owned rows replaced, dweights)."""
    dy, dw = dy.astype(np.float64), np.zeros(inv.shape)
    for t in range(inv.shape[0]):
        for j, p in enumerate(inv[t]):
            if 0 <= p < dy.shape[0]:
                dy[p] = float(weights[t, j]) * dout[t].astype(np.float64)
                dw[t, j] = dout[t].astype(np.float64) @ y[p].astype(np.float64)
    return dy, dw


def topk_backward(logits, ids, dweights) -> np.ndarray:
    T, E = logits.shape
    dl = np.zeros((T, E))
    for t in range(T):
        m = logits[t].astype(np.float64).max()
        if m == -np.inf:
            continue
        p = np.exp(logits[t].astype(np.float64) - m)
        p /= p.sum()
        d = np.zeros(E)
        for j, e in enumerate(ids[t]):
            if 0 <= e < E:
                d[e] += float(dweights[t, j])
        dl[t] = p * (d - p @ d)
    return dl


def swiglu_backward(g, u, dh):
    """(dg, du, h) in fp64."""
    g, u, dh = (np.asarray(a, np.float64) for a in (g, u, dh))
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return dh * u * s * (1.0 + g * (1.0 - s)), dh * g * s, g * s * u


def dgrad(dc, offsets, w, N: int) -> np.ndarray:
    """Rows offsets[0] .. offsets[-1] of dA, w [E*N, K] dequantized."""
    out = np.zeros((dc.shape[0], w.shape[1]))
    for e in range(len(offsets) - 1):
        a, b = offsets[e], offsets[e + 1]
        out[a:b] = dc[a:b].astype(np.float64) @ w[e * N:(e + 1) * N].astype(np.float64)
    return out


def wgrad(dc, a, gather, offsets) -> np.ndarray:
    """[E*N, K]; gather entries outside a's rows read zeros."""
    N, K = dc.shape[1], a.shape[1]
    E = len(offsets) - 1
    out = np.zeros((E * N, K))
    rows = np.arange(dc.shape[0]) if gather is None else np.asarray(gather, np.int64)
    ok = (rows >= 0) & (rows < a.shape[0])
    x = np.where(ok[:, None], a[np.where(ok, rows, 0)].astype(np.float64), 0.0)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        out[e * N:(e + 1) * N] = dc[lo:hi].astype(np.float64).T @ x[lo:hi]
    return out
