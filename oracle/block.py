"""Plain definitions (numpy, fp64) of what stands around the products of a
block: rows in 8-bit integers and their product.  Nothing is shared with the
GPU path.
"""
from __future__ import annotations

import numpy as np


def int8_rows(x: np.ndarray):
    """(codes int8 [rows, cols], scales fp32 [rows]) of fp32 x.  The factor
    127 / a and the scale a / 127 are fp32 quotients; a product of two fp32
    values is exact in fp64, so rint rounds it once, ties to even."""
    codes = np.zeros(x.shape, np.int8)
    scales = np.zeros(x.shape[0], np.float32)
    for r in range(x.shape[0]):
        if not np.all(np.isfinite(x[r])):
            scales[r] = np.nan
            continue
        a = max(np.float32(np.max(np.abs(x[r]), initial=0.0)), np.float32(1e-12))
        f = np.float32(127.0) / a
        codes[r] = np.rint(x[r].astype(np.float64) * np.float64(f)).astype(np.int8)
        scales[r] = a / np.float32(127.0)
    return codes, scales


def int8_product(ac: np.ndarray, asc: np.ndarray, wc: np.ndarray, wsc: np.ndarray) -> np.ndarray:
    """s_a[m] s_w[n] sum_k a[m, k] w[n, k] (fp64; the sum is a whole number
    below 2^53, so exact)."""
    s = ac.astype(np.float64) @ wc.astype(np.float64).T
    return s * asc.astype(np.float64)[:, None] * wsc.astype(np.float64)[None, :]


def rmsnorm(x: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    """x / sqrt(mean(x^2) + eps) * weight of each row (fp64)."""
    out = np.zeros(x.shape)
    for r in range(x.shape[0]):
        v = x[r].astype(np.float64)
        with np.errstate(all="ignore"):
            out[r] = v / np.sqrt(np.sum(v * v) / v.size + eps) * weight.astype(np.float64)
    return out


def rmsnorm_backward(dy: np.ndarray, x: np.ndarray, weight: np.ndarray, eps: float):
    """(dx, dweight) of sum(dy * rmsnorm(x, weight)) from the quotient rule,
    element by element of the definition (fp64)."""
    w = weight.astype(np.float64)
    dx, dw = np.zeros(x.shape), np.zeros(w.shape)
    for r in range(x.shape[0]):
        v, d = x[r].astype(np.float64), dy[r].astype(np.float64)
        root = np.sqrt(np.sum(v * v) / v.size + eps)
        # y_j = w_j v_j / root, d root / d v_k = v_k / (n root)
        dx[r] = d * w / root - np.sum(d * w * v) / root ** 2 * v / (v.size * root)
        dw += d * v / root
    return dx, dw


def softmax(row: np.ndarray) -> np.ndarray:
    """Softmax of one token's logits (fp64); zeros where all are -inf."""
    v = row.astype(np.float64)
    if np.all(v == -np.inf):
        return np.zeros(v.size)
    with np.errstate(invalid="ignore"):
        e = np.exp(v - np.max(v))
        return e / np.sum(e)


def moe_balance(logits: np.ndarray, ids: np.ndarray, coef: float, mask=None):
    """(loss, counts, slopes) over the tokens that count."""
    T, E = logits.shape
    k = ids.shape[1]
    here = [t for t in range(T) if mask is None or mask[t]]
    counts, total = np.zeros(E, np.int64), np.zeros(E)
    for t in here:
        for e in ids[t]:
            if 0 <= e < E:
                counts[e] += 1
        total += softmax(logits[t])
    n = len(here)
    slopes = coef * E * counts / (k * float(n) * n) if n else np.zeros(E)
    return float(np.sum(slopes * total)), counts, slopes


def moe_balance_backward(logits: np.ndarray, slopes: np.ndarray, mask=None, dloss: float = 1.0) -> np.ndarray:
    """Gradient of the loss for the logits, by the softmax's matrix of
    derivatives dp_e / dl_j = p_e ([e = j] - p_j)."""
    out = np.zeros(logits.shape)
    for t in range(logits.shape[0]):
        if mask is None or mask[t]:
            p = softmax(logits[t])
            out[t] = dloss * ((np.diag(p) - np.outer(p, p)) @ slopes)
    return out


def grad_norm(grads) -> float:
    return float(np.sqrt(sum(np.sum(g.astype(np.float64) ** 2) for g in grads)))


def grad_clip(grads, max_norm: float, norm: float):
    with np.errstate(invalid="ignore"):
        by = max_norm / (norm + 1e-6)
        by = 1.0 if by > 1 else by
        return [g.astype(np.float64) * by for g in grads]
