"""Pins of the backward definitions in oracle/grad.py: differences of the
forward definitions, closed forms, and torch's E4M3 cast."""
import numpy as np
import pytest
import torch

import oracle
from oracle import grad

RNG = np.random.default_rng(7)


def _diff(f, x, eps=1e-5):
    """Gradient of the scalar f at x by central differences."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


def test_swiglu_backward_is_the_forwards_difference():
    g, u, dh = RNG.standard_normal((3, 6)) * 3, RNG.standard_normal((3, 6)), RNG.standard_normal((3, 6))
    dg, du, h = grad.swiglu_backward(g, u, dh)
    ref = oracle.swiglu(np.concatenate((g, u), 1), 6)
    assert np.allclose(h, ref, rtol=1e-12)
    f = lambda gg, uu: float((oracle.swiglu(np.concatenate((gg, uu), 1), 6) * dh).sum())  # noqa: E731
    assert np.allclose(dg, _diff(lambda v: f(v, u), g), atol=1e-8)
    assert np.allclose(du, _diff(lambda v: f(g, v), u), atol=1e-8)


def test_topk_backward_is_the_softmaxs_difference():
    lg = RNG.standard_normal((4, 7))
    ids = np.array([[0, 3], [6, -1], [2, 2], [7, 1]])      # a dropped, a repeated, an unknown one
    dw = RNG.standard_normal((4, 2))

    def f(v):
        p = np.exp(v) / np.exp(v).sum(1, keepdims=True)
        return sum(dw[t, j] * p[t, e] for t in range(4) for j, e in enumerate(ids[t]) if 0 <= e < 7)

    assert np.allclose(grad.topk_backward(lg, ids, dw), _diff(f, lg), atol=1e-8)
    assert np.all(grad.topk_backward(np.full((1, 3), -np.inf), ids[:1], dw[:1]) == 0)


def test_combine_and_permute_backward_are_differences():
    ids = np.array([[1, 0], [2, -1], [1, 3], [0, 1]])
    offsets, gather, inv = grad.moe_sort(ids, 4)
    P, N = int(offsets[-1]), 5
    w, y, dout = RNG.random((4, 2)), RNG.standard_normal((P, N)), RNG.standard_normal((4, N))

    def out(ww, yy):
        return sum(ww[t, j] * (yy[inv[t, j]] @ dout[t]) for t in range(4) for j in range(2) if inv[t, j] >= 0)

    dy, dw = grad.combine_backward(dout, y, inv, w, np.zeros((P, N)))
    assert np.allclose(dy, _diff(lambda v: out(w, v), y), atol=1e-8)
    assert np.allclose(dw, _diff(lambda v: out(v, y), w), atol=1e-8)
    x, dxs = RNG.standard_normal((4, N)), RNG.standard_normal((P, N))
    f = lambda v: float((grad.permute(v, inv, np.zeros((P, N))) * dxs).sum())  # noqa: E731
    assert np.allclose(grad.permute_backward(dxs, inv), _diff(f, x), atol=1e-8)


def test_product_gradients_are_differences():
    offsets, gather = np.array([0, 2, 2, 5]), np.array([1, 0, 2, 2, 9])    # an empty expert, an index out of range
    N, K = 3, 4
    w, a, dc = RNG.standard_normal((3 * N, K)), RNG.standard_normal((3, K)), RNG.standard_normal((5, N))
    rows = np.where((gather < 3)[:, None], a[np.minimum(gather, 2)], 0.0)

    def f(r, ww):
        return sum(dc[p] @ (ww[e * N:(e + 1) * N] @ r[p]) for e in range(3) for p in range(offsets[e], offsets[e + 1]))

    assert np.allclose(grad.dgrad(dc, offsets, w, N), _diff(lambda v: f(v, w), rows), atol=1e-8)
    assert np.allclose(grad.wgrad(dc, a, gather, offsets), _diff(lambda v: f(rows, v), w), atol=1e-8)


def test_sort_matches_the_routings_dispatch():
    lg = RNG.standard_normal((37, 16)).astype(np.float32)
    r = oracle.moe_route(lg, 4)
    offsets, gather, inv = grad.moe_sort(r.ids, 16)
    assert np.array_equal(offsets, r.offsets) and np.array_equal(gather, r.gather) and np.array_equal(inv, r.inv)


def test_mxfp8_codes_are_torchs_e4m3_cast():
    x = torch.from_numpy(RNG.standard_normal((4, 64)).astype(np.float32) * 3).bfloat16().float().numpy()
    codes, scales = grad.mx8_quantize("mxfp8", x)
    s = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, axis=1)
    ref = torch.from_numpy((x / s).astype(np.float32)).to(torch.float8_e4m3fn)
    assert np.array_equal(codes, ref.view(torch.uint8).numpy())


@pytest.mark.parametrize("fmt", ("mxint8", "mxfp8"))
def test_mx8_scale_is_the_least_that_does_not_clip(fmt):
    top = grad.MX8_TOP[fmt]
    x = np.zeros((6, 32), np.float32)
    x[0, 3] = top            # exactly the top: scale 1
    x[1, 3] = -top * 2       # scale 2
    x[2, 3] = np.float32(top + top / 127) if fmt == "mxint8" else 480.0   # the next bf16: scale 2
    x[3, 3] = 2.0 ** -130    # far below the least scale
    x[4, 3] = np.nan
    x[5, :] = torch.full((32,), torch.finfo(torch.bfloat16).max).numpy()
    codes, scales = grad.mx8_quantize(fmt, x)
    assert list(scales[:, 0]) == [127, 128, 128, 16, 255, 249 if fmt == "mxint8" else 247]
    v = grad.mx8_dequant(fmt, codes, scales)
    assert v[0, 3] == top and v[1, 3] == -2 * top and np.all(np.isnan(v[4])) and np.all(np.isfinite(v[5]))
    y = RNG.standard_normal((8, 64)).astype(np.float32)
    y = torch.from_numpy(y).bfloat16().float().numpy()
    codes, scales = grad.mx8_quantize(fmt, y)
    v, s = grad.mx8_dequant(fmt, codes, scales), np.repeat(2.0 ** (scales.astype(float) - 127), 32, axis=1)
    assert np.all(np.abs(y) <= top * s) and np.all(np.abs(y).reshape(8, 2, 32).max(2) > top / 2 * s[:, ::32])
    assert np.all(np.abs(v - y) <= (s / 2 if fmt == "mxint8" else np.maximum(np.abs(y) * 2.0 ** -4, s * 2.0 ** -10)))
