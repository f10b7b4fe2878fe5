"""The oracle of the norm, of rows in 8-bit integers and of their product, against differences and by hand."""
import numpy as np

from oracle import block as ob


def test_rmsnorm_by_hand():
    y = ob.rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    r = np.sqrt(12.5)
    assert np.allclose(y, [[3 / r, 8 / r]], rtol=1e-15)


def test_rmsnorm_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, w, dy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    eps, step = 0.1, 1e-6
    dx, dw = ob.rmsnorm_backward(dy, x, w, eps)
    f = lambda x, w: float(np.sum(dy * ob.rmsnorm(x, w, eps)))  # noqa: E731
    for a, g in ((x, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + step
            up = f(x, w)
            a[i] = keep - step
            down = f(x, w)
            a[i] = keep
            # central differences: the third derivative (below 100 here) times step^2, and rounding 2^-50 / step
            assert abs((up - down) / (2 * step) - g[i]) < 1e-8


def test_int8_rows_by_hand():
    c, s = ob.int8_rows(np.array([[127.0, -63.5, 0.5, 1.5, -2.5, 0.0], [0, 0, 0, 0, 0, 0]], np.float32))
    assert c.tolist() == [[127, -64, 0, 2, -2, 0], [0] * 6]      # ties to even
    assert s[0] == 1.0 and s[1] == np.float32(1e-12) / np.float32(127)


def test_int8_rows_largest_is_127():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((2000, 4)) * 10.0 ** rng.uniform(-10, 30, (2000, 1))).astype(np.float32)
    c, s = ob.int8_rows(x)
    assert (np.abs(c.astype(int)).max(1) == 127).all()
    # every value within half a scale, and what 127 / a and a / 127 were rounded by (2^-24 each of 127 scales)
    assert (np.abs(c * s[:, None].astype(np.float64) - x) <= (0.5 + 127 * 2.0 ** -22) * s[:, None]).all()


def test_int8_product_by_hand():
    out = ob.int8_product(np.array([[1, -2]], np.int8), np.array([0.5], np.float32), np.array([[3, 4], [-128, 1]], np.int8),
                          np.array([2.0, 1.0], np.float32))
    assert out.tolist() == [[-5.0, -65.0]]


def test_balance_by_hand():
    logits = np.zeros((4, 2))
    loss, counts, slopes = ob.moe_balance(logits, np.array([[0], [1], [0], [1]]), 0.5)
    assert loss == 0.5 and counts.tolist() == [2, 2]               # spread evenly: coef
    loss, counts, _ = ob.moe_balance(logits, np.array([[0], [0], [0], [5]]), 1.0, mask=[1, 1, 0, 1])
    assert counts.tolist() == [2, 0] and np.isclose(loss, 2 * (2 / 3) * 0.5)
    assert ob.moe_balance(logits, np.zeros((4, 1), int), 1.0, mask=[0] * 4)[0] == 0.0


def test_balance_gradient_against_differences():
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((5, 6))
    logits[1, 2] = -np.inf
    ids = np.stack([rng.permutation(6)[:2] for _ in range(5)])
    mask = [1, 1, 0, 1, 1]
    _, _, slopes = ob.moe_balance(logits, ids, 1.5, mask)
    g = ob.moe_balance_backward(logits, slopes, mask, 2.0)
    for i in np.ndindex(logits.shape):
        if np.isinf(logits[i]):
            assert g[i] == 0
            continue
        keep, step = logits[i], 1e-6
        logits[i] = keep + step
        up = ob.moe_balance(logits, ids, 1.5, mask)[0]
        logits[i] = keep - step
        down = ob.moe_balance(logits, ids, 1.5, mask)[0]
        logits[i] = keep
        assert abs(2.0 * (up - down) / (2 * step) - g[i]) < 1e-8


def test_clip_by_hand():
    g = [np.array([3.0]), np.array([4.0, 0.0])]
    assert ob.grad_norm(g) == 5.0
    out = ob.grad_clip(g, 2.5, 5.0)
    assert np.allclose(out[0], 1.5, rtol=1e-6) and np.allclose(out[1], [2.0, 0.0], rtol=1e-6)
    assert ob.grad_clip(g, 10.0, 5.0)[0] == 3.0
