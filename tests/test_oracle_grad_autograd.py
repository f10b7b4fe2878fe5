"""The backward definitions in oracle/grad.py against torch's differentiation
of the forward definitions, on the CPU in 64 bits: equal to 1e-12 of the
largest value (sums of at most 40 terms, each rounding 2^-53)."""
import numpy as np
import torch

from oracle import grad

RNG = np.random.default_rng(11)


def _leaf(*shape):
    return torch.from_numpy(RNG.standard_normal(shape)).requires_grad_()


def _equal(got, want, what):
    want = want.detach().numpy()
    assert got.shape == want.shape, what
    assert np.all(np.abs(got - want) <= 1e-12 * max(1.0, np.abs(want).max())), what


def test_swiglu():
    g, u, dh = _leaf(5, 8), _leaf(5, 8), RNG.standard_normal((5, 8))
    h = g * torch.sigmoid(g) * u
    h.backward(torch.from_numpy(dh))
    dg, du, again = grad.swiglu_backward(g.detach().numpy(), u.detach().numpy(), dh)
    _equal(dg, g.grad, "dg")
    _equal(du, u.grad, "du")
    _equal(again, h, "h")


def test_gates():
    lg = _leaf(4, 7)
    ids = np.array([[0, 3], [6, -1], [2, 2], [7, 1]])      # a dropped, a repeated, an unknown choice
    dw = RNG.standard_normal((4, 2))
    p = torch.softmax(lg, 1)
    sum(dw[t, j] * p[t, e] for t in range(4) for j, e in enumerate(ids[t]) if 0 <= e < 7).backward()
    _equal(grad.topk_backward(lg.detach().numpy(), ids, dw), lg.grad, "dlogits")


def test_combine_and_permute():
    ids = np.array([[1, 0], [2, -1], [1, 3], [0, 1]])
    offsets, gather, inv = grad.moe_sort(ids, 4)
    P, N = int(offsets[-1]), 6
    w, y, x = _leaf(4, 2), _leaf(P, N), _leaf(4, N)
    dout, dxs = RNG.standard_normal((4, N)), RNG.standard_normal((P, N))
    out = torch.stack([sum(w[t, j] * y[p] for j, p in enumerate(inv[t]) if p >= 0) for t in range(4)])
    out.backward(torch.from_numpy(dout))
    dy, dw = grad.combine_backward(dout, y.detach().numpy(), inv, w.detach().numpy(), np.zeros((P, N)))
    _equal(dy, y.grad, "dy")
    _equal(dw, w.grad, "dw")
    x[torch.from_numpy(gather).long()].backward(torch.from_numpy(dxs))
    _equal(grad.permute_backward(dxs, inv), x.grad, "dx")


def test_products():
    offsets, gather = np.array([0, 2, 2, 5]), np.array([1, 0, 2, 2, 9])    # an empty expert, an index out of range
    N, K = 3, 4
    w, a, dc = _leaf(3 * N, K), _leaf(3, K), RNG.standard_normal((5, N))
    rows = torch.stack([a[i] if i < 3 else torch.zeros(K, dtype=torch.float64) for i in gather])
    rows.retain_grad()
    c = torch.cat([rows[offsets[e]:offsets[e + 1]] @ w[e * N:(e + 1) * N].T for e in range(3)])
    c.backward(torch.from_numpy(dc))
    _equal(grad.dgrad(dc, offsets, w.detach().numpy(), N), rows.grad, "dA")
    _equal(grad.wgrad(dc, a.detach().numpy(), gather, offsets), w.grad, "dW")
