"""The router's balance loss and its gradient on the GPU against the oracle.

A probability is off by the rounding of its exponent (2^-24 of a difference of
logits below 100: 2^-17), the exponential's and the sum's own (below 2^-19):
REL = 2^-16 of each bounds it.  Slopes and the loss are rounded once from 64 bits.
"""
import numpy as np
import pytest
import torch

import w4_gemm_amd as q4
from oracle import block as ob

pytestmark = pytest.mark.gpu
REL = 2.0 ** -16


def make(T, E, k, seed=0, scale=2.0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + E)
    logits = torch.randn(T, E, generator=g) * scale
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int() if T else torch.zeros(0, k).int()
    return logits, ids


def check(logits, ids, coef=1.0, mask=None, dloss=None, pad=0):
    """Runs both calls on (a view of) the logits and compares everything; returns them."""
    T, E = logits.shape
    buf = torch.full((max(T, 1), E + pad), 123.0, device="cuda")
    lg = buf[:T, :E]
    lg.copy_(logits)
    m = None if mask is None else mask.cuda()
    loss, counts, slopes = q4.q4_moe_balance(lg, ids.cuda(), coef, mask=m)
    rl, rc, rs = ob.moe_balance(logits.numpy(), ids.numpy(), coef, None if mask is None else mask.numpy())
    assert loss.shape == () and np.array_equal(counts.cpu().numpy(), rc)
    assert np.all(np.abs(slopes.cpu().double().numpy() - rs) <= 2.0 ** -22 * np.abs(rs))
    assert abs(loss.item() - rl) <= REL * abs(rl)
    d = None if dloss is None else torch.tensor(dloss).cuda()
    out = torch.full((max(T, 1), E + pad), 55.0, device="cuda")
    got = q4.q4_moe_balance_backward(lg, slopes, mask=m, dloss=d, dlogits=out[:T, :E])
    scale = 1.0 if dloss is None else dloss
    ref = ob.moe_balance_backward(logits.numpy(), rs, None if mask is None else mask.numpy(), scale)
    p = np.stack([ob.softmax(r) for r in logits.numpy()]) if T else np.zeros((0, E))
    size = abs(scale) * p * (np.abs(rs) + (p * np.abs(rs)).sum(1, keepdims=True))
    assert np.all(np.abs(got.cpu().double().numpy() - ref) <= REL * size + 1e-38)
    assert (out[:T, E:] == 55.0).all() and (buf[:T, E:] == 123.0).all()
    if mask is not None:
        assert (got[~m.bool()] == 0).all()
    return loss, counts, slopes, got


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (2, 3, 2), (5, 8, 8), (16, 64, 8), (63, 16, 1), (64, 64, 2),
                                   (65, 37, 4), (130, 65, 3), (257, 128, 8), (300, 129, 2), (511, 256, 8), (100, 250, 5),
                                   (77, 257, 3), (40, 512, 32), (33, 1000, 8), (12, 1024, 32), (3000, 64, 8),
                                   (2500, 256, 4), (1025, 62, 2), (513, 100, 4), (300, 1021, 8), (700, 768, 8)])
def test_all(T, E, k):
    logits, ids = make(T, E, k)
    check(logits, ids)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.7
    check(logits, ids, coef=0.01, mask=mask, dloss=-3.0, pad=5)
    check(logits, ids, mask=mask.to(torch.uint8) * 2, pad=4)


def test_long():
    """Many tokens: counts and sums over all workgroups (against torch in 64 bits)."""
    T, E, k = 70001, 64, 8
    logits = torch.randn(T, E, device="cuda")
    ids, _ = q4.q4_moe_topk(logits, k)
    loss, counts, slopes = q4.q4_moe_balance(logits, ids)
    c = torch.bincount(ids.reshape(-1).long(), minlength=E)
    assert torch.equal(counts.long(), c)
    p = torch.softmax(logits.double(), 1)
    s = E * c.double() / (k * float(T) * T)
    assert abs(loss.item() - (s * p.sum(0)).sum().item()) <= REL * loss.item()
    got = q4.q4_moe_balance_backward(logits, slopes)
    inner = (p * s).sum(1, keepdim=True)
    assert ((got.double() - p * (s - inner)).abs() <= REL * p * (s + inner)).all()


def test_masked_and_missing():
    """No token that counts; no tokens; ids outside the range; the same expert twice."""
    logits, ids = make(20, 16, 4)
    loss, counts, slopes, d = check(logits, ids, mask=torch.zeros(20, dtype=torch.bool))
    assert loss.item() == 0 and (counts == 0).all() and (slopes == 0).all() and (d == 0).all()
    loss, counts, slopes, d = check(torch.zeros(0, 16), torch.zeros(0, 4, dtype=torch.int32))
    assert loss.item() == 0 and (counts == 0).all() and d.shape == (0, 16)
    ids[0, 0], ids[1, 1], ids[2, 2], ids[3] = -1, 16, 2 ** 31 - 1, 5
    ids[4] = -2 ** 31
    check(logits, ids)


def test_infinities_and_nan():
    logits, ids = make(40, 33, 3)
    logits[0] = -np.inf                         # no probabilities
    logits[1, 5:] = -np.inf
    logits[2] = torch.finfo(torch.float32).min  # a mask of the lowest value: all alike
    logits[3, 1:] = torch.finfo(torch.float32).min
    loss, _, slopes, d = check(logits, ids)
    assert (d[0] == 0).all() and (d[1, 5:] == 0).all() and torch.isfinite(d).all()
    for bad in (float("nan"), float("inf")):
        hurt = logits.clone()
        hurt[7, 3] = bad
        loss, counts, s2 = q4.q4_moe_balance(hurt.cuda(), ids.cuda())
        assert torch.isnan(loss) and torch.equal(s2, slopes)
        g = q4.q4_moe_balance_backward(hurt.cuda(), s2)
        assert torch.isnan(g[7]).all()
        keep = [t for t in range(40) if t != 7]
        assert torch.equal(g[keep], d[keep])
        mask = torch.ones(40, dtype=torch.bool)
        mask[7] = False                         # masked: what stands there does not matter
        loss, _, s3 = q4.q4_moe_balance(hurt.cuda(), ids.cuda(), mask=mask.cuda())
        assert torch.isfinite(loss)
        assert torch.isfinite(q4.q4_moe_balance_backward(hurt.cuda(), s3, mask=mask.cuda())).all()


def test_accumulate_and_in_step_with_the_gates():
    """The balance gradient on top of the gates' gradient, as a training step has it."""
    logits, _ = make(50, 24, 4, seed=2)
    lg = logits.cuda()
    ids, w = q4.q4_moe_topk(lg, 4)
    dw = torch.randn(50, 4, generator=torch.Generator().manual_seed(1)).cuda()
    gates = q4.q4_moe_topk_backward(lg, ids, dw)
    mask = (torch.arange(50) % 3 != 0).cuda()
    _, _, slopes = q4.q4_moe_balance(lg, ids, 0.01, mask=mask)
    alone = q4.q4_moe_balance_backward(lg, slopes, mask=mask)
    both = gates.clone()
    out = q4.q4_moe_balance_backward(lg, slopes, mask=mask, dlogits=both, accumulate=True)
    assert out is both and torch.equal(both, gates + alone)
    assert torch.equal(both[~mask], gates[~mask])


def test_graph_and_streams():
    """Every replay of a captured pair equals the eager result, and repeats are equal bit for bit."""
    logits, ids = make(1000, 64, 8, seed=3)
    lg, idg = logits.cuda(), ids.cuda()

    def step():
        loss, counts, slopes = q4.q4_moe_balance(lg, idg, 0.1)
        return loss, counts, slopes, q4.q4_moe_balance_backward(lg, slopes, dloss=loss)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        lg.copy_(torch.randn(1000, 64))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), i
    streams, got, want = [torch.cuda.Stream() for _ in range(2)], [], step()
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            got += [step() for _ in range(5)]
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
