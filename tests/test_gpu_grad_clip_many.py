"""Clipping a step of many tensors: its time grows with their number and not with
its square, its norm is the one that the norm's own call makes, and what lies
beside the gradients stays as it is.
"""
import pytest
import torch

import w4_gemm_amd as q4

pytestmark = pytest.mark.gpu
F32 = torch.float32


def time_of(call):
    """Least time of a captured call's replays (its host time left out)."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    best = float("inf")
    for _ in range(4):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def test_time_of_many_tensors():
    """20000 tensors of 256 KB: one call costs what the norm and the clipping by it cost apart (3.8 and 3.7 ms).
    Twice that leaves room for noise; with every workgroup adding all squares again it took 14.7 ms."""
    count, n = 20000, 65536
    grads = list(torch.full((count * n,), 1e-3, device="cuda").split(n))
    out = list(torch.empty(count * n, device="cuda").split(n))
    given = q4.q4_grad_norm(grads)
    alone = time_of(lambda: q4.q4_grad_norm(grads)) + time_of(lambda: q4.q4_grad_clip(grads, 1.0, norm=given, out=out))
    together = time_of(lambda: q4.q4_grad_clip(grads, 1.0, out=out))
    assert together <= 2 * alone, (together, alone)


@pytest.mark.parametrize("count", [1, 127, 128, 129, 256, 257, 700, 3001])
def test_the_norm_is_the_same_in_every_call(count):
    g = torch.Generator(device="cuda").manual_seed(count)
    buf = torch.randn(count * 1000 + 1, device="cuda", generator=g)
    grads = [t[: 1 + 37 * i % 1000] for i, t in enumerate(buf[1:].split(1000))]
    keep = buf.clone()
    norm = q4.q4_grad_norm(grads)
    square = sum(t.double().square().sum() for t in grads)
    want = torch.sqrt(square).item()
    assert abs(norm.item() - want) <= 2.0 ** -22 * want
    out = [torch.full_like(t, 7.0) for t in grads]
    assert torch.equal(q4.q4_grad_clip(grads, 0.5, out=out), norm) and torch.equal(buf, keep)
    by = 0.5 / (want + 1e-6)
    by = min(by, 1.0)
    for t, o in zip(grads[:: max(1, count // 50)], out[:: max(1, count // 50)]):
        assert ((o.double() - t.double() * by).abs() <= 2.0 ** -22 * t.double().abs() * by).all()
    assert torch.equal(q4.q4_grad_clip(grads, 0.5), norm)
    assert all(torch.equal(a, b) for a, b in zip(grads, out))
    inside = torch.zeros_like(buf, dtype=torch.bool)
    for i, t in enumerate(inside[1:].split(1000)):
        t[: 1 + 37 * i % 1000] = True
    assert torch.equal(buf[~inside], keep[~inside])
    # every tensor's values changed by the factor alone (NaN among them goes everywhere)
    grads[-1][0] = float("nan")
    assert torch.isnan(q4.q4_grad_clip(grads, 0.5)) and all(torch.isnan(t).all() for t in grads)
    assert torch.equal(buf[~inside], keep[~inside])


def test_many_in_a_graph():
    """Three launches of squares and of clipping, captured and replayed with other values."""
    buf = torch.randn(300, 500, device="cuda")
    grads = list(buf)

    def step():
        out = [torch.empty_like(t) for t in grads]
        return [q4.q4_grad_clip(grads, 0.25, out=out), *out]

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        buf.copy_(torch.randn(300, 500))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step())), i


def test_what_lies_beside_long_gradients_stays():
    """More bytes than the caches hold, in place: the values in front, between and behind."""
    buf = torch.randn(70_000_009, device="cuda")
    edge = [slice(0, 3), slice(50_000_001, 50_000_004), slice(70_000_002, 70_000_009)]
    grads = [buf[3:50_000_001], buf[50_000_004:70_000_002]]
    keep = [buf[e].clone() for e in edge]
    first = [t[:1000].clone() for t in grads]
    norm = q4.q4_grad_clip(grads, 2.0)
    for e, k in zip(edge, keep):
        assert torch.equal(buf[e], k)
    by = 2.0 / (norm.double() + 1e-6)
    for t, f in zip(grads, first):
        assert ((t[:1000].double() - f.double() * by).abs() <= 2.0 ** -22 * f.double().abs() * by).all()
