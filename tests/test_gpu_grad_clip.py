"""The gradients' norm and their clipping on the GPU against the oracle.

Squares are exact in 64 bits and added there, so the norm is off by its rounding
to fp32 (2^-24; 2^-22 allows for the sums' 2^-53 each).  An output has the
factor's rounding and its own: 2^-22 in fp32, 2^-8 + 2^-22 in bf16, and half the
least number of the type where it vanishes.
"""
import numpy as np
import pytest
import torch

import w4_gemm_amd as q4
from oracle import block as ob

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(sizes, seed=0, shift=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        kind = BF16 if i % 3 == 1 else F32
        out.append((torch.randn(n + shift, generator=g) * scale).to(kind).cuda()[shift:])
    return out


def n64(grads):
    return [g.detach().cpu().double().numpy().reshape(-1) for g in grads]


def check_out(got, ref):
    for a, b in zip(got, ref):
        rel, least = (2.0 ** -22, 2.0 ** -149) if a.dtype is F32 else (2.0 ** -8 + 2.0 ** -22, 2.0 ** -133)
        d = np.abs(a.detach().cpu().double().numpy().reshape(-1) - b)
        assert np.all(d <= rel * np.abs(b) + least), (a.shape, a.dtype)


def check(grads, max_norm):
    ref = n64(grads)
    norm = ob.grad_norm(ref)
    got = q4.q4_grad_norm(grads)
    assert got.shape == () and abs(got.item() - norm) <= 2.0 ** -22 * norm
    want = ob.grad_clip(ref, max_norm, norm)
    out = [torch.full_like(g, 9.0) for g in grads]
    n2 = q4.q4_grad_clip(grads, max_norm, out=out)
    assert torch.equal(n2, got)
    check_out(out, want)
    for g, r in zip(grads, ref):
        assert np.array_equal(g.cpu().double().numpy().reshape(-1), r)      # untouched
    n3 = q4.q4_grad_clip(grads, max_norm)
    assert torch.equal(n3, got)
    for a, b in zip(grads, out):
        assert torch.equal(a, b)


SIZES = [[1], [2], [3, 1, 2], [7, 8, 9], [15, 16, 17], [255, 256, 257], [1000, 0, 5], [8191, 8192, 8193],
         [16383, 16384, 16385, 1], [100003, 65536, 33], list(range(1, 60))]


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s[:4])))
def test_sizes_and_alignment(sizes, shift):
    for max_norm in (0.5, 1e9):
        check(make(sizes, len(sizes), shift), max_norm)


@pytest.mark.parametrize("count", [127, 128, 129, 300])
def test_many_tensors(count):
    """More tensors than a launch takes."""
    rng = np.random.default_rng(count)
    check(make([int(n) for n in rng.integers(0, 3000, count)], count), 1.0)


def test_large():
    g = [torch.randn(5000, 4099, device="cuda"), torch.randn(3, 1 << 20, device="cuda").to(BF16)]
    norm = torch.sqrt(sum(t.double().square().sum() for t in g)).item()
    keep = [t.clone() for t in g]
    got = q4.q4_grad_clip(g, 1.0)
    assert abs(got.item() - norm) <= 2.0 ** -22 * norm
    by = 1.0 / (norm + 1e-6)
    for a, b in zip(g, keep):
        rel = 2.0 ** -22 if a.dtype is F32 else 2.0 ** -8 + 2.0 ** -22
        assert ((a.double() - b.double() * by).abs() <= rel * b.double().abs() * by + 2.0 ** -133).all()


def test_longer_than_the_caches():
    """More bytes than are kept between the two passes, in tensors of both types with odd beginnings."""
    buf = torch.randn(70_000_003, device="cuda")
    g = [buf[3:69_999_990], torch.randn(9_000_001, device="cuda").to(BF16)[1:], buf[69_999_990:]]
    keep = [t.clone() for t in g]
    norm = torch.sqrt(sum(t.double().square().sum() for t in g)).item()
    got = q4.q4_grad_clip(g, 2.0)
    assert abs(got.item() - norm) <= 2.0 ** -22 * norm and torch.equal(buf[:3], buf[:3].clone())
    by = 2.0 / (norm + 1e-6)
    for a, b in zip(g, keep):
        rel = 2.0 ** -22 if a.dtype is F32 else 2.0 ** -8 + 2.0 ** -22
        assert ((a.double() - b.double() * by).abs() <= rel * b.double().abs() * by + 2.0 ** -133).all()


def test_past_32_bits():
    """A tensor of more than 2^31 values: its last ones are counted and scaled."""
    n = (1 << 31) + 40
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[0], g[n - 1], g[1 << 31] = 3.0, 4.0, 12.0
    norm = q4.q4_grad_clip([g], 6.5)
    assert norm.item() == 13.0
    assert abs(g[n - 1].item() - 2.0) < 0.01 and abs(g[1 << 31].item() - 6.0) < 0.03 and g[0].item() == 1.5
    assert g[1:1000].eq(0).all() and g[-1000:-41].eq(0).all()


def test_extremes():
    big = [torch.full((1000,), 3e38, device="cuda"), torch.full((10,), 1e-30, device="cuda")]
    ref = n64(big)
    norm = ob.grad_norm(ref)                    # past fp32's range
    got = q4.q4_grad_clip(big, 1.0)
    assert torch.isinf(got)
    check_out(big, ob.grad_clip(ref, 1.0, norm))
    small = [torch.full((1000,), 1e-30, device="cuda")]
    check(small, 1e-30)
    zero = [torch.zeros(77, device="cuda"), torch.zeros(3, device="cuda", dtype=BF16)]
    assert q4.q4_grad_clip(zero, 1.0).item() == 0 and (zero[0] == 0).all()
    g = make([100, 50])
    assert q4.q4_grad_clip(g, 0.0).item() > 0 and all((t == 0).all() for t in g)
    g = make([100, 50])
    keep = [t.clone() for t in g]
    q4.q4_grad_clip(g, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(g, keep))


def test_infinity_and_nan():
    g = make([100, 200, 300])
    g[1][5] = float("inf")
    assert torch.isinf(q4.q4_grad_norm(g))
    q4.q4_grad_clip(g, 1.0)
    assert torch.isnan(g[1][5]) and (g[0] == 0).all() and (g[2] == 0).all() and torch.isnan(g[1]).sum() == 1
    g = make([100, 200, 300])
    g[2][299] = float("nan")
    assert torch.isnan(q4.q4_grad_norm(g))
    q4.q4_grad_clip(g, 1.0)
    assert all(torch.isnan(t).all() for t in g)


def test_given_norm_and_partial_in_place():
    g = make([1000, 2000, 3001], 5)
    ref = n64(g)
    out = [g[0], torch.empty_like(g[1]), g[2]]
    given = torch.tensor(250.0, device="cuda")
    back = q4.q4_grad_clip(g, 25.0, norm=given, out=out)
    assert back is given and given.item() == 250.0
    check_out(out, ob.grad_clip(ref, 25.0, 250.0))


def test_outputs_of_other_alignment():
    g = make([5000, 5001, 5002], 6)
    ref = n64(g)
    out = [torch.zeros(t.numel() + 3, dtype=t.dtype, device="cuda")[i + 1:][:t.numel()] for i, t in enumerate(g)]
    norm = q4.q4_grad_clip(g, 1.0, out=out)
    check_out(out, ob.grad_clip(ref, 1.0, ob.grad_norm(ref)))
    assert norm.item() > 1


def test_tensors_side_by_side():
    """Gradients that are pieces of one buffer: nothing beside them changes."""
    buf = torch.randn(10007, device="cuda")
    keep = buf.clone()
    g = [buf[1:1000], buf[1000:1003], buf[2001:9000]]
    norm = ob.grad_norm(n64(g))
    q4.q4_grad_clip(g, 1.0)
    by = 1.0 / (norm + 1e-6)
    for a, b in ((0, 1), (1003, 2001), (9000, 10007)):
        assert torch.equal(buf[a:b], keep[a:b])
    for a, b in ((1, 1003), (2001, 9000)):
        assert torch.allclose(buf[a:b], keep[a:b] * by, rtol=1e-6)


def test_same_every_time_graph_and_streams():
    base = make([50000, 777, 1 << 18, 3], 7)

    def step():
        out = [torch.empty_like(t) for t in base]
        return [q4.q4_grad_clip(base, 0.5, out=out), *out]

    first = step()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(4):
        for t in base:
            t.copy_(torch.randn(t.numel()))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))
    want = step()
    torch.cuda.synchronize()
    got = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        with torch.cuda.stream(s):
            got += [step() for _ in range(5)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_behind_the_weight_gradients():
    """dW of a product as the framework writes it, clipped in place with a norm's weight gradient."""
    g = torch.Generator().manual_seed(1)
    dc, a = torch.randn(64, 256, generator=g).to(BF16).cuda(), torch.randn(64, 512, generator=g).to(BF16).cuda()
    dw = q4.q4_gemm_wgrad(dc, q4.quantize(a, "mxint8"))
    _, dn = q4.q4_rmsnorm_backward(a, a, torch.ones(512, dtype=BF16).cuda())
    check([dw, dn], 1.0)
