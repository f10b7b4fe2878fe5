"""The norm, the router's balance loss, the 8-bit product and the clipping together, as a block's serving and training
steps use them: each new result against the oracle on the very tensors that the step gave it, the whole step captured
into graphs, and every call on a stream of its own."""
import numpy as np
import pytest
import torch

import w4_gemm_amd as q4
from oracle import block as ob

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
T, K, E, I, CHOICES = 96, 512, 8, 128, 2


def n64(t):
    return t.detach().cpu().double().numpy()


def near(got, ref, rel, floor=0.0):
    assert np.all(np.abs(n64(got) - ref) <= rel * np.abs(ref) + floor), float(np.max(np.abs(n64(got) - ref)))


class Layer:
    """A norm and an MoE layer behind it, on 4-bit expert weights, with a balance loss on its router."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.x, self.res, self.dout, self.dres = ((torch.randn(T, K, generator=g) * s).to(BF16).cuda()
                                                  for s in (1.0, 2.0, 0.1, 0.1))
        self.norm = (1 + 0.1 * torch.randn(K, generator=g)).cuda()
        self.router = (torch.randn(E, K, generator=g) * 0.05).cuda()
        self.gu = q4.quantize((torch.randn(E * 2 * I, K, generator=g) * 0.05).to(BF16).cuda(), "mxfp4", layout="tiled")
        self.down = q4.quantize((torch.randn(E * K, I, generator=g) * 0.05).to(BF16).cuda(), "mxfp4")
        self.mask = (torch.rand(T, generator=g) < 0.8).cuda()

    def step(self):
        h, y, _ = q4.q4_rmsnorm(self.x, self.norm, EPS, residual=self.res)
        logits = y.float() @ self.router.t()
        out, saved = q4.moe_layer_save(y, logits, CHOICES, self.gu, self.down, I)
        loss, counts, slopes = q4.q4_moe_balance(logits, saved.r.ids, 0.01, mask=self.mask)
        dy, dlogits, dgu, ddown = q4.moe_layer_backward(saved, self.dout, self.gu, self.down)
        gates = dlogits.clone()
        q4.q4_moe_balance_backward(logits, slopes, mask=self.mask, dlogits=dlogits, accumulate=True)
        drouter = dlogits.t() @ y.float()
        dy = (dy.float() + dlogits @ self.router).to(BF16)
        dx, dnorm = q4.q4_rmsnorm_backward(dy, h, self.norm, EPS, dh=self.dres)
        before = [t.clone() for t in (dgu, ddown, drouter, dnorm)]
        norm = q4.q4_grad_clip([dgu, ddown, drouter, dnorm], 0.05)
        return {"h": h, "y": y, "logits": logits, "ids": saved.r.ids, "loss": loss, "counts": counts, "gates": gates,
                "dlogits": dlogits, "dy": dy, "dx": dx, "before": before, "after": [dgu, ddown, drouter, dnorm],
                "norm": norm, "out": out}


def flat(r):
    return [t for v in r.values() for t in (v if isinstance(v, list) else [v])]


def test_training_step():
    layer = Layer()
    r = layer.step()
    torch.cuda.synchronize()
    h = (layer.x.float() + layer.res.float()).to(BF16)
    assert torch.equal(r["h"], h)
    near(r["y"], ob.rmsnorm(n64(h), n64(layer.norm), EPS), 2.0 ** -8 + 2.0 ** -18)
    loss, counts, slopes = ob.moe_balance(n64(r["logits"]), r["ids"].cpu().numpy(), 0.01, layer.mask.cpu().numpy())
    assert np.array_equal(counts, r["counts"].cpu().numpy()) and counts.sum() == CHOICES * int(layer.mask.sum())
    near(r["loss"], loss, 2.0 ** -16)
    add = ob.moe_balance_backward(n64(r["logits"]), slopes, layer.mask.cpu().numpy())
    near(r["dlogits"], n64(r["gates"]) + add, 2.0 ** -23, 2.0 ** -15 * slopes.max())
    dx, dn = ob.rmsnorm_backward(n64(r["dy"]), n64(h), n64(layer.norm), EPS)
    dx += n64(layer.dres)
    near(r["dx"], dx, 2.0 ** -8, 2.0 ** -15 * np.abs(dx).max())
    near(r["before"][3], dn, 0.0, 2.0 ** -16 * np.abs(n64(r["dy"])).sum(0).max() * 8)
    norm = ob.grad_norm([n64(t) for t in r["before"]])
    assert norm > 0.05
    near(r["norm"], norm, 2.0 ** -22)
    for a, b in zip(r["after"], ob.grad_clip([n64(t) for t in r["before"]], 0.05, norm)):
        near(a, b, 2.0 ** -22, 2.0 ** -149)


def test_two_graphs_in_turn():
    """Two captured steps, replayed one after the other with new inputs and eager work in between."""
    layers = [Layer(1), Layer(2)]
    for l in layers:
        l.step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for l in layers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(l.step())
        graphs.append(g)
    for i in range(3):
        for l in layers:
            l.x.copy_(torch.randn(T, K).to(BF16))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for l, o in zip(layers, outs):
            for a, b in zip(flat(o), flat(l.step())):
                assert torch.equal(a, b), i


def test_serving_step():
    """Norm in 8 bits and the products behind it, for one token and for some."""
    g = torch.Generator().manual_seed(4)
    W = q4.quantize((torch.randn(1000, 1024, generator=g) * 0.05).to(BF16).cuda(), "int8_row")
    wd = n64(q4.q4_dequant(W, torch.empty(1000, 1024, dtype=F32, device="cuda")))
    w = (1 + 0.1 * torch.randn(1024, generator=g)).to(BF16).cuda()
    for rows in (1, 7, 130):
        x, res = (torch.randn(rows, 1024, generator=g).to(BF16).cuda() for _ in range(2))
        a = q4.empty_q4("int8_row", rows, 1024)
        h, _, _ = q4.q4_rmsnorm(x, w, EPS, residual=res, h=res, y_q=a)
        assert h is res
        C = q4.q4_gemm(a, W, torch.empty(rows, 1000, dtype=BF16, device="cuda"))
        y = ob.rmsnorm(n64(h), n64(w), EPS)
        exact = y @ wd.T
        # half a code of the activations (1/254 of the row's largest) at random signs, and bf16
        off = np.abs(n64(C) - exact)
        size = np.abs(y).max(1, keepdims=True) / 254 * np.sqrt((wd ** 2).sum(1))[None, :]
        assert np.all(off <= 2.0 ** -8 * np.abs(exact) + 6 * size)
        ad = n64(q4.q4_dequant(a, torch.empty(rows, 1024, dtype=F32, device="cuda")))
        near(C, ad @ wd.T, 2.0 ** -8, 2.0 ** -20 * (np.abs(ad) @ np.abs(wd).T))


def test_a_stream_that_is_named():
    """Every call with stream=, while the current stream is another."""
    layer = Layer(3)
    want_h, want_y, _ = q4.q4_rmsnorm(layer.x, layer.norm, EPS, residual=layer.res)
    logits = torch.randn(T, E, device="cuda")
    ids, _ = q4.q4_moe_topk(logits, CHOICES)
    want_b = q4.q4_moe_balance(logits, ids)
    want_d = q4.q4_moe_balance_backward(logits, want_b[2])
    want_g = q4.q4_rmsnorm_backward(layer.dout, want_h, layer.norm, EPS)
    grads = [torch.randn(1000, device="cuda"), torch.randn(77, device="cuda")]
    want_c = [torch.empty_like(t) for t in grads]
    want_n = q4.q4_grad_clip(grads, 1.0, out=want_c)
    A = q4.quantize(layer.x, "int8_row")
    C = q4.q4_gemm(A, A, torch.empty(T, T, dtype=BF16, device="cuda"))
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        got = q4.q4_rmsnorm(layer.x, layer.norm, EPS, residual=layer.res, stream=s)
        b = q4.q4_moe_balance(logits, ids, stream=s)
        d = q4.q4_moe_balance_backward(logits, b[2], stream=s)
        g = q4.q4_rmsnorm_backward(layer.dout, got[0], layer.norm, EPS, stream=s)
        c = [torch.empty_like(t) for t in grads]
        n = q4.q4_grad_clip(grads, 1.0, out=c, stream=s)
        n2 = q4.q4_grad_norm(grads, stream=s)
        A2 = q4.quantize(layer.x, "int8_row", stream=s)
        C2 = q4.q4_gemm(A2, A2, torch.empty(T, T, dtype=BF16, device="cuda"), stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want_h) and torch.equal(got[1], want_y)
        assert all(torch.equal(p, q) for p, q in zip(b, want_b)) and torch.equal(d, want_d)
        assert all(torch.equal(p, q) for p, q in zip(g, want_g))
        assert torch.equal(n, want_n) and torch.equal(n2, want_n) and all(torch.equal(p, q) for p, q in zip(c, want_c))
        assert torch.equal(A2.codes, A.codes) and torch.equal(C2, C)


@pytest.mark.parametrize("allocates", [True, False])
def test_a_handle_of_zero_is_the_default_stream(allocates):
    """stream=0 inside another stream's context: the default stream, not a new one."""
    from w4_gemm_amd.grad import _place
    x = torch.ones(8, device="cuda")
    with torch.cuda.stream(torch.cuda.Stream()):
        with _place(0, ("x", x), allocates=allocates) as (_, s):
            assert s == torch.cuda.default_stream().cuda_stream == 0
            if allocates:
                assert torch.cuda.current_stream().cuda_stream == 0


def test_stream_zero_is_in_order_with_the_default_stream():
    """Fills on the default stream, then calls with stream=0 and with nothing between: each sees the fill before it."""
    src = torch.zeros(4096, 2048, dtype=BF16, device="cuda")
    dst, back = q4.empty_q4("int8_row", 4096, 2048), torch.empty(4096, 2048, dtype=F32, device="cuda")
    grads = [torch.empty(1 << 24, device="cuda")]
    torch.cuda.synchronize()
    got = []
    for i in range(1, 9):
        for _ in range(8):
            src.fill_(float(i))
            grads[0].fill_(float(i))
        q4.q4_quantize(src, dst, stream=0)
        q4.q4_dequant(dst, back, stream=0)
        norm = q4.q4_grad_norm(grads, stream=0)
        got.append((back.amin(), back.amax(), norm))
    torch.cuda.synchronize()
    for i, (lo, hi, norm) in enumerate(got, 1):
        assert abs(lo.item() - i) <= i * 2.0 ** -22 and abs(hi.item() - i) <= i * 2.0 ** -22
        assert norm.item() == i * 4096.0


def test_calls_at_once():
    """Two threads with a stream each, every call with a workspace or a shared counter: the results of one alone."""
    import threading
    sizes = [(700, 2048), (900, 4096)]
    g = torch.Generator().manual_seed(5)
    sets = []
    for rows, cols in sizes:
        x, dy = (torch.randn(rows, cols, generator=g).to(BF16).cuda() for _ in range(2))
        logits = torch.randn(9000, 200, generator=g).cuda()
        ids, _ = q4.q4_moe_topk(logits, 4)
        grads = [torch.randn(n, generator=g).cuda() for n in (rows * cols, 5, 70001)]
        sets.append((x, dy, torch.rand(cols, generator=g).cuda(), logits, ids, grads))

    def calls(x, dy, w, logits, ids, grads):
        out = [torch.empty_like(t) for t in grads]
        a = q4.empty_q4("int8_row", *x.shape)
        q4.q4_rmsnorm(x, w, EPS, y_q=a)
        C = q4.q4_gemm(a, a, torch.empty(x.shape[0], x.shape[0], dtype=BF16, device="cuda"))
        return (*q4.q4_rmsnorm_backward(dy, x, w, EPS), *q4.q4_moe_balance(logits, ids),
                q4.q4_grad_clip(grads, 1.0, out=out), *out, C)

    want = [[t.clone() for t in calls(*s)] for s in sets]
    torch.cuda.synchronize()
    bad, errors = [], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()) as _:
                for _ in range(20):
                    got = calls(*sets[i])
                    bad.append(sum((p != q).sum() for p, q in zip(got, want[i])))
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # (shown in the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and len(bad) == 40 and all(int(b) == 0 for b in bad)
