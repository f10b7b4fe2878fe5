"""What the balance loss and the clipping of gradients refuse, on the host."""
import ctypes

import pytest
import torch

import w4_gemm_amd as q4

OK, NULL, SHAPE, ALIGN, FMT = 0, -1, -2, -3, -4
B = 0x7F0000000000
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def balance(**kw):
    a = dict(lg=B, ld=64, T=50000, E=64, k=4, ids=B, mask=B, coef=1.0, loss=B, counts=B, slopes=B, ws=B, wb=1 << 20)
    a.update(kw)
    return q4.lib().q4_moe_balance(a["lg"], a["ld"], a["T"], a["E"], a["k"], a["ids"], a["mask"], a["coef"], a["loss"],
                                   a["counts"], a["slopes"], a["ws"], a["wb"], None)


def balance_back(**kw):
    a = dict(lg=B, ld=64, T=8, E=64, mask=B, slopes=B, dloss=B, dl=B, lddl=64, acc=0)
    a.update(kw)
    return q4.lib().q4_moe_balance_backward(a["lg"], a["ld"], a["T"], a["E"], a["mask"], a["slopes"], a["dloss"],
                                            a["dl"], a["lddl"], a["acc"], None)


def test_balance():
    for kw in (dict(T=-1), dict(T=(1 << 26) - 3), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(ld=63),
               dict(T=1 << 26, k=32), dict(wb=0)):
        assert balance(**kw) == SHAPE, kw
    for p in ("lg", "ids", "loss", "counts", "slopes", "ws"):
        assert balance(**{p: None}) == NULL, p
        assert balance(**{p: B + 2}) == ALIGN, p
    n = ctypes.c_size_t()
    assert q4.lib().q4_moe_balance_workspace(50000, 64, ctypes.byref(n)) == OK
    assert balance(wb=n.value - 1) == SHAPE
    assert q4.lib().q4_moe_balance_workspace(8, 64, None) == NULL
    assert q4.lib().q4_moe_balance_workspace(8, 1025, ctypes.byref(n)) == SHAPE
    for kw in (dict(T=-1), dict(T=(1 << 26) - 3), dict(E=0), dict(E=1025), dict(ld=63), dict(lddl=63)):
        assert balance_back(**kw) == SHAPE, kw
    for p in ("lg", "slopes", "dl"):
        assert balance_back(**{p: None}) == NULL
        assert balance_back(**{p: B + 2}) == ALIGN
    assert balance_back(dloss=B + 2) == ALIGN
    assert balance_back(T=0, lg=None) == OK


def clip(spans, out=None, dtypes=None, max_norm=1.0, norm_in=None, ws=B, wb=1 << 24, n=None, norm=B):
    """spans: (address, count) of each gradient."""
    m = len(spans)
    p = (ctypes.c_void_p * max(m, 1))(*[a for a, _ in spans])
    c = (ctypes.c_int64 * max(m, 1))(*[x for _, x in spans])
    d = (ctypes.c_int32 * max(m, 1))(*(dtypes or [1] * m))
    o = None if out is None else (ctypes.c_void_p * max(m, 1))(*out)
    return q4.lib().q4_grad_clip(m if n is None else n, p, c, d, o, norm_in, max_norm, norm, ws, wb, None)


def norm(spans, dtypes=None, out=B, ws=B, wb=1 << 24):
    m = len(spans)
    p = (ctypes.c_void_p * m)(*[a for a, _ in spans])
    c = (ctypes.c_int64 * m)(*[x for _, x in spans])
    d = (ctypes.c_int32 * m)(*(dtypes or [1] * m))
    return q4.lib().q4_grad_norm(m, p, c, d, out, ws, wb, None)


def test_clip():
    G = B + 4096
    one = [(G, 100)]
    assert clip(one, n=-1) == SHAPE and clip(one, n=(1 << 20) + 1) == SHAPE
    assert clip([(G, -1)]) == SHAPE and clip([(G, (1 << 44) + 1)]) == SHAPE
    assert clip([(G, 1 << 44)]) == SHAPE                    # its chunks pass 32 bits
    assert clip(one, dtypes=[2]) == FMT
    assert clip([(None, 5)]) == NULL and clip(one, out=[None]) == NULL
    assert clip([(G + 2, 5)]) == ALIGN and clip([(G + 1, 5)], dtypes=[0]) == ALIGN
    assert clip(one, out=[G + 8192 + 2]) == ALIGN
    for bad in (-1.0, float("nan")):
        assert clip(one, max_norm=bad) == SHAPE
    assert clip(one, ws=None) == NULL and clip(one, ws=B + 8) == ALIGN and clip(one, wb=8) == SHAPE
    assert clip(one, norm_in=B + 2) == ALIGN and clip(one, norm=B + 2) == ALIGN
    assert norm(one, out=None) == NULL and norm(one, out=B + 2) == ALIGN and norm(one, ws=None) == NULL
    assert norm(one, wb=8) == SHAPE and norm([(G + 2, 5)]) == ALIGN and norm(one, dtypes=[3]) == FMT
    L, z = q4.lib(), ctypes.c_size_t()
    assert L.q4_grad_workspace(5, None) == NULL and L.q4_grad_workspace(-1, ctypes.byref(z)) == SHAPE
    assert L.q4_grad_clip(1, None, None, None, None, None, 1.0, B, B, 1 << 24, None) == NULL


def test_clip_refuses_overlaps():
    G, H = B + 4096, B + (1 << 20)
    assert clip([(G, 100), (G, 100)]) == ALIGN              # listed twice, in place
    assert clip([(G, 100), (G + 396, 10)]) == ALIGN         # the last value shared
    assert clip([(G + 396, 10), (G, 100)]) == ALIGN         # in either order
    assert clip([(G, 100), (G + 400, 10)], out=[H, H + 396]) == ALIGN       # outputs share a value
    assert clip([(G, 100), (G + 400, 10)], out=[G, G]) == ALIGN             # an output on another's gradient
    assert clip([(G, 100)], out=[G + 4]) == ALIGN                           # half on its own
    assert clip([(G, 100), (H, 10)], out=[H + 4096, G + 80]) == ALIGN


def test_bindings():
    lg, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=I32)
    for kw, text in [(dict(logits=lg.double()), "logits"), (dict(ids=ids.long()), "ids"), (dict(ids=ids[:3]), "rows"),
                     (dict(mask=torch.ones(4)), "mask"), (dict(mask=torch.ones(3, dtype=torch.bool)), "mask"),
                     (dict(mask=torch.ones(8, dtype=torch.bool)[::2]), "mask"), (dict(), "GPU")]:
        with pytest.raises(ValueError, match=text):
            q4.q4_moe_balance(**{**dict(logits=lg, ids=ids), **kw})
    s = torch.zeros(8)
    for kw, text in [(dict(slopes=s[:7]), "slopes"), (dict(slopes=s.double()), "slopes"), (dict(dloss=s.double()), "dloss"),
                     (dict(dlogits=lg[:3]), "dlogits"), (dict(accumulate=True), "accumulate"), (dict(), "GPU")]:
        with pytest.raises(ValueError, match=text):
            q4.q4_moe_balance_backward(**{**dict(logits=lg, slopes=s), **kw})
    g = [torch.zeros(5), torch.zeros(3, dtype=BF16)]
    for bad, text in [([], "at least one"), ([g[0].half()], "float32"), ([torch.zeros(4, 4).t()[:2]], "contiguous"),
                      ([g[0], None], "tensor"), (g, "GPU")]:
        with pytest.raises(ValueError, match=text):
            q4.q4_grad_norm(bad)
        with pytest.raises(ValueError, match=text):
            q4.q4_grad_clip(bad, 1.0)
    for out, text in [(g[:1], "2 tensors"), ([g[0], torch.zeros(4, dtype=BF16)], "size"), ([g[0], torch.zeros(3)], "size")]:
        with pytest.raises(ValueError, match=text):
            q4.q4_grad_clip(g, 1.0, out=out)
    with pytest.raises(ValueError, match="norm"):
        q4.q4_grad_clip(g, 1.0, norm=torch.zeros((), dtype=torch.float64))
