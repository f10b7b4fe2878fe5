"""What q4_rmsnorm and its gradient refuse, on the host."""
import ctypes

import pytest
import torch

import w4_gemm_amd as q4

OK, NULL, SHAPE, ALIGN, FMT = 0, -1, -2, -3, -4
B = 0x7F0000000000
BF16 = torch.bfloat16


def fwd(**kw):
    a = dict(x=B, ldx=256, res=B, ldr=256, w=B, wt=0, eps=1e-6, rows=4, cols=256, h=B, ldh=256, y=B, ldy=256, q=None)
    a.update(kw)
    q = ctypes.byref(a["q"]) if a["q"] is not None else None
    return q4.lib().q4_rmsnorm(a["x"], a["ldx"], a["res"], a["ldr"], a["w"], a["wt"], a["eps"], a["rows"], a["cols"],
                               a["h"], a["ldh"], a["y"], a["ldy"], q, None)


def bwd(**kw):
    a = dict(dy=B, lddy=256, h=B, ldh=256, w=B, wt=0, eps=1e-6, dh=B, lddh=256, rows=4, cols=256, dx=B, lddx=256, dw=B,
             acc=0, ws=B, wb=1 << 30)
    a.update(kw)
    return q4.lib().q4_rmsnorm_backward(a["dy"], a["lddy"], a["h"], a["ldh"], a["w"], a["wt"], a["eps"], a["dh"],
                                        a["lddh"], a["rows"], a["cols"], a["dx"], a["lddx"], a["dw"], a["acc"],
                                        a["ws"], a["wb"], None)


def qdesc(fmt=q4.INT8_ROW, rows=4, cols=256, layout=0, codes=B, scales=B, gs=None):
    return q4._Q4TensorC(fmt, layout, rows, cols, codes, scales, gs)


def test_forward():
    assert fwd(y=None) == NULL
    assert fwd(wt=2) == FMT
    assert fwd(w=None) == NULL and fwd(w=B + 4) == ALIGN
    assert fwd(h=None) == FMT and fwd(res=None) == FMT          # h and the residual go together
    for eps in (-1e-6, float("nan"), float("inf")):
        assert fwd(eps=eps) == SHAPE
    assert fwd(rows=-1) == SHAPE and fwd(rows=1 << 22) == SHAPE
    assert fwd(cols=252) == SHAPE and fwd(cols=32776) == SHAPE
    for ld in ("ldx", "ldr", "ldh", "ldy"):
        assert fwd(**{ld: 248}) == SHAPE and fwd(**{ld: 260}) == ALIGN
    for p in ("x", "res", "h", "y"):
        assert fwd(**{p: B + 2}) == ALIGN
    assert fwd(x=None) == NULL
    assert fwd(rows=0, x=None) == OK and fwd(cols=0, w=None) == OK


def test_eight_bit_output():
    assert fwd(q=qdesc(q4.MXFP4)) == FMT and fwd(q=qdesc(q4.MXFP8)) == FMT
    assert fwd(q=qdesc(rows=5)) == SHAPE and fwd(q=qdesc(cols=512)) == SHAPE
    assert fwd(q=qdesc(layout=1)) == FMT
    assert fwd(q=qdesc(q4.FP8_ROW, layout=1)) == SHAPE          # tiled: cols % 512
    assert fwd(q=qdesc(gs=B)) == FMT
    assert fwd(q=qdesc(codes=None)) == NULL and fwd(q=qdesc(codes=B + 8)) == ALIGN
    assert fwd(cols=248, q=qdesc(cols=248)) == SHAPE            # 8-bit rows: cols % 16


def test_backward():
    assert bwd(wt=2) == FMT and bwd(w=None) == NULL and bwd(w=B + 8) == ALIGN
    assert bwd(eps=-1.0) == SHAPE
    assert bwd(rows=-1) == SHAPE and bwd(rows=1 << 22) == SHAPE and bwd(cols=32776) == SHAPE and bwd(cols=4) == SHAPE
    for ld in ("lddy", "ldh", "lddh", "lddx"):
        assert bwd(**{ld: 248}) == SHAPE and bwd(**{ld: 260}) == ALIGN
    for p in ("dy", "h", "dh", "dx"):
        assert bwd(**{p: B + 2}) == ALIGN
    for p in ("dy", "h", "dx"):
        assert bwd(**{p: None}) == NULL
    assert bwd(dw=B + 2) == ALIGN
    assert bwd(ws=None) == NULL and bwd(ws=B + 4) == ALIGN
    n = ctypes.c_size_t()
    assert q4.lib().q4_rmsnorm_backward_workspace(4, 256, ctypes.byref(n)) == OK
    assert bwd(wb=n.value - 1) == SHAPE
    assert q4.lib().q4_rmsnorm_backward_workspace(4, 256, None) == NULL
    assert q4.lib().q4_rmsnorm_backward_workspace(1 << 22, 256, ctypes.byref(n)) == SHAPE
    assert bwd(rows=0, dw=None) == OK and bwd(rows=0, acc=1) == OK and bwd(cols=0) == OK


def test_binding():
    x, w = torch.zeros(4, 64, dtype=BF16), torch.ones(64, dtype=BF16)
    bad = [
        (dict(x=x.float()), "x must be"), (dict(weight=w[:32]), "weight"), (dict(weight=w.half()), "weight"),
        (dict(residual=x[:2]), "residual"), (dict(residual=x[:, :32]), "residual"), (dict(h=x), "residual"),
        (dict(y=x[:3]), "y must"), (dict(y_q=q4.empty_q4("mxfp4", 4, 64, device="cpu")), "y_q"),
        (dict(y_q=q4.empty_q4("int8_row", 5, 64, device="cpu")), "y_q"), (dict(), "GPU"),
    ]
    for kw, text in bad:
        with pytest.raises(ValueError, match=text):
            q4.q4_rmsnorm(**{**dict(x=x, weight=w), **kw})
    bad = [
        (dict(dy=x.float()), "dy must be"), (dict(h=x[:3]), "h must"), (dict(h=x[:, :32]), "h must"),
        (dict(weight=w[:8]), "weight"), (dict(dh=x[:1]), "dh"), (dict(dx=x[:1]), "dx"), (dict(dweight=w), "dweight"),
        (dict(dweight=torch.zeros(64), weight_grad=False), "weight_grad"), (dict(accumulate=True), "accumulate"),
        (dict(), "GPU"),
    ]
    for kw, text in bad:
        with pytest.raises(ValueError, match=text):
            q4.q4_rmsnorm_backward(**{**dict(dy=x, h=x, weight=w), **kw})
