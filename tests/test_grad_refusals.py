"""What the backward calls refuse, on the host: the C ABI's status for bad
arguments before any launch, and the binding's ValueError before any library
call."""
import ctypes

import pytest
import torch

import w4_gemm_amd as q4

OK, NULL, SHAPE, ALIGN, FMT = 0, -1, -2, -3, -4
A16 = 0x7F0000000000        # never dereferenced: every call below ends before a launch
ODD = A16 + 2
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _d(fmt=q4.MXINT8, rows=64, cols=256, codes=A16, scales=A16, gs=None, layout=0):
    return q4._Q4TensorC(fmt, layout, rows, cols, codes, scales, gs)


def _r(d):
    return None if d is None else ctypes.byref(d)


def test_formats_of_saved_activations():
    L = q4.lib()
    for f in (q4.MXFP8, q4.MXINT8):
        assert q4.q4_sizes(f, 3, 64) == (192, 6)
        assert L.q4_sizes(f, 1, 3, 512, None, None) == FMT
        assert L.q4_sizes(f, 0, 3, 48, None, None) == SHAPE
        d, w = _d(f), _d(q4.MXFP4)
        assert L.q4_quantize(A16, 256, _r(_d(f, layout=1, cols=512)), None, None) == FMT
        assert L.q4_quantize(A16, 256, _r(d), A16, None) == FMT
        assert L.q4_quantize(A16, 250, _r(d), None, None) == SHAPE
        assert L.q4_quantize(ODD, 256, _r(d), None, None) == ALIGN
        assert L.q4_relayout(_r(d), _r(d), None) == FMT
        assert L.q4_gemv(_r(d), A16, 1, 256, A16, 64, None) == FMT
        assert L.q4_gemm(4, A16, 256, None, _r(d), A16, 64, None) == FMT
        assert L.q4_gemm(64, None, 0, _r(d), _r(w), A16, 64, None) == FMT
        assert L.q4_grouped_gemm(A16, 256, 4, None, A16, 1, 4, _r(d), 64, A16, 64, None) == FMT
        assert L.q4_gemm_dgrad(4, A16, 64, _r(d), A16, 256, None, 0, None) == FMT


def test_sort_refuses():
    L = q4.lib()
    n = ctypes.c_size_t()
    assert L.q4_moe_sort_workspace(10, 2, 8, None) == NULL
    for T, k, E in ((-1, 2, 8), (10, 0, 8), (10, 33, 8), (10, 2, 0), (10, 2, 1025), (1 << 30, 2, 8)):
        assert L.q4_moe_sort_workspace(T, k, E, ctypes.byref(n)) == SHAPE
    assert L.q4_moe_sort_workspace(1, 8, 64, ctypes.byref(n)) == OK and n.value == 0
    assert L.q4_moe_sort_workspace(100000, 8, 64, ctypes.byref(n)) == OK and 0 < n.value <= 256 * 64 * 4
    need = n.value
    assert L.q4_moe_sort(A16, 100000, 8, 64, A16, A16, A16, None, 0, None) == NULL
    assert L.q4_moe_sort(A16, 100000, 8, 64, A16, A16, A16, A16, need - 1, None) == SHAPE
    assert L.q4_moe_sort(A16, 100000, 8, 64, A16, A16, A16, ODD, need, None) == ALIGN
    assert L.q4_moe_sort(None, 4, 2, 8, A16, A16, A16, None, 0, None) == NULL
    assert L.q4_moe_sort(A16, 4, 2, 8, None, A16, A16, None, 0, None) == NULL
    assert L.q4_moe_sort(A16, 4, 2, 8, A16, A16, ODD, None, 0, None) == ALIGN


def test_row_calls_refuse():
    L = q4.lib()
    p = lambda **k: L.q4_moe_permute(*[{**dict(x=A16, ldx=64, inv=A16, T=4, k=2, K=64, P=8, xs=A16, ldxs=64, s=None), **k}[n]  # noqa: E731,E501
                                       for n in ("x", "ldx", "inv", "T", "k", "K", "P", "xs", "ldxs", "s")])
    assert p(T=0) == OK and p(K=0) == OK and p(P=0) == OK
    for bad in (dict(T=-1), dict(K=60), dict(k=0), dict(k=33), dict(P=-1), dict(T=1 << 23), dict(ldx=56), dict(ldxs=56),
                dict(T=1 << 22, K=1 << 14, ldx=1 << 14, ldxs=1 << 14)):
        assert p(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(inv=None), dict(xs=None)):
        assert p(**bad) == NULL, bad
    for bad in (dict(x=ODD), dict(inv=ODD + 1), dict(xs=ODD), dict(ldx=66), dict(ldxs=70)):
        assert p(**bad) == ALIGN, bad
    c = lambda **k: L.q4_moe_combine_backward(*[{**dict(d=A16, ldo=64, y=A16, ldy=64, inv=A16, w=A16, T=4, k=2, N=64, P=8,  # noqa: E731,E501
                                                        dy=A16, lddy=64, dw=A16, s=None), **k}[n]
                                                for n in ("d", "ldo", "y", "ldy", "inv", "w", "T", "k", "N", "P", "dy", "lddy", "dw", "s")])
    assert c(T=0) == OK
    for bad in (dict(N=12), dict(ldy=32), dict(k=40), dict(P=-2)):
        assert c(**bad) == SHAPE, bad
    for bad in (dict(d=None), dict(y=None), dict(inv=None), dict(w=None), dict(dy=None)):
        assert c(**bad) == NULL, bad
    assert c(dw=ODD) == ALIGN and c(dy=ODD) == ALIGN
    b = L.q4_moe_permute_backward
    assert b(A16, 64, A16, 4, 2, 63, 8, A16, 64, None) == SHAPE and b(None, 64, A16, 4, 2, 64, 8, A16, 64, None) == NULL
    t = L.q4_moe_topk_backward
    assert t(A16, 8, 0, 8, 2, None, None, None, 8, None) == OK
    assert t(A16, 8, 4, 1025, 2, A16, A16, A16, 8, None) == SHAPE and t(A16, 7, 4, 8, 2, A16, A16, A16, 8, None) == SHAPE
    assert t(A16, 8, 4, 8, 2, A16, None, A16, 8, None) == NULL and t(A16, 8, 4, 8, 2, A16, ODD + 1, A16, 8, None) == ALIGN
    k = L.q4_moe_topk
    assert k(A16, 8, 4, 8, 9, A16, A16, None) == SHAPE and k(A16, 8, 1 << 26, 8, 2, A16, A16, None) == SHAPE
    assert k(None, 8, 4, 8, 2, A16, A16, None) == NULL


def test_swiglu_refuses():
    L = q4.lib()
    s, b = L.q4_swiglu_save, L.q4_swiglu_backward
    assert s(A16, 256, 64, 120, A16, 120, _r(_d(cols=240 + 16)), None) == SHAPE      # I % 32
    assert s(A16, 256, 63, 128, A16, 128, _r(_d()), None) == SHAPE
    assert s(A16, 256, 64, 128, A16, 128, _r(_d(q4.MXFP4)), None) == FMT
    assert s(None, 256, 64, 128, A16, 128, _r(_d()), None) == NULL
    assert s(A16, 248, 64, 128, A16, 128, _r(_d()), None) == SHAPE
    assert s(A16, 256, 64, 128, ODD, 128, _r(_d()), None) == ALIGN
    assert b(None, 0, None, A16, 128, 64, 128, A16, 256, None, 0, None) == NULL
    assert b(A16, 256, _r(_d()), A16, 128, 64, 128, A16, 256, None, 0, None) == FMT
    assert b(None, 0, _r(_d(q4.FP8_ROW)), A16, 128, 64, 128, A16, 256, None, 0, None) == FMT
    assert b(None, 0, _r(_d()), A16, 128, 65, 128, A16, 256, None, 0, None) == SHAPE
    assert b(A16, 256, None, A16, 128, 64, 124, A16, 256, None, 0, None) == SHAPE
    assert b(None, 0, _r(_d()), None, 128, 64, 128, A16, 256, None, 0, None) == NULL
    assert b(None, 0, _r(_d()), A16, 128, 64, 128, ODD, 256, None, 0, None) == ALIGN
    assert b(None, 0, _r(_d()), A16, 128, 64, 128, A16, 256, A16, 100, None) == SHAPE


def test_products_refuse():
    L = q4.lib()
    n = ctypes.c_size_t()
    for f in (L.q4_dgrad_workspace, L.q4_wgrad_workspace):
        assert f(4, 1, 64, 256, None) == NULL
        for a in ((-1, 1, 64, 256), (4, -1, 64, 256), (4, 65536, 64, 256), (4, 1, -1, 256), (4, 1, 64, 1 << 31),
                  (4, 1, (1 << 21) + 8, 256), (1, 65535, (1 << 31) - 8, (1 << 31) - 128)):
            assert f(*a, ctypes.byref(n)) == SHAPE
        assert f((1 << 31) - 1, 65535, 1 << 21, 1 << 21, ctypes.byref(n)) == OK and n.value == 0
    big = 1 << 40
    W = _d(q4.MXFP4)
    g = lambda **k: L.q4_grouped_gemm_dgrad(*[{**dict(dc=A16, ld=32, off=A16, E=2, P=8, W=W, N=32, da=A16, lda=256, ws=A16,  # noqa: E731,E501
                                                      n=big, s=None), **k}[x] if x != "W" else _r({**dict(W=W), **k}["W"])
                                              for x in ("dc", "ld", "off", "E", "P", "W", "N", "da", "lda", "ws", "n", "s")])
    assert g(P=0) == OK and g(E=0, W=_d(q4.MXFP4, rows=0)) == OK
    for bad in (dict(N=33), dict(E=3), dict(P=-1), dict(ld=24), dict(lda=248), dict(W=_d(q4.MXFP4, rows=24), N=12),
                dict(W=_d(q4.MXFP4, rows=48, cols=512, layout=1), N=24), dict(W=_d(q4.MXFP4, cols=96))):
        assert g(**bad) == SHAPE, bad
    for bad in (dict(dc=None), dict(off=None), dict(da=None), dict(W=None)):
        assert g(**bad) == NULL, bad
    for bad in (dict(dc=ODD), dict(off=ODD + 1), dict(da=ODD), dict(ld=36)):
        assert g(**bad) == ALIGN, bad
    assert g(W=_d(q4.FP8_ROW)) == FMT
    far = 1 << 22
    assert g(ld=far) == SHAPE and g(W=_d(q4.MXFP4, cols=far), lda=far) == SHAPE and g(P=1 << 29) == SHAPE
    w = lambda **k: L.q4_grouped_gemm_wgrad(*[{**dict(dc=A16, ld=32, a=None, lda=0, q=None, T=64, gather=A16, off=A16, E=2, P=8,  # noqa: E731,E501
                                                      N=32, K=256, dw=A16, dt=1, ldw=256, acc=0, ws=A16, n=big, s=None), **k}[x]
                                              for x in ("dc", "ld", "a", "lda", "q", "T", "gather", "off", "E", "P", "N", "K", "dw",
                                                        "dt", "ldw", "acc", "ws", "n", "s")])
    q = _r(_d())
    assert w(q=q, N=0) == OK and w(q=q, E=0) == OK
    assert w() == NULL and w(q=q, a=A16) == FMT and w(q=_r(_d(q4.MXFP4))) == FMT
    assert w(q=q, dt=2) == FMT and w(q=q, dt=0, acc=1) == FMT
    for bad in (dict(q=q, T=63), dict(q=q, K=128), dict(q=q, N=12), dict(q=q, ldw=248), dict(q=q, gather=None, P=65, ld=32),
                dict(a=A16, lda=256, K=252), dict(a=A16, lda=248)):
        assert w(**bad) == SHAPE, bad
    for bad in (dict(q=q, ld=far), dict(a=A16, lda=far), dict(a=A16, lda=far, K=far, ldw=far), dict(q=q, P=(1 << 30) + 8),
                dict(q=q, N=1 << 31), dict(q=q, N=1 << 28),
                dict(q=q, P=1, N=far, ld=far)):
        assert w(**bad) == SHAPE, bad
    for bad in (dict(q=q, dc=None), dict(q=q, off=None), dict(q=q, dw=None)):
        assert w(**bad) == NULL, bad
    for bad in (dict(q=q, dw=ODD), dict(q=q, ldw=258), dict(q=q, dt=0, ldw=260), dict(q=q, gather=ODD + 1), dict(a=ODD, lda=256)):
        assert w(**bad) == ALIGN, bad


# ---------------------------------------------------------------- the binding

class _Guard:
    def __init__(self, real):
        self._real = real

    def __getattr__(self, name):
        if name in ("q4_sizes", "q4_status_string", "q4_last_hip_error"):
            return getattr(self._real, name)
        raise AssertionError(f"{name} was called with invalid arguments")


@pytest.fixture
def guard(monkeypatch):
    monkeypatch.setattr(q4, "_LIB", _Guard(q4.lib()))


def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses(guard):
    ids, w = z(4, 2, dtype=I32), z(4, 2, dtype=F32)
    _raises("ids must be", q4.q4_moe_sort, ids.long(), 8)
    _raises("ids must be a 2-D", q4.q4_moe_sort, ids.reshape(-1), 8)
    _raises("experts", q4.q4_moe_sort, ids, 0)
    _raises("gather must be contiguous with at least 8", q4.q4_moe_sort, ids, 8, gather=z(7, dtype=I32))
    _raises("GPU tensor", q4.q4_moe_sort, ids, 8)
    _raises("x must have 4 rows", q4.q4_moe_permute, z(5, 64), ids)
    _raises("xs must have 64 columns", q4.q4_moe_permute, z(4, 64), ids, z(8, 72))
    _raises("GPU tensor", q4.q4_moe_permute, z(4, 64), ids)
    _raises("dxs must be torch.bfloat16", q4.q4_moe_permute_backward, z(8, 64, dtype=F32), ids)
    _raises("dx must be at least 4", q4.q4_moe_permute_backward, z(8, 64), ids, z(3, 64))
    _raises("weights must be", q4.q4_moe_combine_backward, z(4, 64), z(8, 64), ids, w[:, :1])
    _raises("y is needed", q4.q4_moe_combine_backward, z(4, 64), None, ids, w)
    _raises("dy must have 8 rows", q4.q4_moe_combine_backward, z(4, 64), z(8, 64), ids, w, dy=z(7, 64))
    _raises("gates=False", q4.q4_moe_combine_backward, z(4, 64), z(8, 64), ids, w, dweights=w, gates=False)
    _raises("GPU tensor", q4.q4_moe_combine_backward, z(4, 64), z(8, 64), ids, w)
    _raises("logits must be torch.float32", q4.q4_moe_topk, z(4, 8), 2)
    _raises("logits must have 4 rows", q4.q4_moe_topk_backward, z(5, 8, dtype=F32), ids, w)
    _raises("dweights must be", q4.q4_moe_topk_backward, z(4, 8, dtype=F32), ids, w.double())
    saved = q4.empty_q4("mxint8", 4, 128, device="cpu")
    _raises("saved must be in", q4.q4_swiglu_save, z(4, 128), 64, q4.empty_q4("mxfp4", 4, 128, device="cpu"))
    _raises("saved must be 4 x 64", q4.q4_swiglu_save, z(4, 128), 32, saved)
    _raises("gu must be at least 0 x 128", q4.q4_swiglu_save, z(4, 96), 64, saved)
    _raises("GPU tensor", q4.q4_swiglu_save, z(4, 128), 64, saved)
    _raises("gu must be 5 x 128", q4.q4_swiglu_backward, saved, z(5, 64))
    _raises("dgu must be at least 4 x 128", q4.q4_swiglu_backward, saved, z(4, 64), dgu=z(4, 64))
    _raises("GPU tensor", q4.q4_swiglu_backward, z(4, 128), z(4, 64))
    W = q4.empty_q4("mxfp4", 64, 512, device="cpu")
    off = z(3, dtype=I32)
    _raises("dC must have 64 columns", q4.q4_gemm_dgrad, z(4, 32), W)
    _raises("dA must be at least 4 x 512", q4.q4_gemm_dgrad, z(4, 64), W, dA=z(4, 256))
    _raises("experts", q4.q4_grouped_gemm_dgrad, z(4, 64), off, W, 16)
    _raises("GPU tensor", q4.q4_grouped_gemm_dgrad, z(4, 32), off, W, 32)
    _raises("A must have 5 rows", q4.q4_gemm_wgrad, z(5, 64), saved)
    _raises("accumulate needs dW", q4.q4_gemm_wgrad, z(4, 64), saved, accumulate=True)
    _raises("accumulate needs a float32", q4.q4_gemm_wgrad, z(4, 64), saved, dW=z(64, 128), accumulate=True)
    _raises("dW must be float32 or bf16", q4.q4_gemm_wgrad, z(4, 64), saved, dW=z(64, 128, dtype=torch.float16))
    _raises("A must be in a saved", q4.q4_gemm_wgrad, z(64, 64), W)
    _raises("at least 5 rows", q4.q4_grouped_gemm_wgrad, z(5, 64), saved, None, off)
    _raises("gather must be contiguous with at least 5", q4.q4_grouped_gemm_wgrad, z(5, 64), saved, off, off)
    _raises("GPU tensor", q4.q4_grouped_gemm_wgrad, z(4, 64), saved, None, off)
