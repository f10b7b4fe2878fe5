"""GPU parity of the backward calls with the plain definitions (oracle/grad.py).

Tolerances, per element, from the roundings alone (u = 2^-24, half an fp32
step; a bf16 rounding is off by at most 2^-8 of the value):
  * integers, copies and 8-bit codes: equal bit for bit;
  * bf16 outputs of sums: 2^-8 |ref| + n 2^-23 S, S the sum of the terms'
    magnitudes and n their number (each fp32 addition and product off by u of
    a value of at most S, doubled for the rounding inside a matrix step);
    INT4 weights add 2^-8 S (rounded to bf16 before the product);
  * fp32 sums: n 2^-23 S;
  * SwiGLU: the sigmoid is off by (|g| + 8) 2^-22 relative (the argument's
    rounding, exp2 and the reciprocal), so dg by that times
    |dh u| s (1 + |g|)^2 before its bf16 rounding;
  * gate gradients: a probability is off by (r + E) 2^-22 relative, r the
    range of the logits, its parts |p d| and p sum|p d|.
"""
import zlib

import numpy as np
import pytest
import torch

import oracle
import w4_gemm_amd as q4
from oracle import grad
from q4_helpers import log, to_f32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _rng(*key):
    return np.random.default_rng([zlib.crc32(k.encode()) if isinstance(k, str) else k for k in key])


def _bf16(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(BF16)


def _strided(t, extra=16):
    """t on the GPU as a view whose rows are `extra` elements further apart, the gaps NaN."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=DEV)
    buf[:, :t.shape[1]] = t.to(DEV)
    return buf[:, :t.shape[1]]


def _close(got, ref, bound, what):
    got = to_f32(got).astype(np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    bad = np.argwhere(~(np.abs(got - ref) <= bound))
    assert bad.size == 0, (what, len(bad), [(tuple(i), got[tuple(i)], ref[tuple(i)]) for i in bad[:4]])


# ------------------------------------------------------------------ sort

def _ids(rng, T, k, E, drop):
    ids = np.stack([rng.permutation(max(E, k))[:k] % E for _ in range(T)]) if T else np.zeros((0, k))
    ids = ids.astype(np.int32)
    if drop:
        m = rng.random((T, k))
        ids = np.where(m < drop / 2, -1, np.where(m < drop, E + 3, ids)).astype(np.int32)
    return ids


SORT = [(0, 4, 8, 0), (1, 1, 1, 0), (1, 8, 64, 0), (3, 8, 8, 0.5), (513, 8, 64, 0.1), (512, 8, 64, 0), (4097, 1, 3, 0.2),
        (1371, 3, 37, 0.3), (700, 32, 1024, 0.1), (20000, 8, 64, 0.125), (40000, 7, 1000, 0), (5000, 2, 16, 1.0)]


@pytest.mark.parametrize("T,k,E,drop", SORT)
def test_sort(T, k, E, drop):
    log("sort", T, k, E, drop)
    ids = _ids(_rng("sort", T, k, E), T, k, E, drop)
    ro, rg, ri = grad.moe_sort(ids, E)
    gather = torch.full((T * k,), -7, dtype=I32, device=DEV)
    offsets, gather, inv = q4.q4_moe_sort(torch.from_numpy(ids).to(DEV), E, gather=gather)
    assert np.array_equal(offsets.cpu().numpy(), ro)
    assert np.array_equal(inv.cpu().numpy(), ri)
    g = gather.cpu().numpy()
    assert np.array_equal(g[:len(rg)], rg) and np.all(g[len(rg):] == -7)


def test_sort_of_one_expert_and_repeats():
    ids = np.full((9000, 4), 5, np.int32)
    ro, rg, ri = grad.moe_sort(ids, 7)
    offsets, gather, inv = q4.q4_moe_sort(torch.from_numpy(ids).to(DEV), 7)
    assert np.array_equal(offsets.cpu().numpy(), ro) and np.array_equal(inv.cpu().numpy(), ri)
    assert np.array_equal(gather.cpu().numpy(), rg)


@pytest.mark.parametrize("T,E,k", [(300, 64, 8), (77, 16, 2), (5, 1024, 32)])
def test_topk_and_sort_are_the_route(T, E, k):
    lg = torch.from_numpy(_rng("route", T, E).standard_normal((T, E)).astype(np.float32)).to(DEV)
    r = q4.q4_moe_route(lg, k)
    ids, w = q4.q4_moe_topk(lg, k)
    offsets, gather, inv = q4.q4_moe_sort(ids, E)
    for a, b in ((ids, r.ids), (w, r.weights), (offsets, r.offsets), (gather, r.gather), (inv, r.inv)):
        assert torch.equal(a, b)


# -------------------------------------------------- permute, combine, gates

ROWS = [(1, 8, 64, 7168, 0), (5, 3, 8, 8, 0.4), (130, 2, 4, 1032, 0.2), (64, 32, 40, 520, 0.1), (7, 1, 2, 2048, 1.0),
        (33, 5, 16, 4104, 0)]


def _routed(T, k, E, drop, tag):
    rng = _rng(tag, T, k, E)
    _, _, inv = grad.moe_sort(_ids(rng, T, k, E, drop), E)
    return rng, inv, torch.from_numpy(inv).to(DEV)


@pytest.mark.parametrize("strided", (False, True))
@pytest.mark.parametrize("T,k,E,K,drop", ROWS)
def test_permute(T, k, E, K, drop, strided):
    log("permute", T, k, E, K, drop, strided)
    rng, inv, inv_d = _routed(T, k, E, drop, "permute")
    x, old = _bf16(rng, T, K), _bf16(rng, T * k + 3, K)
    put = _strided if strided else (lambda t: t.to(DEV))
    xs = put(old)
    q4.q4_moe_permute(put(x), inv_d, xs)
    assert np.array_equal(to_f32(xs), grad.permute(to_f32(x), inv, to_f32(old)))
    dxs = _bf16(rng, T * k, K)
    dxs[_unowned(inv, T * k)] = float("nan")       # rows without a choice are not read
    dx = put(torch.full((T, K), float("nan"), dtype=BF16))
    q4.q4_moe_permute_backward(put(dxs), inv_d, dx)
    d = to_f32(dxs)
    ref = grad.permute_backward(d, inv)
    _close(dx, ref, 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -23 * grad.permute_backward(np.abs(d), inv), "dx")


def _unowned(inv, P):
    own = np.zeros(P, bool)
    own[inv[inv >= 0]] = True
    return torch.from_numpy(~own)


@pytest.mark.parametrize("strided", (False, True))
@pytest.mark.parametrize("T,k,E,N,drop", ROWS)
def test_combine_backward(T, k, E, N, drop, strided):
    log("combine backward", T, k, E, N, drop, strided)
    rng, inv, inv_d = _routed(T, k, E, drop, "combine")
    P = T * k
    dout, y, old = _bf16(rng, T, N, std=0.1), _bf16(rng, P, N), _bf16(rng, P, N)
    y[_unowned(inv, P)] = float("inf")
    w = rng.random((T, k)).astype(np.float32)
    put = _strided if strided else (lambda t: t.to(DEV))
    dy = put(old)
    _, dw = q4.q4_moe_combine_backward(put(dout), put(y), inv_d, torch.from_numpy(w).to(DEV), dy=dy)
    rdy, rdw = grad.combine_backward(to_f32(dout), to_f32(y), inv, w, to_f32(old))
    own = ~_unowned(inv, P).numpy()
    assert np.array_equal(to_f32(dy)[~own], to_f32(old)[~own])
    _close(dy, rdy, 2.0 ** -8 * np.abs(rdy) * (1 + 2.0 ** -14), "dy")
    ya = np.where(own[:, None], np.abs(to_f32(y)), 0.0)
    _, s = grad.combine_backward(np.abs(to_f32(dout)), ya, inv, w, to_f32(old))
    _close(dw, rdw, N * 2.0 ** -23 * s, "dw")
    dy2 = put(old)
    _, none = q4.q4_moe_combine_backward(put(dout), None, inv_d, torch.from_numpy(w).to(DEV), dy=dy2, gates=False)
    assert none is None and torch.equal(dy2, dy)


def test_combine_leaves_out_dropped_choices():
    T, k, E, N = 40, 4, 8, 512
    rng, inv, inv_d = _routed(T, k, E, 0.4, "fwd")
    y, w = _bf16(rng, T * k, N), rng.random((T, k)).astype(np.float32)
    r = q4.Routing(inv_d, torch.from_numpy(w).to(DEV), inv_d, inv_d, inv_d)
    out = q4.q4_moe_combine(y.to(DEV), r)
    yf = to_f32(y).astype(np.float64)
    ref, s = (sum(np.where((inv[:, j] >= 0)[:, None], w[:, j:j + 1] * v[inv[:, j]], 0.0) for j in range(k))
              for v in (yf, np.abs(yf)))
    _close(out, ref, 2.0 ** -8 * np.abs(ref) + k * 2.0 ** -23 * s, "combine")


@pytest.mark.parametrize("T,E,k", [(1, 8, 8), (300, 64, 8), (9, 37, 3), (6, 1024, 32), (4, 1, 1)])
def test_topk_backward(T, E, k):
    log("topk backward", T, E, k)
    rng = _rng("topk", T, E, k)
    lg = (rng.standard_normal((T, E)) * 3).astype(np.float32)
    if T > 3 and E > 4:
        lg[1, : E - 1] = -np.inf          # masked experts
        lg[2] = -np.inf                   # nothing left
        lg[3, 0] = 80.0
    ids = _ids(rng, T, k, E, 0.2)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    buf = torch.full((T, E + 3), -5.0, device=DEV)
    lgd = torch.full((T, E + 1), float("nan"), device=DEV)
    lgd[:, :E] = torch.from_numpy(lg)
    out = q4.q4_moe_topk_backward(lgd[:, :E], torch.from_numpy(ids).to(DEV), torch.from_numpy(dw).to(DEV),
                                  dlogits=buf[:, :E])
    ref = grad.topk_backward(lg, ids, dw)
    with np.errstate(invalid="ignore"):
        p = np.exp(lg.astype(np.float64) - lg.max(1, keepdims=True).astype(np.float64))
    p = np.nan_to_num(p / p.sum(1, keepdims=True))
    d = np.zeros((T, E))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if 0 <= e < E:
                d[t, e] += abs(float(dw[t, j]))
    fin = np.where(np.isfinite(lg), lg, 0.0)
    rel = (np.ptp(fin, axis=1)[:, None] + E + k) * 2.0 ** -22
    _close(out, ref, rel * p * (d + (p * d).sum(1, keepdims=True)) + 1e-37, "dlogits")
    assert torch.all(buf[:, E:] == -5.0)


# -------------------------------------------------------- 8-bit activations

def _special(rng, rows, cols):
    x = rng.standard_normal((rows, cols)).astype(np.float32) * np.float32(2.0) ** rng.integers(-20, 20, (rows, 1))
    x = torch.from_numpy(x).to(BF16)
    x[0, :32] = 0.0
    x[0, 1] = -0.0
    if rows > 4:
        x[1, 5], x[2, 6], x[3, 7] = float("inf"), float("nan"), float("-inf")
        x[4, :32] = torch.finfo(BF16).max
        x[4, 1] = 2.0 ** -133
        x[4, 32:64] = 2.0 ** -120
        x[4, 40] = 127.0 * 2.0 ** -111 if cols > 64 else 1.0
    return x


@pytest.mark.parametrize("fmt", ("mxint8", "mxfp8"))
@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 96), (33, 2048), (5, 8224)])
def test_mx8_bits(fmt, rows, cols):
    log("mx8", fmt, rows, cols)
    x = _special(_rng("mx8", rows, cols), rows, cols)
    codes, scales = grad.mx8_quantize(fmt, to_f32(x))
    for src in (x.to(DEV), _strided(x)):
        q = q4.q4_quantize(src, q4.empty_q4(fmt, rows, cols, device=DEV))
        assert np.array_equal(q.scales.cpu().numpy(), scales)
        assert np.array_equal(q.codes.cpu().numpy(), codes)
    ref = grad.mx8_dequant(fmt, codes, scales)
    for dt in (F32, BF16):
        d = q4.q4_dequant(q, torch.empty(rows, cols, dtype=dt, device=DEV))
        assert np.array_equal(to_f32(d).astype(np.float64), ref, equal_nan=True)


@pytest.mark.parametrize("fmt", ("mxint8", "mxfp8"))
def test_mx8_every_bf16_value(fmt):
    bits = np.arange(65536, dtype=np.uint16)
    x = torch.from_numpy(bits.view(np.int16).copy()).view(BF16).reshape(-1, 1).repeat(1, 32)
    x[:, 1:] = torch.where(torch.isfinite(x[:, :1]), x[:, :1], 0.0) * torch.linspace(0, 1, 31).to(BF16)
    codes, scales = grad.mx8_quantize(fmt, to_f32(x[::7]))
    q = q4.quantize(x[::7].to(DEV), fmt)
    assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(q.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("strided", (False, True))
@pytest.mark.parametrize("fmt", ("mxint8", "mxfp8"))
@pytest.mark.parametrize("P,I", [(1, 32), (33, 2048), (130, 96), (3, 544)])
def test_swiglu_save_and_backward(fmt, P, I, strided):
    log("swiglu", fmt, P, I, strided)
    rng = _rng("swiglu", P, I)
    gu, dh = _bf16(rng, P, 2 * I, std=3.0), _bf16(rng, P, I)
    gu[0, :8] = torch.tensor([0.0, -0.0, 60.0, -60.0, 1e-30, 120.0, -120.0, -1.278]).to(BF16)
    put = _strided if strided else (lambda t: t.to(DEV))
    saved = q4.empty_q4(fmt, P, 2 * I, device=DEV)
    h = q4.q4_swiglu_save(put(gu), I, saved)
    f = to_f32(gu).astype(np.float64)
    g, u = f[:, :I], f[:, I:]
    ref = grad.swiglu_backward(g, u, np.zeros_like(g))[2]
    _close(h, ref, (2.0 ** -8 + (np.abs(g) + 8) * 2.0 ** -22) * np.abs(ref) + 1e-34, "h")
    q = q4.quantize(gu.to(DEV), fmt)
    assert torch.equal(q.codes, saved.codes) and torch.equal(q.scales, saved.scales)
    kept = grad.mx8_dequant(fmt, saved.codes.cpu().numpy(), saved.scales.cpu().numpy())
    for src, v in ((saved, kept), (put(gu), f)):
        g, u = v[:, :I], v[:, I:]
        dg, du, rh = grad.swiglu_backward(g, u, to_f32(dh))
        h2, dgu = put(torch.zeros(P, I, dtype=BF16)), put(torch.zeros(P, 2 * I, dtype=BF16))
        q4.q4_swiglu_backward(src, put(dh), dgu=dgu, h=h2)
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-g))
        e = (np.abs(g) + 8) * 2.0 ** -22
        a = np.abs(to_f32(dh).astype(np.float64))
        _close(dgu[:, :I], dg, 2.0 ** -8 * np.abs(dg) + e * a * np.abs(u) * s * (1 + np.abs(g)) ** 2 + 1e-34, "dg")
        _close(dgu[:, I:], du, (2.0 ** -8 + e) * np.abs(du) + 1e-34, "du")
        _close(h2, rh, (2.0 ** -8 + e) * np.abs(rh) + 1e-34, "h again")


def test_swiglu_backward_of_bf16_with_narrow_rows():
    gu, dh = _bf16(_rng("narrow"), 9, 48), _bf16(_rng("narrow", 2), 9, 24)       # 24 % 32 != 0
    dgu = q4.q4_swiglu_backward(gu.to(DEV), dh.to(DEV))
    f = to_f32(gu)
    dg, du, _ = grad.swiglu_backward(f[:, :24], f[:, 24:], to_f32(dh))
    ref = np.concatenate((dg, du), 1)
    _close(dgu, ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -16, "dgu")


# ------------------------------------------------------------- the products

def _segments(rng, E, P, kind):
    if kind == "empty_first":
        cuts = np.sort(rng.integers(0, P + 1, max(E - 2, 0)))
        cuts = np.concatenate(([0], cuts))[:E - 1]
    else:
        cuts = np.sort(rng.integers(0, P + 1, E - 1))
    return np.concatenate(([0], cuts, [P])).astype(np.int32)


def _dgrad_bound(dc, offsets, w, N, ref, exact):
    s = grad.dgrad(np.abs(dc), offsets, np.abs(w), N)
    return 2.0 ** -8 * np.abs(ref) + ((N + 8) * 2.0 ** -23 + (0 if exact else 2.0 ** -8)) * s + 1e-37


FORMATS = ("int4", "mxfp4", "nvfp4", "int4_zp")


@pytest.mark.parametrize("layout", ("rows", "tiled"))
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 16, 512), (77, 512, 512), (130, 264, 1024), (300, 72, 512), (257, 1000, 1536)])
def test_dgrad_dense(M, N, K, fmt, layout):
    log("dgrad", M, N, K, fmt, layout)
    rng = _rng("dgrad", M, N, K)
    w, dc = _bf16(rng, N, K, std=0.02), _bf16(rng, M, N)
    W = q4.quantize(w.to(DEV), fmt, layout=layout)
    wd = oracle.dequant(oracle.quantize(fmt, to_f32(w)))
    off = np.array([0, M], np.int32)
    ref = grad.dgrad(to_f32(dc), off, wd, N)
    bound = _dgrad_bound(to_f32(dc), off, wd, N, ref, fmt in ("mxfp4", "nvfp4"))
    _close(q4.q4_gemm_dgrad(dc.to(DEV), W), ref, bound, "dA")
    out = _strided(torch.zeros(M + 2, K, dtype=BF16))
    q4.q4_gemm_dgrad(_strided(dc), W, dA=out)
    _close(out[:M], ref, bound, "dA strided")
    assert torch.all(out[M:] == 0)


def test_dgrad_rows_layout_with_128_columns():
    rng = _rng("dgrad128")
    for fmt in FORMATS:
        w, dc = _bf16(rng, 40, 384, std=0.02), _bf16(rng, 19, 40)
        W = q4.quantize(w.to(DEV), fmt)
        wd = oracle.dequant(oracle.quantize(fmt, to_f32(w)))
        off = np.array([0, 19], np.int32)
        ref = grad.dgrad(to_f32(dc), off, wd, 40)
        _close(q4.q4_gemm_dgrad(dc.to(DEV), W), ref, _dgrad_bound(to_f32(dc), off, wd, 40, ref, False), fmt)


@pytest.mark.parametrize("layout", ("rows", "tiled"))
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("E,P,N,K,kind", [(1, 5, 16, 512, ""), (4, 3, 32, 512, ""), (8, 300, 48, 1024, "empty_first"),
                                          (70, 900, 16, 512, ""), (3, 1100, 128, 512, "")])
def test_dgrad_grouped(E, P, N, K, kind, fmt, layout):
    log("dgrad grouped", E, P, N, K, kind, fmt, layout)
    rng = _rng("dgradg", E, P, N)
    off = _segments(rng, E, P, kind)
    w, dc = _bf16(rng, E * N, K, std=0.02), _bf16(rng, P + 5, N)
    W = q4.quantize(w.to(DEV), fmt, layout=layout)
    wd = oracle.dequant(oracle.quantize(fmt, to_f32(w)))
    dc[P:] = float("nan")                      # rows behind the last expert are neither read nor written
    out = torch.full((P + 5, K), 7.0, dtype=BF16, device=DEV)
    q4.q4_grouped_gemm_dgrad(dc.to(DEV), torch.from_numpy(off).to(DEV), W, N, dA=out)
    ref = grad.dgrad(to_f32(dc)[:P], off, wd, N)
    _close(out[:P], ref, _dgrad_bound(to_f32(dc)[:P], off, wd, N, ref, fmt in ("mxfp4", "nvfp4")), "dA")
    assert torch.all(out[P:] == 7.0)


def _activation(rng, kind, T, K):
    """(operand on the GPU, its values) of activations kept as `kind`."""
    x = _bf16(rng, T, K)
    x[:, :: 37] *= 20
    if kind == "bf16":
        return x.to(DEV), to_f32(x)
    q = q4.quantize(x.to(DEV), kind)
    return q, grad.mx8_dequant(kind, *grad.mx8_quantize(kind, to_f32(x)))


def _wgrad_bound(dc, a, gather, off):
    n = max((b - c for b, c in zip(off[1:], off[:-1])), default=0)
    return (n + 8) * 2.0 ** -23 * grad.wgrad(np.abs(dc), np.abs(a), gather, off) + 1e-37


@pytest.mark.parametrize("kind", ("bf16", "mxint8", "mxfp8"))
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (77, 512, 512), (130, 72, 1056), (1000, 264, 96), (64, 1000, 288)])
def test_wgrad_dense(M, N, K, kind):
    log("wgrad", M, N, K, kind)
    rng = _rng("wgrad", M, N, K)
    dc = _bf16(rng, M, N)
    A, a = _activation(rng, kind, M, K)
    off = np.array([0, M], np.int32)
    ref = grad.wgrad(to_f32(dc), a, None, off)
    bound = _wgrad_bound(to_f32(dc), a, None, off)
    _close(q4.q4_gemm_wgrad(dc.to(DEV), A), ref, bound, "dW")
    out = torch.full((N + 1, K + 8), 3.0, device=DEV)
    q4.q4_gemm_wgrad(_strided(dc), _strided(A) if kind == "bf16" else A, dW=out[:, :K])
    _close(out[:N, :K], ref, bound, "dW strided")
    assert torch.all(out[N:] == 3.0) and torch.all(out[:, K:] == 3.0)
    old = _rng("old").standard_normal((N, K)).astype(np.float32)
    out[:N, :K] = torch.from_numpy(old)
    q4.q4_gemm_wgrad(dc.to(DEV), A, dW=out[:, :K], accumulate=True)
    _close(out[:N, :K], old + ref, bound + 2.0 ** -23 * (np.abs(old) + np.abs(ref)), "dW accumulated")
    b = q4.q4_gemm_wgrad(dc.to(DEV), A, dW=torch.empty(N, K, dtype=BF16, device=DEV))
    _close(b, ref, bound * 1.01 + 2.0 ** -8 * np.abs(ref), "dW bf16")


@pytest.mark.parametrize("K", (8, 40, 104))
def test_wgrad_bf16_narrow(K):
    rng = _rng("narrow", K)
    dc, x = _bf16(rng, 50, 24), _bf16(rng, 50, K)
    off = np.array([0, 50], np.int32)
    ref = grad.wgrad(to_f32(dc), to_f32(x), None, off)
    _close(q4.q4_gemm_wgrad(dc.to(DEV), x.to(DEV)), ref, _wgrad_bound(to_f32(dc), to_f32(x), None, off), "dW")


@pytest.mark.parametrize("gathered", (True, False))
@pytest.mark.parametrize("kind", ("bf16", "mxint8", "mxfp8"))
@pytest.mark.parametrize("E,T,P,N,K,seg", [(1, 5, 5, 16, 32, ""), (4, 9, 3, 32, 64, ""), (8, 100, 300, 48, 544, "empty_first"),
                                           (70, 333, 900, 16, 32, ""), (3, 600, 1100, 128, 288, "")])
def test_wgrad_grouped(E, T, P, N, K, seg, kind, gathered):
    log("wgrad grouped", E, T, P, N, K, seg, kind, gathered)
    rng = _rng("wgradg", E, P, N)
    if not gathered:
        T = P + 2
    off = _segments(rng, E, P, seg)
    dc = _bf16(rng, P, N)
    A, a = _activation(rng, kind, T, K)
    gather = rng.integers(0, T, P).astype(np.int32) if gathered else None
    if gathered and P > 20:
        gather[[3, 17]] = [-1, T]              # rows outside A read zeros
    offd = torch.from_numpy(off).to(DEV)
    gd = torch.from_numpy(gather).to(DEV) if gathered else None
    ref = grad.wgrad(to_f32(dc), a[:P] if not gathered else a, gather, off)
    bound = _wgrad_bound(to_f32(dc), a, gather, off)
    dW = q4.q4_grouped_gemm_wgrad(dc.to(DEV), A, gd, offd)
    _close(dW, ref, bound, "dW")
    q4.q4_grouped_gemm_wgrad(dc.to(DEV), A, gd, offd, dW=dW, accumulate=True)
    _close(dW, 2 * ref, 2 * bound + 2.0 ** -22 * np.abs(ref), "dW twice")


@pytest.mark.parametrize("layout", ("rows", "tiled"))
@pytest.mark.parametrize("fmt", FORMATS)
def test_dgrad_large_blocks(fmt, layout):
    """Sizes whose blocks fill the GPU: no part sums, the largest block; ragged rows, two experts and one."""
    log("dgrad large", fmt, layout)
    rng = _rng("dgradl")
    for E, P, N, K in ((1, 2101, 40, 7680), (2, 4211, 48, 4608)):
        off = np.array([0, 2107, P] if E == 2 else [0, P], np.int32)
        w, dc = _bf16(rng, E * N, K, std=0.02), _bf16(rng, P, N)
        W = q4.quantize(w.to(DEV), fmt, layout=layout)
        wd = oracle.dequant(oracle.quantize(fmt, to_f32(w)))
        got = (q4.q4_gemm_dgrad(dc.to(DEV), W) if E == 1 else
               q4.q4_grouped_gemm_dgrad(dc.to(DEV), torch.from_numpy(off).to(DEV), W, N))
        ref = grad.dgrad(to_f32(dc), off, wd, N)
        _close(got, ref, _dgrad_bound(to_f32(dc), off, wd, N, ref, fmt in ("mxfp4", "nvfp4")), (E, "dA"))


@pytest.mark.parametrize("kind", ("bf16", "mxint8", "mxfp8"))
def test_wgrad_large_blocks(kind):
    log("wgrad large", kind)
    rng = _rng("wgradl")
    for E, T, P, N, K, gathered in ((1, 301, 301, 4104, 4128, False), (3, 400, 931, 2568, 2336, True)):
        dc = _bf16(rng, P, N)
        x = _bf16(rng, T, K)
        A = x.to(DEV) if kind == "bf16" else q4.quantize(x.to(DEV), kind)
        a = to_f32(x) if kind == "bf16" else to_f32(q4.q4_dequant(A, torch.empty(T, K, device=DEV)))
        off = np.array([0, 299, 640, P] if E == 3 else [0, P], np.int32)
        gather = rng.integers(0, T, P).astype(np.int32) if gathered else None
        got = (q4.q4_gemm_wgrad(dc.to(DEV), A) if E == 1 else
               q4.q4_grouped_gemm_wgrad(dc.to(DEV), A, torch.from_numpy(gather).to(DEV), torch.from_numpy(off).to(DEV)))
        ref = grad.wgrad(to_f32(dc), a, gather, off)
        _close(got, ref, _wgrad_bound(to_f32(dc), a, gather, off), (E, "dW"))


@pytest.mark.parametrize("P,N,K", [(2, 4096, 512), (33, 1040, 1024), (1500, 8, 32), (5000, 24, 96)])
def test_products_in_parts(P, N, K):
    """Few blocks and a long sum (dgrad over N, wgrad over P): part sums joined, twice the same bits, the output's other rows
    left alone."""
    log("parts", P, N, K)
    rng = _rng("parts", P, N, K)
    dc, x = _bf16(rng, P, N), _bf16(rng, P, K)
    off = np.array([1, P // 2, P - 1], np.int32)
    offd = torch.from_numpy(off).to(DEV)
    if K % 128 == 0:
        w = _bf16(rng, 2 * N, K, std=0.02)
        W = q4.quantize(w.to(DEV), "nvfp4", layout="tiled")
        wd = oracle.dequant(oracle.quantize("nvfp4", to_f32(w)))
        out = torch.full((P, K), 7.0, dtype=BF16, device=DEV)
        q4.q4_grouped_gemm_dgrad(dc.to(DEV), offd, W, N, dA=out)
        ref = grad.dgrad(to_f32(dc), off, wd, N)
        _close(out[1:P - 1], ref[1:P - 1], _dgrad_bound(to_f32(dc), off, wd, N, ref, True)[1:P - 1], "dA")
        assert torch.all(out[0] == 7.0) and torch.all(out[P - 1] == 7.0)
    A = q4.quantize(x.to(DEV), "mxint8")
    a = to_f32(q4.q4_dequant(A, torch.empty(P, K, device=DEV)))
    ref = grad.wgrad(to_f32(dc), a, None, off)
    bound = _wgrad_bound(to_f32(dc), a, None, off)
    got = q4.q4_grouped_gemm_wgrad(dc.to(DEV), A, None, offd)
    _close(got, ref, bound, "dW")
    assert torch.equal(got, q4.q4_grouped_gemm_wgrad(dc.to(DEV), A, None, offd))
    acc = torch.full((2 * N, K), 2.0, device=DEV)
    q4.q4_grouped_gemm_wgrad(dc.to(DEV), A, None, offd, dW=acc, accumulate=True)
    _close(acc, 2.0 + ref, bound + 2.0 ** -23 * (2.0 + np.abs(ref)), "dW accumulated")
    b = q4.q4_grouped_gemm_wgrad(dc.to(DEV), A, None, offd, dW=torch.empty(2 * N, K, dtype=BF16, device=DEV))
    _close(b, ref, 1.01 * bound + 2.0 ** -8 * np.abs(ref), "dW bf16")


def test_wgrad_of_no_rows_is_zero():
    dc = torch.empty(0, 16, dtype=BF16, device=DEV)
    for A in (torch.empty(0, 64, dtype=BF16, device=DEV), q4.empty_q4("mxint8", 0, 64, device=DEV)):
        assert torch.all(q4.q4_gemm_wgrad(dc, A) == 0)
        off = torch.zeros(4, dtype=I32, device=DEV)
        assert torch.all(q4.q4_grouped_gemm_wgrad(dc, A, None, off) == 0)
        old = torch.ones(48, 64, device=DEV)
        assert torch.all(q4.q4_grouped_gemm_wgrad(dc, A, None, off, dW=old, accumulate=True) == 1)


def test_products_pass_nan_and_inf_on_where_they_belong():
    """An infinity in one row reaches that row's outputs (dgrad) or that expert's (wgrad) and no others."""
    rng = _rng("nan")
    N, K, P = 48, 512, 70
    off = torch.tensor([0, 33, 33, 70], dtype=I32, device=DEV)
    W = q4.quantize(_bf16(rng, 3 * N, K, std=0.02).to(DEV), "mxfp4", layout="tiled")
    dc = _bf16(rng, P, N).to(DEV)
    clean = q4.q4_grouped_gemm_dgrad(dc, off, W, N)
    bad = dc.clone()
    bad[32, 5], bad[40, 7] = float("inf"), float("nan")
    got = q4.q4_grouped_gemm_dgrad(bad, off, W, N)
    rows = torch.ones(P, dtype=torch.bool)
    rows[[32, 40]] = False
    assert torch.equal(got[rows], clean[rows]) and not torch.isfinite(got[32].float()).all()
    assert torch.isnan(got[40].float()).all()
    # nothing of an earlier call's values is left where a sum or a block ends
    for t in (dc, bad):
        q4.q4_grouped_gemm_dgrad(torch.full_like(dc, float("nan")), off, W, N)
        again = q4.q4_grouped_gemm_dgrad(t, off, W, N)
        assert torch.equal(again[rows], clean[rows])
    xq = q4.quantize(_bf16(rng, P, K).to(DEV), "mxint8")
    first = q4.q4_grouped_gemm_wgrad(dc, xq, None, off)
    q4.q4_grouped_gemm_wgrad(torch.full_like(dc, float("nan")), xq, None, off)
    assert torch.equal(q4.q4_grouped_gemm_wgrad(dc, xq, None, off), first)
    x = _bf16(rng, P, K)
    x[34, 3] = float("inf")                     # expert 2
    for A, wide in ((x.to(DEV), 1), (q4.quantize(x.to(DEV), "mxint8"), 32), (q4.quantize(x.to(DEV), "mxfp8"), 32)):
        dW = q4.q4_grouped_gemm_wgrad(dc, A, None, off)
        fin = torch.isfinite(dW)
        assert fin[:2 * N].all() and fin[2 * N:, 32 if wide > 1 else 4:].all()
        assert not fin[2 * N:, 3].any()


# ------------------------------------------------------------ run together

def _layer(fmt_w, fmt_a, T=70, E=6, k=2, K=512, inter=256, seed=1):
    rng = _rng("layer", seed)
    wgu, wd = _bf16(rng, E * 2 * inter, K, std=0.05), _bf16(rng, E * K, inter, std=0.05)
    x, lg = _bf16(rng, T, K), torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32))
    Wgu, Wd = (q4.quantize(w.to(DEV), fmt_w) for w in (wgu, wd))
    return wgu, wd, x, lg, Wgu, Wd, _bf16(rng, T, K)


@pytest.mark.parametrize("fmt_w,fmt_a", [("mxfp4", "mxint8"), ("int4", "mxfp8"), ("nvfp4", "mxint8")])
def test_moe_layer_step(fmt_w, fmt_a):
    """The layer's gradients against the formulas in fp64 on the dequantized weights.  Four bf16 roundings (gate/up, h, y,
    then dh and dgu) of 2^-8 each and the saved activations' (2^-7 of a block's largest value in integers, 2^-4 of each
    value in E4M3) lie on the way of the gradients: 2-norms within 2^-5 (integers) or 2^-3 (E4M3)."""
    log("moe layer step", fmt_w, fmt_a)
    E, k, K, inter = 6, 2, 512, 256
    wgu, wd, x, lg, Wgu, Wd, dout = _layer(fmt_w, fmt_a)
    xd, ld = x.to(DEV), lg.to(DEV)
    out, saved = q4.moe_layer_save(xd, ld, k, Wgu, Wd, inter, fmt=fmt_a)
    dx, dl, dWgu, dWd = q4.moe_layer_backward(saved, dout.to(DEV), Wgu, Wd)
    plain, r = q4.moe_layer(xd, ld, k, Wgu, Wd, inter)
    assert torch.equal(saved.r.inv, r.inv)
    gu_w = oracle.dequant(oracle.quantize(fmt_w, to_f32(wgu))).astype(np.float64).reshape(E, 2 * inter, K)
    d_w = oracle.dequant(oracle.quantize(fmt_w, to_f32(wd))).astype(np.float64).reshape(E, K, inter)
    lt = lg.double().requires_grad_()
    xt = x.double().requires_grad_()
    a, b = torch.from_numpy(gu_w).requires_grad_(), torch.from_numpy(d_w).requires_grad_()
    p = torch.softmax(lt, 1)
    ids = saved.r.ids.cpu().long()
    ref = torch.zeros(x.shape, dtype=torch.float64)
    for j in range(k):
        for e in range(E):
            t = torch.nonzero(ids[:, j] == e)[:, 0]
            z = xt[t] @ a[e].T
            y = (z[:, :inter] * torch.sigmoid(z[:, :inter]) * z[:, inter:]) @ b[e].T
            ref = ref.index_add(0, t, p[t, e, None] * y)
    ref.backward(dout.double())
    lim = 2.0 ** -5 if fmt_a == "mxint8" else 2.0 ** -3
    for name, got, want in (("out", out, ref.detach()), ("dx", dx, xt.grad), ("dlogits", dl, lt.grad),
                            ("dW_gu", dWgu, a.grad.reshape(-1, K)), ("dW_down", dWd, b.grad.reshape(-1, inter))):
        err = float((got.cpu().double() - want).norm() / want.norm())
        log(name, err)
        assert err <= lim, (name, err)
    dx2, dl2, n1, n2 = q4.moe_layer_backward(q4.moe_layer_save(xd, ld, k, Wgu, Wd, inter, fmt=fmt_a, weights_grad=False)[1],
                                             dout.to(DEV), Wgu, Wd)
    assert n1 is None and n2 is None and torch.equal(dx2, dx) and torch.equal(dl2, dl)


def test_moe_layer_step_without_tokens_and_with_one():
    _, _, x, lg, Wgu, Wd, dout = _layer("mxfp4", "mxint8", seed=3)
    for T in (0, 1):
        out, saved = q4.moe_layer_save(x[:T].to(DEV), lg[:T].to(DEV), 2, Wgu, Wd, 256)
        dx, dl, a, b = q4.moe_layer_backward(saved, dout[:T].to(DEV), Wgu, Wd)
        assert out.shape == dx.shape == (T, 512) and dl.shape == (T, 6)
        assert a.shape == (6 * 512, 512) and b.shape == (6 * 512, 256)
        used = torch.zeros(6, dtype=torch.bool)
        used[saved.r.ids.cpu().long().flatten()] = True
        for g in (a, b):
            nz = g.reshape(6, -1).abs().sum(1).cpu() > 0
            assert torch.equal(nz, used)
        for t in (out, dx, dl, a, b):
            assert torch.isfinite(t.float()).all()


def test_moe_layer_step_in_a_graph():
    """The whole step captured and replayed on other data, with eager work between: every replay gives the eager bits."""
    k, inter = 2, 256
    _, _, x, lg, Wgu, Wd, dout = _layer("mxfp4", "mxint8", seed=2)
    xd, ld, dd = x.to(DEV), lg.to(DEV), dout.to(DEV)

    def step():
        out, saved = q4.moe_layer_save(xd, ld, k, Wgu, Wd, inter)
        return (out,) + q4.moe_layer_backward(saved, dd, Wgu, Wd)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(3):
        xd.copy_(_bf16(_rng("replay", i), *x.shape))
        ld.copy_(torch.from_numpy(_rng("replayl", i).standard_normal(lg.shape).astype(np.float32)))
        eager = [t.clone() for t in step()]
        for t in outs:
            t.fill_(3.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b), i


def test_calls_on_another_stream():
    """Each call on a side stream behind the stream that makes its inputs."""
    s = torch.cuda.Stream()
    rng = _rng("stream")
    dc, x = _bf16(rng, 200, 64).to(DEV), _bf16(rng, 200, 256).to(DEV)
    ids = torch.from_numpy(_ids(rng, 6000, 4, 16, 0.1)).to(DEV)
    want = (q4.q4_gemm_wgrad(dc, q4.quantize(x, "mxint8")), *q4.q4_moe_sort(ids, 16)[::2])
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        s.wait_stream(torch.cuda.current_stream())
        q = q4.empty_q4("mxint8", 200, 256, device=DEV)
        s.wait_stream(torch.cuda.current_stream())
        q4.q4_quantize(x, q, stream=stream)
        got = (q4.q4_gemm_wgrad(dc, q, stream=stream), *q4.q4_moe_sort(ids, 16, stream=stream)[::2])
        torch.cuda.current_stream().wait_stream(s)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ("mxint8", "mxfp8"))
def test_wgrad_dense_of_many_rows(kind):
    """A dense layer in the largest block, without gather; every size odd for it."""
    log("wgrad many rows", kind)
    rng = _rng("wgradm")
    M, N, K = 1061, 4104, 4128
    dc = _bf16(rng, M, N)
    A = q4.quantize(_bf16(rng, M, K).to(DEV), kind)
    a = to_f32(q4.q4_dequant(A, torch.empty(M, K, device=DEV)))
    off = np.array([0, M], np.int32)
    bound = _wgrad_bound(to_f32(dc), a, None, off)
    ref = grad.wgrad(to_f32(dc), a, None, off)
    _close(q4.q4_gemm_wgrad(_strided(dc), A), ref, bound, "dW")


@pytest.mark.parametrize("gathered", (True, False))
def test_products_of_many_experts(gathered):
    """More blocks than the XCDs' first turns hold, experts of very different sizes, empty ones among them."""
    log("many experts", gathered)
    rng = _rng("many", gathered)
    E, P, N, K, T = 331, 1777, 72, 384, 1800
    off = _segments(rng, E, P, "empty_first")
    off[100:130] = off[100]
    w, dc, x = _bf16(rng, E * N, K, std=0.02), _bf16(rng, P, N), _bf16(rng, T, K)
    W = q4.quantize(w.to(DEV), "mxfp4")
    wd = oracle.dequant(oracle.quantize("mxfp4", to_f32(w)))
    offd = torch.from_numpy(off).to(DEV)
    ref = grad.dgrad(to_f32(dc), off, wd, N)
    _close(q4.q4_grouped_gemm_dgrad(dc.to(DEV), offd, W, N), ref,
           _dgrad_bound(to_f32(dc), off, wd, N, ref, True), "dA")
    gather = rng.integers(0, T, P).astype(np.int32) if gathered else None
    gd = torch.from_numpy(gather).to(DEV) if gathered else None
    for kind in ("bf16", "mxint8"):
        A = x.to(DEV) if kind == "bf16" else q4.quantize(x.to(DEV), kind)
        a = to_f32(x) if kind == "bf16" else to_f32(q4.q4_dequant(A, torch.empty(T, K, device=DEV)))
        a_ref = a if gathered else a[:P]
        _close(q4.q4_grouped_gemm_wgrad(dc.to(DEV), A, gd, offd), grad.wgrad(to_f32(dc), a_ref, gather, off),
               _wgrad_bound(to_f32(dc), a_ref, gather, off), (kind, "dW"))


def test_results_do_not_vary():
    rng = _rng("again")
    dc = _bf16(rng, 3000, 128).to(DEV)
    A = q4.quantize(_bf16(rng, 3000, 256).to(DEV), "mxint8")
    off = torch.from_numpy(_segments(rng, 5, 3000, "")).to(DEV)
    W = q4.quantize(_bf16(rng, 128, 512, std=0.02).to(DEV), "mxfp4", layout="tiled")
    first = None
    for _ in range(3):
        now = (q4.q4_gemm_wgrad(dc, A), q4.q4_grouped_gemm_wgrad(dc, A, None, off), q4.q4_gemm_dgrad(dc, W))
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(now, first))
