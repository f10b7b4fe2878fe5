"""The norm, its 8-bit outputs and its gradient on the GPU against the oracle.

The sum of squares adds K <= 32768 positive terms in fp32: 32 in a lane one by
one, then 10 pairwise steps, each off by at most 2^-24: below 2^-18 of the sum,
half of that in its root, and a few products more.  FP32 = 2^-18 bounds all of
it relative to a value; a bf16 output adds 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import w4_gemm_amd as q4
from oracle import block as ob

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
FP32 = 2.0 ** -18
EPS = 1e-6


def make(rows, cols, seed=0, wt=BF16):
    g = torch.Generator().manual_seed(seed * 1000003 + rows * 8191 + cols)
    x, res = torch.randn(rows, cols, generator=g).to(BF16), (torch.randn(rows, cols, generator=g) * 2).to(BF16)
    return x, res, (1 + 0.2 * torch.randn(cols, generator=g)).to(wt)


def n64(t):
    return t.detach().cpu().double().numpy()


def near(got, ref, rel, floor=0.0, what=""):
    g = n64(got) if isinstance(got, torch.Tensor) else got
    bad = np.argwhere(~(np.abs(g - ref) <= rel * np.abs(ref) + floor))
    assert bad.size == 0, (what, len(bad), [(tuple(i), g[tuple(i)], ref[tuple(i)]) for i in bad[:3]])


def check8(q, y, fmt):
    """Codes and scales of a per-row output against y in 64 bits: the scale within FP32 of amax / top, each code one
    that its quotient, known within FP32, rounds to."""
    top = 127.0 if fmt == "int8_row" else 448.0
    s = np.maximum(np.abs(y).max(1), 1e-12) / top
    near(q.scales, s, FP32, what="scale")
    t = y / s[:, None]
    if fmt == "int8_row":
        c = q.codes.cpu().double().numpy()
        assert (np.abs(c - t) <= 0.5 + FP32 * np.abs(t)).all()
    else:
        rows = q.rows
        codes = q.codes.cpu()
        if q.layout == q4.LAYOUT_TILED:
            codes = untile8(codes, rows, q.cols)
        v = codes.view(torch.float8_e4m3fn).double().numpy()
        # half a step: 2^-4 of the value, 2^-10 below the least normal
        assert (np.abs(v - t) <= np.maximum(2.0 ** -4 * np.abs(t), 2.0 ** -10) + FP32 * np.abs(t)).all()


def untile8(codes, rows, cols):
    """The tiled order of include/q4.h for FP8 rows: operand byte 4 (2w + h) + i of lane 16 g + n is k = 32g + 8w + 2i + h."""
    RT, S = (rows + 15) // 16, cols // 128
    c = codes.view(RT, S, 2, 4, 16, 2, 2, 4)       # t, s, w >> 1, g, n, w & 1, h, i
    c = c.permute(0, 4, 1, 3, 2, 5, 7, 6)          # t, n, s, g, w >> 1, w & 1, i, h
    return c.reshape(RT * 16, cols)[:rows].contiguous()


SIZES = [(1, 8), (3, 16), (5, 64), (4, 504), (2, 512), (7, 520), (6, 2048), (3, 2056), (1, 4096), (2, 7168), (3, 8192),
         (2, 8200), (1, 16384), (2, 32768), (259, 128), (33, 1024)]


@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, wt):
    x, res, w = make(rows, cols, wt=wt)
    h, y, q = q4.q4_rmsnorm(x.cuda(), w.cuda(), EPS, residual=res.cuda())
    want = (x.float() + res.float()).to(BF16)
    assert q is None and torch.equal(h.cpu(), want)
    near(y, ob.rmsnorm(n64(want), n64(w), EPS), 2.0 ** -8 + FP32)
    xg = x.cuda()
    h, y, _ = q4.q4_rmsnorm(xg, w.cuda(), 0.5)
    assert h is xg
    near(y, ob.rmsnorm(n64(x), n64(w), 0.5), 2.0 ** -8 + FP32)


@pytest.mark.parametrize("fmt,layout", [("int8_row", 0), ("fp8_row", 0), ("fp8_row", 1)])
@pytest.mark.parametrize("rows,cols", SIZES[1:])
def test_eight_bits(rows, cols, fmt, layout):
    if cols % 16 or (layout and cols % 512):
        pytest.skip("no such tensor")
    x, res, w = make(rows, cols, 1)
    q = q4.empty_q4(fmt, rows, cols, layout=layout)
    q.codes.view(torch.uint8).fill_(0x55)
    h, y, got = q4.q4_rmsnorm(x.cuda(), w.cuda(), EPS, residual=res.cuda(), y_q=q)
    assert y is None and got is q
    ref = ob.rmsnorm(n64((x.float() + res.float()).to(BF16)), n64(w), EPS)
    check8(q, ref, fmt)
    if layout and rows % 16:   # padding rows hold code 0
        full = untile8(q.codes.cpu(), (rows + 15) // 16 * 16, cols)
        assert (full[rows:] == 0).all()
    # both outputs at once: the same codes, and y as without them
    y2, q2 = torch.empty(rows, cols, dtype=BF16, device="cuda"), q4.empty_q4(fmt, rows, cols, layout=layout)
    q4.q4_rmsnorm(x.cuda(), w.cuda(), EPS, residual=res.cuda(), y=y2, y_q=q2)
    assert torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales)
    assert torch.equal(y2, q4.q4_rmsnorm(x.cuda(), w.cuda(), EPS, residual=res.cuda())[1])


def test_eight_bits_small_and_large_values():
    x = torch.randn(6, 256).to(BF16)
    x[0], x[1], x[2], x[3] = 0, x[1] * 1e-15, x[2] * 1e15, x[3] * 1e-4
    w = torch.ones(256, dtype=F32)
    for fmt in ("int8_row", "fp8_row"):
        q = q4.empty_q4(fmt, 6, 256)
        q4.q4_rmsnorm(x.cuda(), w.cuda(), EPS, y_q=q)
        check8(q, ob.rmsnorm(n64(x), n64(w), EPS), fmt)


@pytest.mark.parametrize("cols", [128, 2048, 4096, 16384])
def test_rows_without_numbers(cols):
    """Infinities, NaN, squares past fp32 and zeros without eps give NaN there and leave the other rows alone."""
    x = torch.randn(8, cols).to(BF16)
    clean = x.clone()
    x[1, 3], x[3, cols - 1], x[4, 7], x[6] = float("inf"), float("nan"), 3e38, 0
    w = torch.ones(cols, dtype=BF16).cuda()
    bad = [1, 3, 4, 6]
    good = [0, 2, 5, 7]
    for fmt in ("int8_row", "fp8_row"):
        q, y = q4.empty_q4(fmt, 8, cols), torch.empty(8, cols, dtype=BF16, device="cuda")
        q4.q4_rmsnorm(x.cuda(), w, 0.0, y=y, y_q=q)
        d = q4.q4_dequant(q, torch.empty(8, cols, dtype=F32, device="cuda")).cpu()
        assert torch.isnan(y.cpu()[bad]).all() and torch.isnan(d[bad]).all()
        near(y[good], ob.rmsnorm(n64(clean)[good], np.ones(cols), 0.0), 2.0 ** -8 + FP32)
        assert not torch.isnan(d[good]).any()


def test_strides_and_in_place():
    rows, cols = 37, 1024
    x, res, w = make(rows, cols, 2)
    want_h, want_y, _ = q4.q4_rmsnorm(x.cuda(), w.cuda(), EPS, residual=res.cuda())
    bufs = [torch.full((rows, cols + 24), 9.0, dtype=BF16, device="cuda") for _ in range(4)]
    xs, rs, hs, ys = (b[:, 8:8 + cols] for b in bufs)
    xs.copy_(x), rs.copy_(res)
    h, y, _ = q4.q4_rmsnorm(xs, w.cuda(), EPS, residual=rs, h=hs, y=ys)
    assert h is hs and y is ys and torch.equal(h, want_h) and torch.equal(y, want_y)
    for b in bufs:
        assert (b[:, :8] == 9).all() and (b[:, 8 + cols:] == 9).all()
    r2 = res.cuda()
    h, y, _ = q4.q4_rmsnorm(x.cuda(), w.cuda(), EPS, residual=r2, h=r2)
    assert h is r2 and torch.equal(r2, want_h) and torch.equal(y, want_y)
    x2 = x.cuda()
    h, y, _ = q4.q4_rmsnorm(x2, w.cuda(), EPS, residual=res.cuda(), h=x2)
    assert torch.equal(x2, want_h) and torch.equal(y, want_y)


def test_no_rows():
    w = torch.ones(64, dtype=BF16).cuda()
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    assert q4.q4_rmsnorm(e, w)[1].shape == (0, 64)
    dx, dw = q4.q4_rmsnorm_backward(e, e, w)
    assert dx.shape == (0, 64) and (dw == 0).all()
    dw.fill_(2.0)
    q4.q4_rmsnorm_backward(e, e, w, dweight=dw, accumulate=True)
    assert (dw == 2.0).all()


def grad_ref(dy, h, w, eps, dh=None):
    """(dx, dw) and the sums of magnitudes that their roundings go by."""
    d, v, wf = n64(dy), n64(h), n64(w)
    dx, dw = ob.rmsnorm_backward(d, v, wf, eps)
    r = 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    g, n = np.abs(d * wf), np.abs(v * r)
    size = r * (g + n * (g * n).mean(1, keepdims=True))
    if dh is not None:
        dx, size = dx + n64(dh), size + np.abs(n64(dh))
    return dx, dw, size, np.abs(d * v * r).sum(0)


@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SIZES + [(2049, 256), (600, 4096), (1, 2048)])
def test_backward(rows, cols, wt):
    h, dh, w = make(rows, cols, 3, wt)
    dy = (torch.randn(rows, cols, generator=torch.Generator().manual_seed(rows)) * 0.01).to(BF16)
    for add in (None, dh):
        dx, dw = q4.q4_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), EPS, dh=None if add is None else add.cuda())
        rx, rw, size, sw = grad_ref(dy, h, w, EPS, add)
        near(dx, rx, 2.0 ** -8, 2.0 ** -16 * size, "dx")
        # at most 5 + 32 + 16 additions one behind the other for these rows: 2^-18 of the sum of magnitudes, and n's own error
        near(dw, rw, 0.0, 2.0 ** -17 * sw, "dw")
        more = torch.ones(cols, dtype=F32, device="cuda")
        q4.q4_rmsnorm_backward(dy.cuda(), h.cuda(), w.cuda(), EPS, dweight=more, accumulate=True)
        near(more, rw + 1, 2.0 ** -23, 2.0 ** -17 * sw, "accumulated")


def test_backward_without_weight_and_in_place():
    h, dh, w = make(65, 1536, 4)
    dy = torch.randn(65, 1536).to(BF16).cuda()
    dx, dw = q4.q4_rmsnorm_backward(dy, h.cuda(), w.cuda(), EPS, dh=dh.cuda())
    alone, none = q4.q4_rmsnorm_backward(dy, h.cuda(), w.cuda(), EPS, dh=dh.cuda(), weight_grad=False)
    assert none is None and torch.equal(alone, dx)
    at = dh.cuda()
    out, dw2 = q4.q4_rmsnorm_backward(dy, h.cuda(), w.cuda(), EPS, dh=at, dx=at)
    assert out is at and torch.equal(at, dx) and torch.equal(dw2, dw)
    at = dy.clone()
    out, dw2 = q4.q4_rmsnorm_backward(at, h.cuda(), w.cuda(), EPS, dh=dh.cuda(), dx=at)
    assert torch.equal(out, dx) and torch.equal(dw2, dw)
    wide = torch.full((65, 1600), 5.0, dtype=BF16, device="cuda")
    out, _ = q4.q4_rmsnorm_backward(dy, h.cuda(), w.cuda(), EPS, dh=dh.cuda(), dx=wide[:, 16:1552])
    assert torch.equal(out, dx) and (wide[:, :16] == 5).all() and (wide[:, 1552:] == 5).all()


def test_backward_is_the_same_every_time():
    h, dh, w = make(5000, 768, 5)
    dy = torch.randn(5000, 768).to(BF16).cuda()
    first = q4.q4_rmsnorm_backward(dy, h.cuda(), w.cuda(), EPS, dh=dh.cuda())
    for _ in range(3):
        again = q4.q4_rmsnorm_backward(dy, h.cuda(), w.cuda(), EPS, dh=dh.cuda())
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_backward_rows_without_numbers():
    h, _, w = make(9, 640, 6)
    dy = torch.randn(9, 640).to(BF16)
    rx, rw, size, sw = grad_ref(dy, h, w, EPS)
    bad = h.clone()
    bad[4, 100] = float("inf")
    dx, dw = q4.q4_rmsnorm_backward(dy.cuda(), bad.cuda(), w.cuda(), EPS)
    assert torch.isnan(dx[4]).all() and torch.isnan(dw).all()
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    near(dx[keep], rx[keep], 2.0 ** -8, (2.0 ** -16 * size)[keep])


def test_graph_and_streams():
    """Forward and backward captured together and replayed with new inputs; two streams at once, each with its own."""
    h, dh, w = make(130, 2560, 7)
    wg, x, res = w.cuda(), h.cuda(), dh.cuda()
    dy = torch.randn(130, 2560).to(BF16).cuda()

    def step():
        q = q4.empty_q4("int8_row", 130, 2560)
        hh, y, _ = q4.q4_rmsnorm(x, wg, EPS, residual=res, y_q=q)
        return (hh, q.codes, q.scales, *q4.q4_rmsnorm_backward(dy, hh, wg, EPS, dh=dy))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(torch.randn(130, 2560).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b), i
    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(5):
                got.append(step())
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)


def test_feeds_the_products():
    """Norm in 8 bits and the products that read it: W8A8 from int8_row, W4A8 from fp8_row in both layouts."""
    rows, K, N = 40, 1024, 264
    x, res, w = make(rows, K, 8)
    wq = (torch.randn(N, K) * 0.05).to(BF16).cuda()
    for fmt, layout, wf in (("int8_row", 0, "int8_row"), ("fp8_row", 0, "int4"), ("fp8_row", 1, "int4")):
        a = q4.empty_q4(fmt, rows, K, layout=layout)
        q4.q4_rmsnorm(x.cuda(), w.cuda(), EPS, residual=res.cuda(), y_q=a)
        W = q4.quantize(wq, wf, layout=layout)
        C = q4.q4_gemm(a, W, torch.empty(rows, N, dtype=BF16, device="cuda"))
        ad = n64(q4.q4_dequant(a, torch.empty(rows, K, dtype=F32, device="cuda")))
        wd = n64(q4.q4_dequant(W, torch.empty(N, K, dtype=F32, device="cuda")))
        ref, size = ad @ wd.T, np.abs(ad) @ np.abs(wd).T
        near(C, ref, 2.0 ** -8, 2.0 ** -16 * size, fmt)


@pytest.mark.parametrize("rows,cols", [(6200, 8192), (50000, 1008)])
def test_longer_than_the_caches(rows, cols):
    """Sizes at which rows are read and written past the caches: the same values as for the rows alone."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, res, dy, dh = (torch.randn(rows, cols, device="cuda", generator=g).to(BF16) for _ in range(4))
    w = torch.rand(cols, device="cuda", generator=g).to(BF16)
    pick = [0, 1, rows // 2, rows - 2, rows - 1]
    for fmt in ("int8_row", "fp8_row"):
        q, y = q4.empty_q4(fmt, rows, cols), torch.empty_like(x)
        h, _, _ = q4.q4_rmsnorm(x, w, EPS, residual=res, y=y, y_q=q)
        small = q4.empty_q4(fmt, len(pick), cols)
        hs, ys, _ = q4.q4_rmsnorm(x[pick], w, EPS, residual=res[pick], y=torch.empty_like(x[pick]), y_q=small)
        assert torch.equal(h[pick], hs) and torch.equal(y[pick], ys)
        assert torch.equal(q.codes[pick], small.codes) and torch.equal(q.scales[pick], small.scales)
    assert torch.equal(h, (x.float() + res.float()).to(BF16))
    dx, dw = q4.q4_rmsnorm_backward(dy, h, w, EPS, dh=dh)
    assert torch.equal(dx[pick], q4.q4_rmsnorm_backward(dy[pick], h[pick], w, EPS, dh=dh[pick])[0])
    ref, size = torch.zeros(cols, dtype=torch.float64, device="cuda"), torch.zeros(cols, dtype=torch.float64, device="cuda")
    for a, b in zip(dy.split(4096), h.split(4096)):
        n = b.double() * torch.rsqrt(b.double().square().mean(1, keepdim=True) + EPS) * a.double()
        ref, size = ref + n.sum(0), size + n.abs().sum(0)
    # sums of at most 98 rows one behind the other, then of 16 and 32 parts: below 2^-17 of the magnitudes
    assert ((dw.double() - ref).abs() <= 2.0 ** -16 * size).all()
