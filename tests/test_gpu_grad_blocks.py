"""The gradient products in every block that they choose by size (64, 128 and
256 rows, with the sum whole and in parts), for every format and layout.  Each
case names the block it is for and asks the library whether its sizes take it,
so that another rule cannot leave one unrun.

The reference sums, in fp64, what enters the matrix cores: the weights as the
oracle dequantizes them, INT4's (with or without a zero point) rounded once to
bf16 as include/q4.h says.  Products of bf16 values are exact in fp32, so
what is left are the sums, off by (n + 8) 2^-23 S (n terms, S the sum of their
magnitudes; NVFP4's tensor scale is one of the 8), and one rounding to bf16,
2^-8 of the value.  A summed row left out or taken twice is S / n on average:
far outside at every size here.
"""
import ctypes
import zlib

import numpy as np
import pytest
import torch

import oracle
import w4_gemm_amd as q4
from oracle import grad
from q4_helpers import log, to_f32

DEV = "cuda:0"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
FORMATS = ("int4", "mxfp4", "nvfp4", "int4_zp")
KINDS = ("bf16", "mxint8", "mxfp8")


def _rng(*key):
    return np.random.default_rng([zlib.crc32(k.encode()) if isinstance(k, str) else k for k in key])


def _bf16(rng, *shape, std=1.0):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(std)).to(BF16)


def _strided(t, extra=16):
    """t on the GPU as a view whose rows are `extra` elements further apart, the gaps NaN."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=DEV)
    buf[:, :t.shape[1]] = t.to(DEV)
    return buf[:, :t.shape[1]]


def _close(got, ref, bound, what):
    got = to_f32(got).astype(np.float64)
    assert got.shape == ref.shape, (got.shape, ref.shape)
    bad = np.argwhere(~(np.abs(got - ref) <= bound))
    assert bad.size == 0, (what, len(bad), [(i.tolist(), got[tuple(i)], ref[tuple(i)], bound[tuple(i)]) for i in bad[:3]])


def _entering(fmt, w):
    """The weight's values in the products."""
    wd = oracle.dequant(oracle.quantize(fmt, to_f32(w)))
    return to_f32(torch.from_numpy(wd).to(BF16)) if fmt.startswith("int4") else wd


# rows of a block, whether in parts, N, K, the experts' offsets (one pair: a dense weight).  Stages of 32 summed rows (64
# in blocks of 256): odd and even numbers of them, the last one whole and not.  Experts end in less, as much and more than
# half a block.
DGRAD = [
    (64, False, 264, 1024, (0, 130)),
    (64, False, 208, 512, (2, 42, 42, 170, 263)),
    (64, True, 1048, 1024, (0, 33)),
    (64, True, 1040, 512, (1, 14, 14, 31)),
    (128, False, 200, 7680, (0, 1060)),
    (128, False, 232, 7680, (0, 1100)),
    (128, False, 208, 7680, (3, 171, 399, 463, 463, 703)),
    (128, False, 240, 7680, (0, 129, 193, 450, 834, 835)),
    (256, False, 200, 7680, (0, 2101)),
    (256, False, 264, 7680, (0, 2304)),
    (256, False, 208, 4608, (5, 2112, 4216)),
    (256, False, 272, 4608, (0, 0, 2049, 6145)),
]


def _dgrad_plan(N, K, off):
    # (rows behind the last expert belong to the call)
    return q4.q4_dgrad_plan(off[-1] + (5 if len(off) > 2 else 0), len(off) - 1, N, K)


@pytest.mark.parametrize("rows,in_parts,N,K,off", DGRAD)
def test_dgrad_sizes_take_their_block(rows, in_parts, N, K, off):
    got, parts = _dgrad_plan(N, K, off)
    assert got == rows and (parts > 1) == in_parts


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ("rows", "tiled"))
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,in_parts,N,K,off", DGRAD)
def test_dgrad_blocks(rows, in_parts, N, K, off, fmt, layout):
    log("dgrad blocks", rows, in_parts, N, K, off, fmt, layout)
    assert _dgrad_plan(N, K, off)[0] == rows
    rng = _rng("dgradb", N, K, off[-1])
    E, end = len(off) - 1, off[-1]
    P = end + (5 if E > 1 else 0)
    w, dc = _bf16(rng, E * N, K, std=0.02), _bf16(rng, P, N)
    W, wd = q4.quantize(w.to(DEV), fmt, layout=layout), _entering(fmt, w)
    dc[:off[0]], dc[end:] = float("nan"), float("nan")          # rows outside every expert are neither read nor written
    offd = torch.tensor(off, dtype=I32, device=DEV)
    out = _strided(torch.full((P, K), 7.0, dtype=BF16))
    run = (lambda t: q4.q4_gemm_dgrad(t, W, dA=out)) if E == 1 else \
        (lambda t: q4.q4_grouped_gemm_dgrad(t, offd, W, N, dA=out))
    run(_strided(dc))
    first = out.clone()
    d = to_f32(dc)
    rows_of = slice(off[0], end)
    ref = grad.dgrad(d, off, wd, N)[rows_of]
    s = grad.dgrad(np.abs(d), off, np.abs(wd), N)[rows_of]
    _close(out[rows_of], ref, 2.0 ** -8 * np.abs(ref) + (N + 8) * 2.0 ** -23 * s, "dA")
    assert torch.all(out[:off[0]] == 7.0) and torch.all(out[end:] == 7.0)
    run(dc.to(DEV))
    assert torch.equal(out, first)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,layout", [("int4", "tiled"), ("mxfp4", "rows"), ("nvfp4", "tiled"), ("int4_zp", "rows")])
def test_dgrad_parts_of_the_block_of_128_rows(fmt, layout):
    """As many blocks of 128 rows as CUs and a long sum: two parts, the last rows in half a block."""
    log("dgrad 128 in parts", fmt, layout)
    M, N, K = 1925, 6424, 4096
    assert q4.q4_dgrad_plan(M, 1, N, K) == (128, 2)
    rng = _rng("dgradp")
    w, dc = _bf16(rng, N, K, std=0.02), _bf16(rng, M, N)
    W, wd = q4.quantize(w.to(DEV), fmt, layout=layout), _entering(fmt, w)
    got = q4.q4_gemm_dgrad(dc.to(DEV), W)
    assert torch.equal(got, q4.q4_gemm_dgrad(dc.to(DEV), W))
    rows = np.r_[0:16, 100:140, 1000:1016, M - 70:M]             # the last blocks of 128 and 64 rows whole
    d, off = to_f32(dc)[rows], (0, len(rows))
    ref, s = grad.dgrad(d, off, wd, N), grad.dgrad(np.abs(d), off, np.abs(wd), N)
    _close(got[torch.from_numpy(rows).to(DEV)], ref, 2.0 ** -8 * np.abs(ref) + (N + 8) * 2.0 ** -23 * s, "dA")


# rows of a block for operands in 8 bits, whether in parts, N, K, the experts' offsets.  (bf16: 128 where these have 256.)
WGRAD = [
    (64, False, 72, 288, (0, 20, 20, 49, 60)),
    (64, True, 264, 288, (0, 1500)),
    (64, True, 72, 288, (3, 1400, 1400, 2999)),
    (128, True, 648, 32, (0, 15989)),
    (128, True, 520, 32, (7, 9001, 9001, 15990)),
    (128, False, 2056, 4128, (0, 211)),
    (128, False, 1032, 2336, (2, 251, 251, 610)),
    (256, False, 4104, 4128, (0, 1061)),
    (256, False, 2568, 2336, (0, 299, 640, 931)),
    (256, False, 2568, 2336, (9, 459, 459, 1090)),
]


def _wgrad_plan(N, K, off, a_is_bf16):
    # (rows behind the last expert belong to the call)
    return q4.q4_wgrad_plan(off[-1] + (3 if len(off) > 2 else 0), len(off) - 1, N, K, a_is_bf16)


@pytest.mark.parametrize("rows,in_parts,N,K,off", WGRAD)
def test_wgrad_sizes_take_their_block(rows, in_parts, N, K, off):
    for a_is_bf16 in (False, True):
        got, parts = _wgrad_plan(N, K, off, a_is_bf16)
        assert got == (min(rows, 128) if a_is_bf16 else rows) and (parts > 1) == in_parts


@pytest.mark.gpu
@pytest.mark.parametrize("gathered", (True, False))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,in_parts,N,K,off", WGRAD)
def test_wgrad_blocks(rows, in_parts, N, K, off, kind, gathered):
    log("wgrad blocks", rows, in_parts, N, K, off, kind, gathered)
    rng = _rng("wgradb", N, K, off[-1])
    assert _wgrad_plan(N, K, off, kind == "bf16")[0] == (min(rows, 128) if kind == "bf16" else rows)
    E, end = len(off) - 1, off[-1]
    P = end + (3 if E > 1 else 0)
    T = P // 2 + 5 if gathered else P
    dc, x = _bf16(rng, P, N), _bf16(rng, T, K)
    dc[:off[0]], dc[end:] = float("nan"), float("nan")
    x[:, ::37] *= 20
    A = x.to(DEV) if kind == "bf16" else q4.quantize(x.to(DEV), kind)
    a = to_f32(x) if kind == "bf16" else to_f32(q4.q4_dequant(A, torch.empty(T, K, device=DEV)))
    gather = None
    if gathered:
        gather = rng.integers(0, T, P).astype(np.int32)
        gather[[off[0], end - 1]] = [-1, T]                    # rows outside A read zeros
    offd = torch.tensor(off, dtype=I32, device=DEV)
    gd = None if gather is None else torch.from_numpy(gather).to(DEV)
    run = (lambda dW, acc=False: q4.q4_gemm_wgrad(dcd, A, dW=dW, accumulate=acc)) if E == 1 and not gathered else \
        (lambda dW, acc=False: q4.q4_grouped_gemm_wgrad(dcd, A, gd, offd, dW=dW, accumulate=acc))
    dcd = _strided(dc)
    d = np.nan_to_num(to_f32(dc))
    ref, s = grad.wgrad(d, a, gather, off), grad.wgrad(np.abs(d), np.abs(a), gather, off)
    n = max(b - c for b, c in zip(off[1:], off[:-1]))
    bound = (n + 8) * 2.0 ** -23 * s
    out = torch.full((E * N + 1, K + 8), 3.0, device=DEV)
    dW = out[:, :K]
    run(dW)
    _close(dW[:E * N], ref, bound, "dW")
    first = dW[:E * N].clone()
    run(dW, True)
    _close(dW[:E * N], 2 * ref, 2 * bound + 2.0 ** -23 * np.abs(ref), "dW twice")
    assert torch.all(out[E * N:] == 3.0) and torch.all(out[:, K:] == 3.0)
    low = run(torch.empty(E * N, K, dtype=BF16, device=DEV))
    assert torch.equal(low, first.to(BF16))                    # the same fp32 sums, rounded once


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_layer_step_on_tiled_weights(fmt):
    """The layer's backward pass through tiled weights has the bits of that through row-major ones; its forward pass and
    gradients are the formulas' in fp64 on the dequantized weights (the four bf16 roundings and the saved activations' on
    the way, as 2-norms: 2^-5)."""
    log("layer step, tiled", fmt)
    T, E, k, K, inter = 70, 6, 2, 512, 512
    rng = _rng("layert")
    wgu, wdn = _bf16(rng, E * 2 * inter, K, std=0.05), _bf16(rng, E * K, inter, std=0.05)
    x, lg, dout = _bf16(rng, T, K), torch.from_numpy(rng.standard_normal((T, E), dtype=np.float32)), _bf16(rng, T, K)
    both = [[q4.quantize(w.to(DEV), fmt, layout=layout) for w in (wgu, wdn)] for layout in ("tiled", "rows")]
    out, saved = q4.moe_layer_save(x.to(DEV), lg.to(DEV), k, *both[0], inter)
    grads, again = (q4.moe_layer_backward(saved, dout.to(DEV), *w) for w in both)
    for a, b in zip(grads, again):
        assert torch.equal(a, b)
    gu_w = torch.from_numpy(oracle.dequant(oracle.quantize(fmt, to_f32(wgu)))).double().reshape(E, 2 * inter, K)
    d_w = torch.from_numpy(oracle.dequant(oracle.quantize(fmt, to_f32(wdn)))).double().reshape(E, K, inter)
    leaves = [t.requires_grad_() for t in (x.double(), lg.double(), gu_w, d_w)]
    p, ids = torch.softmax(leaves[1], 1), saved.r.ids.cpu().long()
    ref = torch.zeros(T, K, dtype=torch.float64)
    for j in range(k):
        for e in range(E):
            t = torch.nonzero(ids[:, j] == e)[:, 0]
            z = leaves[0][t] @ gu_w[e].T
            y = (z[:, :inter] * torch.sigmoid(z[:, :inter]) * z[:, inter:]) @ d_w[e].T
            ref = ref.index_add(0, t, p[t, e, None] * y)
    ref.backward(dout.double())
    for name, got, want in zip(("out", "dx", "dlogits", "dW_gu", "dW_down"), (out, *grads),
                               (ref.detach(), *(t.grad for t in leaves))):
        err = float((got.cpu().double() - want.reshape(got.shape)).norm() / want.norm())
        log(name, err)
        assert err <= 2.0 ** -5, (name, err)


def test_plans_refuse():
    """The queries' errors are those of the workspace queries; nothing is launched for empty products."""
    L = q4.lib()
    rows, parts = ctypes.c_int32(7), ctypes.c_int32(7)
    for f, tail in ((L.q4_dgrad_plan, ()), (L.q4_wgrad_plan, (0,))):
        assert f(4, 1, 64, 256, *tail, None, ctypes.byref(parts)) == -1
        assert f(4, 1, 64, 256, *tail, ctypes.byref(rows), None) == -1
        for bad in ((-1, 1, 64, 256), (4, 65536, 64, 256), (4, 1, (1 << 21) + 8, 256), (4, 1, 64, -128)):
            assert f(*bad, *tail, ctypes.byref(rows), ctypes.byref(parts)) == -2
        assert rows.value == parts.value == 7
    for got in (q4.q4_dgrad_plan(0, 1, 64, 256), q4.q4_dgrad_plan(4, 0, 64, 256), q4.q4_wgrad_plan(4, 1, 0, 256),
                q4.q4_wgrad_plan(4, 1, 64, 0, True)):
        assert got == (0, 0)
