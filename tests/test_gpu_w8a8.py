"""Rows in 8-bit integers and their product on the GPU against the oracle.

Codes and scales are equal bit for bit.  A product differs from the exact one by
the conversion of the sum to fp32 (2^-24 of it), two fp32 multiplications (2^-24
each) and the rounding to bf16 (2^-8 at most half a step, in all bounded by
2^-8 + 2^-22 of the value); nothing in it depends on the order of the sum.
"""
import numpy as np
import pytest
import torch

import w4_gemm_amd as q4
from oracle import block as ob

pytestmark = pytest.mark.gpu
REL = 2.0 ** -8 + 2.0 ** -22


def codes(rng, rows, cols, full=False):
    """Codes -127..127 (with full: -128 too, which a caller may write)."""
    return rng.integers(-128 if full else -127, 128, (rows, cols)).astype(np.int8)


def tensor(c, s, dev="cuda"):
    return q4.Q4Tensor(q4.INT8_ROW, c.shape[0], c.shape[1], torch.from_numpy(c).to(dev), torch.from_numpy(s).to(dev))


def operand(rng, rows, cols, full=False):
    c, s = codes(rng, rows, cols, full), rng.uniform(0.001, 0.1, rows).astype(np.float32)
    return c, s, tensor(c, s)


def check(got, ref):
    g = got.float().cpu().numpy().astype(np.float64)
    bad = np.argwhere(np.abs(g - ref) > REL * np.abs(ref))
    assert bad.size == 0, (len(bad), bad[:3].tolist(), [(g[tuple(i)], ref[tuple(i)]) for i in bad[:3]])


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (5, 512), (4, 528), (7, 2048), (2, 2064), (3, 4096), (2, 8192),
                                       (2, 8208), (1, 32768), (2, 32784), (1, 70000), (257, 128)])
def test_quantize(rows, cols):
    rng = np.random.default_rng(rows * 100003 + cols)
    x = torch.from_numpy(rng.standard_normal((rows, cols)).astype(np.float32)).bfloat16()
    x[0, cols // 2] = 20.0
    q = q4.quantize(x.cuda(), "int8_row")
    c, s = ob.int8_rows(x.float().numpy())
    assert np.array_equal(q.codes.cpu().numpy(), c)
    assert np.array_equal(q.scales.cpu().numpy(), s)
    for dt in (torch.bfloat16, torch.float32):
        d = q4.q4_dequant(q, torch.empty(rows, cols, dtype=dt, device="cuda"))
        want = (torch.from_numpy(c).float() * torch.from_numpy(s)[:, None]).to(dt)
        assert torch.equal(d.cpu(), want)


def test_quantize_every_value():
    """Every finite bf16 value, beside a largest one of each exponent: ties, tiny rows, the largest numbers."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v.float())]
    v = torch.cat((v, v[:(-v.numel()) % 256])).view(-1, 256)
    q = q4.quantize(v.cuda(), "int8_row")
    c, s = ob.int8_rows(v.float().numpy())
    assert np.array_equal(q.codes.cpu().numpy(), c)
    assert np.array_equal(q.scales.cpu().numpy(), s)


def test_quantize_rows_without_numbers():
    """All zeros; below the least scale; an infinity; a NaN: the neighbours' rows stay as they are."""
    x = torch.randn(6, 272).bfloat16()
    x[0] = 0
    x[1] = 1e-20
    x[2, 5] = float("inf")
    x[3, 270] = float("nan")
    x[4, 0] = -float("inf")
    q = q4.quantize(x.cuda(), "int8_row")
    c, s = ob.int8_rows(x.float().numpy())
    got = q.scales.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.array([False, False, True, True, True, False]))
    fine = ~np.isnan(got)
    assert np.array_equal(got[fine], s[fine]) and np.array_equal(q.codes.cpu().numpy()[fine], c[fine])
    d = q4.q4_dequant(q, torch.empty(6, 272, dtype=torch.bfloat16, device="cuda")).cpu()
    assert torch.isnan(d[2:5]).all() and not torch.isnan(d[fine]).any()


def test_quantize_strided_rows():
    x = torch.randn(9, 640).bfloat16().cuda()
    a, b = q4.quantize(x[:, 8:280], "int8_row"), q4.quantize(x[:, 8:280].contiguous(), "int8_row")
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


SHAPES = [(1, 16, 128), (1, 1, 128), (2, 17, 256), (16, 64, 384), (17, 96, 512), (33, 130, 640), (64, 256, 1024),
          (65, 257, 1152), (127, 1000, 512), (128, 128, 128), (130, 512, 2048), (205, 1016, 896), (256, 256, 4096),
          (257, 264, 1280), (300, 1, 256), (512, 768, 1024), (1, 4096, 8192), (8, 2048, 7168), (48, 7168, 2048),
          (1000, 1000, 1024),
          # every kind of block, with one workgroup per CU and with two: 16 x 32, 32 x 32, 48 x 32, 32 x 64, 64 x 64,
          # 128 x 64, 128 x 128, 256 x 256 (ragged in both directions, the shortest and odd numbers of stages)
          (9, 8000, 2176), (1, 2048, 7168), (30, 8190, 1152), (125, 2040, 3200), (45, 8100, 2176), (40, 8192, 128),
          (62, 8170, 1664), (64, 8192, 128), (121, 8150, 896), (250, 8192, 128),
          (5, 8199, 640), (3, 16400, 128), (31, 8200, 384), (20, 24000, 256), (60, 20000, 128), (60, 30000, 384),
          (250, 8100, 1152), (500, 8192, 640), (511, 8070, 2304), (1020, 8150, 1152), (2040, 8190, 128),
          (2040, 8190, 1408), (4090, 1020, 4224),
          (24, 28000, 640), (100, 9000, 2560), (511, 8180, 1024), (3620, 6700, 1280)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    rng = np.random.default_rng(M * 7919 + N * 31 + K)
    ac, asc, A = operand(rng, M, K, full=True)
    wc, wsc, W = operand(rng, N, K, full=True)
    C = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    q4.q4_gemm(A, W, C)
    check(C, ob.int8_product(ac, asc, wc, wsc))


@pytest.mark.parametrize("M", [1, 16, 40, 200])
def test_largest_sums(M):
    """All codes -128 over the longest K: the sum 2^14 K just stays below 2^31."""
    K, N = (1 << 17) - 128, 40
    ac, wc = np.full((M, K), -128, np.int8), np.full((N, K), -128, np.int8)
    one = lambda n: np.ones(n, np.float32)  # noqa: E731
    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    q4.q4_gemm(tensor(ac, one(M)), tensor(wc, one(N)), C)
    check(C, np.full((M, N), float(16384 * K)))


@pytest.mark.parametrize("M,N,K,ldc,off", [(5, 40, 256, 41, 0), (70, 132, 128, 140, 1), (300, 520, 384, 523, 3),
                                           (20, 64, 256, 72, 8)])
def test_outputs_of_any_stride(M, N, K, ldc, off):
    """Rows of C at any offset and stride: what lies between them stays as it was."""
    rng = np.random.default_rng(M)
    ac, asc, A = operand(rng, M, K)
    wc, wsc, W = operand(rng, N, K)
    buf = torch.full((M * ldc + off,), 3.0, dtype=torch.bfloat16, device="cuda")
    C = buf[off:].view(M, ldc)[:, :N]
    q4.q4_gemm(A, W, C)
    check(C, ob.int8_product(ac, asc, wc, wsc))
    assert (buf[:off] == 3.0).all() and (buf[off:].view(M, ldc)[:, N:] == 3.0).all()


def test_rows_of_scale_nan_and_zero():
    rng = np.random.default_rng(5)
    ac, asc, _ = operand(rng, 40, 256)
    wc, wsc, _ = operand(rng, 72, 256)
    asc[3], wsc[9], asc[7] = np.nan, np.nan, 0.0
    C = torch.empty(40, 72, dtype=torch.bfloat16, device="cuda")
    q4.q4_gemm(tensor(ac, asc), tensor(wc, wsc), C)
    want = torch.zeros(40, 72, dtype=torch.bool)
    want[3], want[:, 9] = True, True
    got = C.cpu()
    assert torch.equal(torch.isnan(got), want)
    assert (got[7][~want[7]] == 0).all()


def test_quantized_on_the_way():
    """Activations quantized by the library against fp64 on what the codes stand for."""
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(75, 1024, generator=g).bfloat16(), (torch.randn(520, 1024, generator=g) * 0.02).bfloat16()
    W = q4.quantize(w.cuda(), "int8_row")
    C = torch.empty(75, 520, dtype=torch.bfloat16, device="cuda")
    q4.q4_gemm(q4.quantize(x.cuda(), "int8_row"), W, C)
    check(C, ob.int8_product(*ob.int8_rows(x.float().numpy()), *ob.int8_rows(w.float().numpy())))


def test_wide_offsets():
    """A weight of more than 2^31 codes: rows behind that offset are read where they are."""
    N, K = 16416, (1 << 17) - 128
    W = q4.empty_q4("int8_row", N, K)
    W.codes.zero_()
    W.scales.fill_(1.0)
    rows = [0, 16383, 16384, N - 1]
    W.codes[rows] = torch.tensor([1, 2, 3, 4], dtype=torch.int8, device="cuda")[:, None]
    A = q4.empty_q4("int8_row", 2, K)
    A.codes.fill_(1)
    A.scales.fill_(1.0)
    C = torch.empty(2, N, dtype=torch.bfloat16, device="cuda")
    q4.q4_gemm(A, W, C)
    want = torch.zeros(N, dtype=torch.bfloat16)
    want[rows] = (torch.tensor([1.0, 2.0, 3.0, 4.0]) * K).bfloat16()
    assert torch.equal(C.cpu(), want.expand(2, N))


def test_no_rows():
    A, W = q4.empty_q4("int8_row", 0, 256), q4.quantize(torch.randn(8, 256).bfloat16().cuda(), "int8_row")
    C = torch.empty(0, 8, dtype=torch.bfloat16, device="cuda")
    assert q4.q4_gemm(A, W, C) is C
    q4.q4_gemm(q4.quantize(torch.randn(4, 256).bfloat16().cuda(), "int8_row"), q4.empty_q4("int8_row", 0, 256),
               torch.empty(4, 0, dtype=torch.bfloat16, device="cuda"))


def test_graph():
    """Quantize and product captured together, replayed with new inputs between eager work."""
    g = torch.Generator().manual_seed(4)
    W = q4.quantize(torch.randn(264, 512, generator=g).bfloat16().cuda(), "int8_row")
    x = torch.randn(19, 512, generator=g).bfloat16().cuda()
    A, C = q4.empty_q4("int8_row", 19, 512), torch.empty(19, 264, dtype=torch.bfloat16, device="cuda")
    q4.q4_gemm(q4.q4_quantize(x, A), W, C)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.q4_gemm(q4.q4_quantize(x, A), W, C)
    for i in range(4):
        x.copy_(torch.randn(19, 512, generator=g).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(C)
        q4.q4_gemm(q4.quantize(x, "int8_row"), W, want)
        assert torch.equal(C, want)
