"""Rows whose squares fp32 does not hold: the norm and its gradient stay what the
formulas say, with eps = 0 or an eps as small as they are.

Without eps, y does not change when a row is scaled by a power of two, dx changes
by its reciprocal and dweight not at all; every step of the kernels commutes with
such a scale (sums, one division, one root), so results are equal bit for bit.
Elsewhere the bounds are those of rows of ordinary size: 2^-18 of a value for the
fp32 arithmetic, and 2^-8 where it is rounded to bf16.
"""
import numpy as np
import pytest
import torch

import w4_gemm_amd as q4
from oracle import block as ob

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
FP32 = 2.0 ** -18
COLS = [16, 128, 512, 2048, 2064, 8192, 16384, 32768]


def n64(t):
    return t.detach().cpu().double().numpy()


def near(got, ref, rel, floor=0.0, what=""):
    g = n64(got)
    bad = np.argwhere(~(np.abs(g - ref) <= rel * np.abs(ref) + floor))
    assert bad.size == 0, (what, len(bad), [(tuple(i), g[tuple(i)], ref[tuple(i)]) for i in bad[:3]])


def both(x, w, eps, fmt="int8_row", res=None):
    rows, cols = x.shape
    q, y = q4.empty_q4(fmt, rows, cols), torch.empty(rows, cols, dtype=BF16, device="cuda")
    q4.q4_rmsnorm(x, w, eps, residual=res, y=y, y_q=q)
    return y, q


def values(rows, cols, seed):
    """Normal values without those below 2^-8, so that 2^-100 of them are normal numbers too."""
    g = torch.Generator().manual_seed(seed * 7919 + cols)
    v = torch.randn(rows, cols, generator=g)
    return torch.where(v.abs() < 2.0 ** -8, torch.ones(()), v).to(BF16)


@pytest.mark.parametrize("wt", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_scaled_rows(cols, wt):
    rows = 6
    x, res = values(rows, cols, 1).cuda(), values(rows, cols, 2).cuda()
    w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).to(wt).cuda()
    want = {f: both(x, w, 0.0, f) for f in ("int8_row", "fp8_row")}
    dy = (values(rows, cols, 4) * 2.0 ** -20).cuda()
    dx, dw = q4.q4_rmsnorm_backward(dy, x, w, 0.0)
    for k in (20, 29, 30, 31, 49, 50, 62, 70, 100):
        small = x * 2.0 ** -k
        for f, (y, q) in want.items():
            y2, q2 = both(small, w, 0.0, f)
            assert torch.equal(y2, y) and torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales), (k, f)
        dx2, dw2 = q4.q4_rmsnorm_backward(dy, small, w, 0.0)
        assert torch.equal(dw2, dw), k
        assert torch.equal(dx2.double(), dx.double() * 2.0 ** k), k
        # the residual's sum, in place, in front
        h = (small.float() + (res * 2.0 ** -k).float()).to(BF16)
        at = (res * 2.0 ** -k).contiguous()
        got, y2, _ = q4.q4_rmsnorm(small, w, 0.0, residual=at, h=at)
        assert torch.equal(at, h) and torch.equal(y2, q4.q4_rmsnorm(h, w, 0.0)[1])
        near(y2, ob.rmsnorm(n64(h), n64(w), 0.0), 2.0 ** -8 + FP32)


@pytest.mark.parametrize("cols", COLS)
def test_against_the_definition(cols):
    """Subnormal values, a single one in a row, rows beside ordinary ones and an eps of the squares' size."""
    x = values(8, cols, 5).double()
    x[0] *= 1e-25
    x[1] *= 1e-38                              # mostly below the least normal number
    x[2] = 0
    x[2, cols // 2] = 2.0 ** -133              # the least there is
    x[3] *= 1e-12
    x[4] *= 1e-19
    x[5, 1:] *= 1e-30
    x[6] *= 2.0 ** -30
    x = x.to(BF16)
    w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(6)))
    g = torch.Generator().manual_seed(cols)
    dy = (torch.randn(8, cols, generator=g) * 1e-6).to(BF16)
    dh = (torch.randn(8, cols, generator=g) * 1e-6).to(BF16)
    for eps in (0.0, 2.0 ** -149, 1e-42, 1e-30, 1e-18, 1e-6):
        # the call takes eps in fp32, where 1e-42 is 714 * 2^-149 = 1.00053e-42: that is the formula's eps
        eps32 = float(np.float32(eps))
        ref = ob.rmsnorm(n64(x), n64(w), eps32)
        for fmt, top in (("int8_row", 127.0), ("fp8_row", 448.0)):
            y, q = both(x.cuda(), w.cuda(), eps, fmt)
            near(y, ref, 2.0 ** -8 + FP32, 2.0 ** -134, (eps, "y"))
            s = np.maximum(np.abs(ref).max(1), 1e-12) / top
            near(q.scales, s, FP32, what=(eps, "scale"))
            t = ref / s[:, None]
            if fmt == "int8_row":
                assert (np.abs(q.codes.cpu().double().numpy() - t) <= 0.5 + FP32 * np.abs(t)).all()
            else:
                v = q.codes.cpu().view(torch.float8_e4m3fn).double().numpy()
                assert (np.abs(v - t) <= np.maximum(2.0 ** -4 * np.abs(t), 2.0 ** -10) + FP32 * np.abs(t)).all()
        keep = [r for r in range(8) if not (r in (1, 2) and eps < 1e-30)]   # (there dx passes bf16's range)
        for add in (None, dh):
            dx, dw = q4.q4_rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), eps, dh=None if add is None else add.cuda())
            d, v, wf = n64(dy), n64(x), n64(w)
            rx, rw = ob.rmsnorm_backward(d, v, wf, eps32)
            r = 1 / np.sqrt((v * v).mean(1, keepdims=True) + eps32)
            gw, n = np.abs(d * wf), np.abs(v * r)
            size = r * (gw + n * (gw * n).mean(1, keepdims=True))
            if add is not None:
                rx, size = rx + n64(add), size + np.abs(n64(add))
            near(dx[keep], rx[keep], 2.0 ** -8, 2.0 ** -16 * size[keep], (eps, "dx"))
            near(dw, rw, 0.0, 2.0 ** -17 * np.abs(d * v * r).sum(0), (eps, "dw"))


def test_the_least_number_in_a_row_alone():
    """One value of 2^-133 in a row of zeros: n there is sqrt(cols), and dx of a gradient small enough for it."""
    cols = 1024
    x = torch.zeros(3, cols, dtype=BF16)
    x[1, 7] = 2.0 ** -133
    x[0], x[2] = 1.0, 2.0
    w = torch.ones(cols)
    y = q4.q4_rmsnorm(x.cuda(), w.cuda(), 0.0)[1].cpu()
    assert y[1, 7] == 32.0 and (y[1, :7] == 0).all() and (y[1, 8:] == 0).all()
    dy = torch.zeros(3, cols, dtype=BF16)
    dy[1, 3] = 2.0 ** -40                        # across the row's only value: dx = r dy, r = 32 * 2^133
    dx, dw = q4.q4_rmsnorm_backward(dy.cuda(), x.cuda(), w.cuda(), 0.0)
    assert dx[1, 3].item() == 2.0 ** 98 and torch.isfinite(dx).all() and (dw == 0).all()


def test_zeros_without_eps_stay_without_numbers():
    x = torch.zeros(4, 256, dtype=BF16)
    x[1], x[3] = 1.0, 1e-30
    w = torch.ones(256).cuda()
    for fmt in ("int8_row", "fp8_row"):
        y, q = both(x.cuda(), w, 0.0, fmt)
        assert torch.isnan(y[[0, 2]]).all() and torch.isnan(q.scales[[0, 2]]).all()
        assert (y[[1, 3]] == 1).all() and torch.isfinite(q.scales[[1, 3]]).all()
    dx, _ = q4.q4_rmsnorm_backward(torch.ones_like(x).cuda(), x.cuda(), w, 0.0)
    assert torch.isnan(dx[[0, 2]]).all() and torch.isfinite(dx[1]).all()


def test_among_more_rows_than_the_caches_hold():
    """Small rows where rows are read and h is written past the caches: a small row's sums read h again."""
    rows, cols = 6200, 8192
    g = torch.Generator(device="cuda").manual_seed(9)
    x, res = (torch.randn(rows, cols, device="cuda", generator=g).to(BF16) for _ in range(2))
    x[1::3] *= 1e-25
    res[1::3] *= 1e-25
    w = (1 + 0.2 * torch.randn(cols, device="cuda", generator=g)).to(BF16)
    pick = [0, 1, 2, 4, 3000, 3001, 6196, 6199]
    assert sum(r % 3 == 1 for r in pick) == 5
    for fmt in ("int8_row", "fp8_row"):
        y, q = both(x, w, 0.0, fmt, res)
        h = q4.q4_rmsnorm(x, w, 0.0, residual=res)[0]
        ys, qs = both(x[pick], w, 0.0, fmt, res[pick])
        assert torch.equal(h, (x.float() + res.float()).to(BF16))
        assert torch.equal(y[pick], ys) and torch.equal(q.codes[pick], qs.codes) and torch.equal(q.scales[pick], qs.scales)
        near(ys, ob.rmsnorm(n64(h[pick]), n64(w), 0.0), 2.0 ** -8 + FP32)
        assert torch.isfinite(y).all() and torch.isfinite(q.scales).all()
    dy = torch.randn(rows, cols, device="cuda", generator=g).to(BF16) * 2.0 ** -20
    dx, dw = q4.q4_rmsnorm_backward(dy, h, w, 0.0)
    assert torch.equal(dx[pick], q4.q4_rmsnorm_backward(dy[pick], h[pick], w, 0.0)[0])
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
