"""The 8-bit block formats at every bf16 value: the definition of
oracle/grad.py computed for all blocks at once (checked against it here), and
the GPU's codes and scales equal to it bit for bit."""
import numpy as np
import pytest
import torch

import w4_gemm_amd as q4
from oracle import grad
from q4_helpers import log, to_f32

BF16 = torch.bfloat16
FORMATS = ("mxint8", "mxfp8")


def quantize_blocks(fmt, x):
    """(codes [n, 32], scales [n, 1]) of n blocks: grad.mx8_quantize without its loops."""
    x = x.astype(np.float64)
    broken = ~np.isfinite(x).all(axis=1, keepdims=True)
    v = np.where(broken, 0.0, x)
    # the least e with amax <= top 2^e: a quotient of 1 only at equality (the amax have 8 bits), so no rounding decides it
    m, e = np.frexp(np.abs(v).max(axis=1, keepdims=True) / grad.MX8_TOP[fmt])
    e = np.where(m == 0.0, grad.MX8_LEAST, np.maximum(e - (m == 0.5), grad.MX8_LEAST))
    y = np.abs(v) * 2.0 ** -e
    # values stay below 2^128
    if fmt == "mxint8":
        c = np.minimum(np.rint(y), np.ceil(2.0 ** (128 - e)) - 1)
        codes = (np.where(x < 0, -c, c)).astype(np.int64) & 0xFF
    else:
        hi = np.clip(np.searchsorted(grad.E4M3, y), 1, 126)
        below, above = y - grad.E4M3[hi - 1], grad.E4M3[hi] - y
        c = np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)
        c = np.minimum(c, np.searchsorted(grad.E4M3, 2.0 ** (128 - e)) - 1)
        codes = c | np.where(np.signbit(x), 0x80, 0)
    codes = np.where(broken, 0 if fmt == "mxint8" else 0x7F, codes)
    return codes.astype(np.uint8), np.where(broken, 255, e + 127).astype(np.uint8)


def every_value():
    """65536 blocks: one bf16 value each, and smaller ones of either sign beside it (nothing beside what is not finite)."""
    x = torch.from_numpy(np.arange(65536, dtype=np.uint16).view(np.int16).copy()).view(BF16).reshape(-1, 1).repeat(1, 32)
    f = x[:, 1:].float()
    part = torch.linspace(-1, 1, 31)
    x[:, 1:] = torch.where(torch.isfinite(f), f, 0.0).mul(part).to(BF16)
    return x


@pytest.mark.parametrize("fmt", FORMATS)
def test_all_blocks_at_once_is_the_definition(fmt):
    x = to_f32(every_value())[::131]
    special = np.zeros((6, 32), np.float32)
    special[0, 3], special[1, 3], special[2, 3] = grad.MX8_TOP[fmt], -2 * grad.MX8_TOP[fmt], 2.0 ** -130
    special[3, 3], special[4, 3] = np.nan, -np.inf
    special[5] = float(torch.finfo(BF16).max)
    for v in (x, special, to_f32(every_value())[[0x7F7F, 0xFF7F, 0x7F00, 0x0001, 0x8000]]):
        codes, scales = grad.mx8_quantize(fmt, v)
        got = quantize_blocks(fmt, v)
        assert np.array_equal(got[1], scales) and np.array_equal(got[0], codes)


@pytest.mark.parametrize("fmt", FORMATS)
def test_errors_are_those_that_the_header_states(fmt):
    x = to_f32(every_value())
    x = x[np.isfinite(x).all(axis=1)].astype(np.float64)
    codes, scales = quantize_blocks(fmt, x)
    err = np.abs(grad.mx8_dequant(fmt, codes, scales) - x)
    s, amax = 2.0 ** (scales.astype(np.float64) - 127), np.abs(x).max(axis=1, keepdims=True)
    if fmt == "mxint8":
        top = float(torch.finfo(BF16).max)
        assert np.all(err[np.abs(x) == top] <= 0.75 * s.max())
        assert np.all((err <= s / 2) | (np.abs(x) == top))
        normal = amax > 127 * 2.0 ** -111
        assert np.all((s / 2 <= amax / 127)[normal]) and np.all((s / 2 >= amax / 254)[normal])
    else:
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FORMATS)
def test_every_bf16_value(fmt):
    log("mx8 every value", fmt)
    x = every_value()
    codes, scales = quantize_blocks(fmt, to_f32(x))
    q = q4.quantize(x.to("cuda:0"), fmt)
    assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(q.codes.cpu().numpy(), codes)
    back = q4.q4_dequant(q, torch.empty(x.shape, device="cuda:0"))
    assert np.array_equal(to_f32(back).astype(np.float64), grad.mx8_dequant(fmt, codes, scales), equal_nan=True)
