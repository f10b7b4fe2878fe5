"""The backward calls at values where a shortcut would show: logits that are
not numbers, sigmoids below the smallest normal number."""
import numpy as np
import pytest
import torch

import w4_gemm_amd as q4
from oracle import grad
from q4_helpers import log, to_f32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.mark.parametrize("E", (5, 64, 100, 700))
def test_gates_of_logits_that_are_not_numbers(E):
    """A NaN among a token's logits (alone, or beside nothing but -inf) makes its whole gradient NaN, as the formula does;
    only a token whose logits are all -inf gets zeros."""
    log("gates, NaN", E)
    rng = np.random.default_rng(E)
    lg = rng.standard_normal((6, E)).astype(np.float32)
    lg[0] = np.nan
    lg[1], lg[1, E - 1] = -np.inf, np.nan
    lg[2, 0] = np.nan
    lg[3] = -np.inf
    lg[4, 1:] = -np.inf
    ids = np.stack([rng.permutation(E)[:3] for _ in range(6)]).astype(np.int32)
    dw = rng.standard_normal((6, 3)).astype(np.float32)
    out = q4.q4_moe_topk_backward(*(torch.from_numpy(a).to(DEV) for a in (lg, ids, dw))).cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref = grad.topk_backward(lg, ids, dw)
    assert np.array_equal(np.isnan(out), np.isnan(ref))
    assert np.isnan(out[:3]).all() and np.all(out[3] == 0) and np.isfinite(out[4:]).all()


# every bf16 g whose sigmoid exp(g) is around the smallest normal fp32 number (2^-126: g = -87.34) and still has a
# finite exp(-g) (-88.72)
G = (-80.0, -86.5, -87.0, -87.5, -88.0, -88.5)
U = (1.0, -3.0, 0.25, 2.0 ** 100, -2.0 ** 126)


@pytest.mark.parametrize("fmt", ("mxint8", "mxfp8"))
def test_swiglu_of_very_negative_gates(fmt):
    """h is q4_swiglu's to the last bf16 place (or the smallest bf16 number), and the gradients are the formula's within
    the roundings: the sigmoid (|g| + 8) 2^-22 (as denormal number of 2^-149 steps: 2^-21), one bf16 rounding."""
    log("swiglu, very negative gates", fmt)
    g, u = (a.reshape(-1, 1) for a in np.meshgrid(G, U))
    gu = torch.from_numpy(np.concatenate((np.repeat(g, 32, 1), np.repeat(u, 32, 1)), 1).astype(np.float32)).to(BF16)
    P = gu.shape[0]
    saved = q4.empty_q4(fmt, P, 64, device=DEV)
    h = to_f32(q4.q4_swiglu_save(gu.to(DEV), 32, saved)).astype(np.float64)
    plain, f = to_f32(q4.q4_swiglu(gu.to(DEV), 32)).astype(np.float64), to_f32(gu).astype(np.float64)
    bad = ~(np.abs(h - plain) <= np.maximum(2.0 ** -7 * np.abs(plain), 2.0 ** -133))
    assert np.all(plain != 0) and not bad.any(), f[bad.any(1)][:, [0, 32]].tolist()
    dh = torch.full((P, 32), 2.0, dtype=BF16)
    dg, du, rh = grad.swiglu_backward(f[:, :32], f[:, 32:], to_f32(dh))
    h2 = torch.empty(P, 32, dtype=BF16, device=DEV)
    dgu = to_f32(q4.q4_swiglu_backward(gu.to(DEV), dh.to(DEV), h=h2)).astype(np.float64)
    e = 2.0 ** -8 + (np.abs(f[:, :32]) + 8) * 2.0 ** -22 + 2.0 ** -21
    for what, got, ref in (("dg", dgu[:, :32], dg), ("du", dgu[:, 32:], du), ("h again", to_f32(h2), rh)):
        bad = ~(np.abs(got - ref) <= e * np.abs(ref) + 2.0 ** -133)
        assert not bad.any(), (what, f[bad.any(1)][:, [0, 32]].tolist())
