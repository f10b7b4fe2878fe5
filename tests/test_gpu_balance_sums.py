"""The balance loss adds probabilities over many tokens in 64 bits.

With equal logits every exponential is 1 and every sum of them the number of
experts, exactly; a probability is that number's reciprocal within 2^-23, and the
loss, whose exact value is coef, is rounded once more (2^-24): 2^-22 of it bounds
both, however many tokens there are.
"""
import pytest
import torch

import w4_gemm_amd as q4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E", [((1 << 20) + 3, 64), ((1 << 20) + 3, 128), ((1 << 20) + 3, 250), (1 << 22, 256),
                                 ((1 << 18) + 1, 1000), (5000, 100), (300, 250)])
@pytest.mark.parametrize("off", [0, 3])
def test_equal_logits(T, E, off):
    """off: every off-th token left out."""
    k = 4
    logits = torch.full((T, E), -1.25, device="cuda")
    ids = (torch.arange(T * k, device="cuda") % E).int().view(T, k)
    mask = None if not off else torch.arange(T, device="cuda") % off != 0
    loss, counts, slopes = q4.q4_moe_balance(logits, ids, 0.5, mask=mask)
    here = ids if mask is None else ids[mask]
    assert torch.equal(counts.long(), torch.bincount(here.reshape(-1).long(), minlength=E))
    assert abs(loss.item() - 0.5) <= 2.0 ** -22 * 0.5


@pytest.mark.parametrize("T,E,k", [(40001, 100, 8), (50001, 200, 4), (40003, 250, 8), (33000, 256, 2), (20001, 257, 3),
                                   (10007, 1000, 8), (9001, 1024, 32)])
def test_many_tokens(T, E, k):
    """Several turns of every workgroup, at each number of lanes per token, against torch in 64 bits; a probability
    is off by 2^-16 of itself at most (its exponent's rounding, the exponential's, the sum's)."""
    g = torch.Generator(device="cuda").manual_seed(E)
    wide = torch.randn(T, E + 3, device="cuda", generator=g) * 2
    for logits in (wide[:, :E].contiguous(), wide[:, 1:E + 1]):
        ids = torch.topk(logits, k, dim=1).indices.int().contiguous()
        mask = torch.rand(T, device="cuda", generator=g) < 0.8
        for m in (None, mask):
            loss, counts, slopes = q4.q4_moe_balance(logits, ids, mask=m)
            p, here = torch.softmax(logits.double(), 1), ids
            if m is not None:
                p, here = p[m], ids[m]
            n = here.shape[0]
            c = torch.bincount(here.reshape(-1).long(), minlength=E)
            assert torch.equal(counts.long(), c)
            s = E * c.double() / (k * float(n) * n)
            assert ((slopes.double() - s).abs() <= 2.0 ** -22 * s).all()
            want = (s * p.sum(0)).sum().item()
            assert abs(loss.item() - want) <= 2.0 ** -16 * want
