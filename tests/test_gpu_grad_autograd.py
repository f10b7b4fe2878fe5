"""How the calls stand to torch's differentiation: nothing is recorded by
itself, and a torch.autograd.Function made of a call and its gradient is
differentiated with these gradients."""
import numpy as np
import pytest
import torch

import w4_gemm_amd as q4

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


class Layer(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, logits, w_gu, w_down, k, inter):
        out, ctx.kept = q4.moe_layer_save(x, logits, k, w_gu, w_down, inter, weights_grad=False)
        ctx.weights = w_gu, w_down
        return out

    @staticmethod
    def backward(ctx, dout):
        dx, dlogits, _, _ = q4.moe_layer_backward(ctx.kept, dout, *ctx.weights)
        return dx, dlogits, None, None, None, None


def test_calls_are_not_recorded_and_a_function_of_them_is():
    g = torch.Generator().manual_seed(3)
    T, E, k, K, inter = 33, 4, 2, 512, 128
    x = torch.randn(T, K, generator=g).to(DEV, BF16).requires_grad_()
    logits = torch.randn(T, E, generator=g).to(DEV).requires_grad_()
    w = [q4.quantize((torch.randn(*s, generator=g) * 0.05).to(DEV, BF16), "mxfp4") for s in ((E * 2 * inter, K), (E * K, inter))]
    plain, _ = q4.moe_layer(x, logits, k, *w, inter)
    out, kept = q4.moe_layer_save(x, logits, k, *w, inter, weights_grad=False)
    assert not plain.requires_grad and not out.requires_grad
    dout = torch.randn(T, K, generator=g).to(DEV, BF16)
    want = q4.moe_layer_backward(kept, dout, *w)
    y = Layer.apply(x, logits, *w, k, inter)
    assert torch.equal(y, out) and y.requires_grad
    (y + x).backward(dout)
    assert torch.equal(logits.grad, want[1])
    ref = want[0].float() + dout.float()                # added in bf16: one rounding, 2^-8 of the value
    assert np.all((x.grad.float() - ref).abs().cpu().numpy() <= 2.0 ** -8 * ref.abs().cpu().numpy())
