"""Calls of the backward pass that the header allows and that nothing else
runs: products without summed columns, rows that no choice has, calls on two
streams at once, replayed graphs of the larger kernels."""
import numpy as np
import pytest
import torch

import w4_gemm_amd as q4
from q4_helpers import log

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(DEV, BF16)


@pytest.mark.parametrize("layout", ("rows", "tiled"))
@pytest.mark.parametrize("fmt", ("int4", "mxfp4", "nvfp4", "int4_zp"))
def test_dgrad_without_columns_is_zero(fmt, layout):
    log("dgrad, N = 0", fmt, layout)
    W = q4.empty_q4(fmt, 0, 512, device=DEV, layout=layout)
    if fmt == "nvfp4":
        W.global_scale.fill_(1.0)
    dc = torch.empty(70, 0, dtype=BF16, device=DEV)
    out = torch.full((71, 512), 7.0, dtype=BF16, device=DEV)
    q4.q4_gemm_dgrad(dc, W, dA=out)
    assert torch.all(out[:70] == 0) and torch.all(out[70] == 7.0)
    out.fill_(7.0)
    q4.q4_grouped_gemm_dgrad(dc, torch.tensor([2, 9, 9, 66], dtype=I32, device=DEV), W, 0, dA=out)
    assert torch.all(out[2:66] == 0) and torch.all(out[:2] == 7.0) and torch.all(out[66:] == 7.0)


def test_experts_without_rows():
    """No expert has a row: dA is left alone, dW is zero (or kept, accumulated)."""
    g = _gen(1)
    off = torch.zeros(5, dtype=I32, device=DEV)
    W = q4.quantize(_bf16(g, 4 * 32, 512, std=0.02), "mxfp4")
    dc, x = _bf16(g, 90, 32), _bf16(g, 90, 512)
    out = torch.full((90, 512), 7.0, dtype=BF16, device=DEV)
    q4.q4_grouped_gemm_dgrad(dc, off, W, 32, dA=out)
    assert torch.all(out == 7.0)
    for A in (x, q4.quantize(x, "mxint8")):
        assert torch.all(q4.q4_grouped_gemm_wgrad(dc, A, None, off) == 0)
        old = torch.full((128, 512), 3.0, device=DEV)
        assert torch.all(q4.q4_grouped_gemm_wgrad(dc, A, None, off, dW=old, accumulate=True) == 3.0)


def test_rows_that_no_choice_has():
    """Every choice dropped, with no expert rows at all; and no columns."""
    T, k, N = 9, 3, 64
    g = _gen(2)
    ids = torch.full((T, k), -1, dtype=I32, device=DEV)
    offsets, _, inv = q4.q4_moe_sort(ids, 5)
    assert torch.all(offsets == 0) and torch.all(inv == -1)
    dout, w = _bf16(g, T, N), torch.rand(T, k, generator=g).to(DEV)
    dy, dw = q4.q4_moe_combine_backward(dout, torch.empty(0, N, dtype=BF16, device=DEV), inv, w)
    assert dy.shape == (0, N) and torch.all(dw == 0)
    assert torch.all(q4.q4_moe_permute_backward(torch.empty(0, N, dtype=BF16, device=DEV), inv) == 0)
    assert q4.q4_moe_permute(dout, inv, torch.empty(0, N, dtype=BF16, device=DEV)).shape == (0, N)
    _, dw = q4.q4_moe_combine_backward(dout[:, :0], torch.empty(T * k, 0, dtype=BF16, device=DEV), inv, w)
    assert torch.all(dw == 0)


def _large(seed):
    """Inputs of a sort in chunks and of products in parts and in blocks of 128 and 256 rows."""
    g = _gen(seed)
    ids = torch.randint(-1, 40, (3000, 4), generator=g).to(DEV, I32)
    W = q4.quantize(_bf16(g, 264, 7680, std=0.02), "int4", layout="tiled")
    Wp = q4.quantize(_bf16(g, 4096, 512, std=0.02), "mxfp4", layout="tiled")
    x = q4.quantize(_bf16(g, 1500, 288), "mxfp8")
    return ids, W, Wp, x, _bf16(g, 2101, 264), _bf16(g, 60, 4096), _bf16(g, 1500, 264)


def _calls(a):
    ids, W, Wp, x, dc, dcp, dcw = a
    offsets, _, inv = q4.q4_moe_sort(ids, 40)
    return (offsets, inv, q4.q4_gemm_dgrad(dc, W), q4.q4_gemm_dgrad(dc[:1100], W), q4.q4_gemm_dgrad(dcp, Wp),
            q4.q4_gemm_wgrad(dcw, x))


def test_sizes_are_those():
    assert q4.q4_dgrad_plan(2101, 1, 264, 7680)[0] == 256 and q4.q4_dgrad_plan(1100, 1, 264, 7680)[0] == 128
    assert q4.q4_dgrad_plan(60, 1, 4096, 512)[1] > 1 and q4.q4_wgrad_plan(1500, 1, 264, 288)[1] > 1


def test_two_streams_at_once():
    log("two streams")
    inputs = [_large(s) for s in (3, 4)]
    want = [_calls(a) for a in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_calls(inputs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


def test_two_graphs_replayed():
    """Two graphs of the same calls on their own inputs, replayed in turn with eager work and new inputs between."""
    log("two graphs")
    inputs = [_large(s) for s in (5, 6)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _calls(inputs[0])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a in inputs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_calls(a))
        graphs.append(g)
    for r in range(4):
        for i, a in enumerate(inputs):
            fresh = _large(10 + 2 * r + i)
            for j in (0, 4, 5, 6):
                a[j].copy_(fresh[j])
        eager = [[t.clone() for t in _calls(a)] for a in inputs]
        torch.cuda.synchronize()
        for i in (r % 2, 1 - r % 2):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], eager[i])), (r, i)
