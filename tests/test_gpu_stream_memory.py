"""What a call allocates belongs to the stream that the call runs on: memory taken
from the current stream's pool could still be in use there, and would go back to it
while the named stream works on it.
"""
import pytest
import torch

import w4_gemm_amd as q4

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def owner(t: torch.Tensor) -> int:
    """Handle of the stream whose pool a tensor's memory is from."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not torch's memory")


@pytest.fixture(params=["object", "handle"])
def stream(request):
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    yield s, (s if request.param == "object" else s.cuda_stream)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt,layout", [("int4", 0), ("mxfp4", 1), ("nvfp4", 0), ("fp8_row", 1), ("int8_row", 0), ("mxfp8", 0)])
def test_quantize(stream, fmt, layout):
    s, named = stream
    src = torch.randn(300, 1024, device="cuda").to(BF16)
    want = q4.quantize(src, fmt, layout=layout)
    torch.cuda.synchronize()
    got = q4.quantize(src, fmt, stream=named, layout=layout)
    torch.cuda.synchronize()
    assert owner(want.codes) == torch.cuda.current_stream().cuda_stream
    for t in (got.codes, got.scales, got.global_scale):
        assert t is None or owner(t) == s.cuda_stream
    n = want.rows if layout == 0 else want.codes.numel()   # (a tiled tensor's padding rows are written too)
    assert torch.equal(got.codes[:n].view(torch.uint8), want.codes[:n].view(torch.uint8))
    assert torch.equal(got.scales.view(torch.uint8), want.scales.view(torch.uint8))


def test_relayout(stream):
    s, named = stream
    q = q4.quantize(torch.randn(48, 1024, device="cuda").to(BF16), "int4")
    torch.cuda.synchronize()
    t = q4.relayout(q, q4.LAYOUT_TILED, stream=named)
    back = q4.relayout(t, q4.LAYOUT_ROWS, stream=named)
    torch.cuda.synchronize()
    for x in (t, back):
        assert owner(x.codes) == owner(x.scales) == s.cuda_stream
    assert torch.equal(back.codes, q.codes) and torch.equal(back.scales, q.scales)


@pytest.mark.parametrize("fused", [False, True])
def test_moe_layer(stream, fused, monkeypatch):
    """The layer's results, and what it holds in between, which it gives back on return."""
    s, named = stream
    E, K, inter, T, k = 4, 512, 512, 40, 2
    g = torch.Generator().manual_seed(1)
    x, logits = torch.randn(T, K, generator=g).to(BF16).cuda(), torch.randn(T, E, generator=g).cuda()
    gu = (torch.randn(E * 2 * inter, K, generator=g) * 0.05).to(BF16).cuda()
    W_gu = q4.quantize(q4.interleave_gate_up(gu, E, inter) if fused else gu, "mxfp4", layout=q4.LAYOUT_TILED)
    W_down = q4.quantize((torch.randn(E * K, inter, generator=g) * 0.05).to(BF16).cuda(), "mxfp4", layout=q4.LAYOUT_TILED)
    want, _ = q4.moe_layer(x, logits, k, W_gu, W_down, inter, fused=fused)
    torch.cuda.synchronize()
    seen = []
    plain, fused_call = q4.q4_grouped_gemm, q4.q4_grouped_gemm_swiglu
    monkeypatch.setattr(q4, "q4_grouped_gemm", lambda *a, **kw: seen.append(owner(a[5])) or plain(*a, **kw))
    monkeypatch.setattr(q4, "q4_grouped_gemm_swiglu", lambda *a, **kw: seen.append(owner(a[5])) or fused_call(*a, **kw))
    out, r = q4.moe_layer(x, logits, k, W_gu, W_down, inter, stream=named, fused=fused)
    torch.cuda.synchronize()
    assert seen == [s.cuda_stream] * 2
    for t in (out, r.ids, r.weights, r.offsets, r.gather, r.inv):
        assert owner(t) == s.cuda_stream
    assert torch.equal(out, want)


def test_calls_that_make_their_output(stream):
    s, named = stream
    gu = torch.randn(64, 512, device="cuda").to(BF16)
    logits = torch.randn(16, 8, device="cuda")
    torch.cuda.synchronize()
    h = q4.q4_swiglu(gu, 256, stream=named)
    r = q4.q4_moe_route(logits, 2, stream=named)
    y = q4.q4_moe_combine(gu[:32], r, stream=named)
    torch.cuda.synchronize()
    for t in (h, r.ids, r.gather, y):
        assert owner(t) == s.cuda_stream
