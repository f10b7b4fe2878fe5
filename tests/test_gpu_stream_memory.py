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
