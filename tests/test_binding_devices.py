"""Every call of the binding runs on its tensors' device and refuses tensors of
several devices.  Without a GPU: tensors that say which device they are on, a
library that only records the stream, and the switch to a device replaced by a
record of it.
"""
import pytest
import torch

import w4_gemm_amd as q4
from w4_gemm_amd import grad

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
STREAM = 77


class OnGpu(torch.Tensor):
    """A tensor of the host that says that it is on a GPU."""
    where = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.where


def put(t, where):
    if isinstance(t, q4.Q4Tensor):
        gs = None if t.global_scale is None else put(t.global_scale, where)
        return q4.Q4Tensor(t.fmt, t.rows, t.cols, put(t.codes, where), put(t.scales, where), gs, t.layout)
    if isinstance(t, q4.Routing):
        return q4.Routing(*(put(getattr(t, n), where) for n in ("ids", "weights", "offsets", "gather", "inv")))
    if not isinstance(t, torch.Tensor):
        return t
    t = t.as_subclass(OnGpu)
    t.where = where
    return t


class Library:
    """Records (call, stream); sizes are the real library's."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name == "q4_sizes":
            return self.real.q4_sizes

        def call(*a):
            self.calls.append((name, a[-1]))
            return 0
        return call


@pytest.fixture
def machine(monkeypatch):
    """(calls, devices that were switched to); device 0 is the current one."""
    L, entered = Library(q4.lib()), []

    class There:
        def __init__(self, device, stream):
            entered.append(device)

        def __enter__(self):
            return "cpu", STREAM      # (what a call allocates then is the host's)

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(q4, "_LIB", L)
    monkeypatch.setattr(grad, "_There", There)
    monkeypatch.setattr(grad, "_current_device", lambda: 0)
    return L.calls, entered


def w(fmt="mxfp4", rows=64, cols=512, layout=q4.LAYOUT_ROWS):
    return q4.empty_q4(fmt, rows, cols, device="cpu", layout=layout)


def routing():
    return q4.Routing(torch.zeros(4, 2, dtype=I32), torch.zeros(4, 2), torch.zeros(5, dtype=I32),
                      torch.zeros(8, dtype=I32), torch.zeros(4, 2, dtype=I32))


def b(*shape):
    return torch.zeros(*shape, dtype=BF16)


OFF, GA = torch.zeros(5, dtype=I32), torch.zeros(8, dtype=I32)
CALLS = {
    "q4_quantize": lambda: (b(64, 512), w("fp8_row")),
    "quantize": lambda: (b(64, 512), "int8_row"),
    "q4_dequant": lambda: (w(), b(64, 512)),
    "q4_relayout": lambda: (w(), w(layout=q4.LAYOUT_TILED)),
    "relayout": lambda: (w(),),
    "q4_gemv": lambda: (w(), b(4, 512), b(4, 64)),
    "q4_gemm": lambda: (b(4, 512), w(), b(4, 64)),
    "q4_gemm_quantized": lambda: (b(4, 512), w(layout=q4.LAYOUT_TILED), w(rows=4, cols=64)),
    "q4_grouped_gemm": lambda: (b(4, 512), GA, OFF, w(rows=4 * 16), 16, b(8, 16)),
    "q4_grouped_gemm_swiglu": lambda: (b(4, 512), GA, OFF, w(rows=4 * 32), 16, b(8, 16)),
    "q4_moe_route": lambda: (torch.zeros(4, 8), 2),
    "q4_swiglu": lambda: (b(4, 64), 32),
    "q4_moe_combine": lambda: (b(8, 32), routing()),
    "q4_read_probe": lambda: (b(1024), torch.zeros(1, dtype=I32)),
    "q4_mfma_probe": lambda: ("bf16", 1, torch.zeros(1, dtype=I32)),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_tensors_device(machine, name):
    calls, entered = machine
    getattr(q4, name)(*(put(a, 1) for a in CALLS[name]()))
    assert entered == [1] and len(calls) == 1 and calls[0][1] == STREAM


@pytest.mark.parametrize("name", [n for n in CALLS if n not in ("quantize", "relayout", "q4_moe_route", "q4_swiglu", "q4_mfma_probe")])
def test_tensors_of_several_devices(machine, name):
    args = CALLS[name]()
    tensors = [i for i, a in enumerate(args) if isinstance(a, (torch.Tensor, q4.Q4Tensor, q4.Routing))]
    for odd in tensors[1:]:
        with pytest.raises(ValueError, match="like the other tensors"):
            getattr(q4, name)(*(put(a, 1 if i == odd else 0) for i, a in enumerate(args)))
    assert machine[0] == []


def test_a_stream_of_another_device(machine, monkeypatch):
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 5
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    for name, make in CALLS.items():
        with pytest.raises(ValueError, match="stream must be of cuda:0"):
            getattr(q4, name)(*(put(a, 0) for a in make()), stream=Stream())
    assert machine == ([], [])
