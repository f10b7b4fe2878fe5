"""A norm inside a gradient or an output of the clipping is refused: workgroups read
one while others write the other.
"""
import ctypes

import pytest

import w4_gemm_amd as q4

OK, ALIGN = 0, -3
B = 0x7F0000000000
G, H, N = B + 4096, B + (1 << 20), B + (1 << 21)


def clip(spans, out=None, norm_in=None, norm_out=None):
    m = len(spans)
    p = (ctypes.c_void_p * m)(*[a for a, _ in spans])
    c = (ctypes.c_int64 * m)(*[x for _, x in spans])
    d = (ctypes.c_int32 * m)(*[1] * m)
    o = None if out is None else (ctypes.c_void_p * m)(*out)
    return q4.lib().q4_grad_clip(m, p, c, d, o, norm_in, 1.0, norm_out, B, 1 << 24, None)


@pytest.mark.parametrize("at", [G, G + 4, G + 396])
def test_norm_in_a_gradient(at):
    assert clip([(G, 100)], norm_in=at) == ALIGN                    # in place: it is scaled while it is read
    assert clip([(G, 100)], norm_out=at) == ALIGN
    assert clip([(G, 100)], out=[H], norm_out=at) == ALIGN          # written while the gradient is read
    assert clip([(G, 100), (H, 10)], out=[G, N], norm_in=at) == ALIGN


@pytest.mark.parametrize("at", [H, H + 4, H + 396])
def test_norm_in_an_output(at):
    assert clip([(G, 100)], out=[H], norm_in=at) == ALIGN
    assert clip([(G, 100)], out=[H], norm_out=at) == ALIGN
