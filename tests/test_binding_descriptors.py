"""A q4_tensor argument of the library takes a descriptor and nothing else: what
Q4Tensor.packed() makes, a reference to the structure, or None.  An address, bytes
of another length or another structure's reference never reach the library as one.
"""
import ctypes

import pytest

import w4_gemm_amd as q4

ADDRESS = 0x7F0000000000


class Other(ctypes.Structure):
    _fields_ = [("x", ctypes.c_int64)] * 1


def structure(fmt=q4.INT8_ROW, rows=4, cols=512):
    return q4._Q4TensorC(fmt, 0, rows, cols, ADDRESS, ADDRESS, None)


def gemm(a, w):
    """A call that ends at its checks (no output)."""
    return q4.lib().q4_gemm(4, None, 0, a, w, None, 512, None)


BAD = [ADDRESS, 5, ctypes.c_void_p(ADDRESS), b"", b"\0" * 47, b"\0" * 49, "text", ctypes.byref(Other()),
       ctypes.byref(ctypes.c_int64()), bytearray(48), 1.0]


@pytest.mark.parametrize("bad", BAD, ids=lambda v: type(v).__name__ + (str(len(v)) if isinstance(v, bytes) else ""))
def test_other_values_are_refused(bad):
    good = structure()
    with pytest.raises(ctypes.ArgumentError):
        gemm(ctypes.byref(good), bad)
    with pytest.raises(ctypes.ArgumentError):
        gemm(bad, ctypes.byref(good))
    with pytest.raises(ctypes.ArgumentError):
        q4.lib().q4_dequant(bad, ADDRESS, 0, 512, None)


def test_descriptors_are_taken():
    good = structure()
    packed = bytes(good)
    assert len(packed) == ctypes.sizeof(q4._Q4TensorC)
    t = q4.empty_q4("int8_row", 4, 512, device="cpu")
    assert bytes(t.c()) == t.packed()
    NULL, FMT = -1, -4
    for d in (ctypes.byref(good), ctypes.pointer(good), packed):
        assert gemm(d, d) == NULL                       # both are right; there is no output
        assert gemm(None, d) == FMT and gemm(d, None) == NULL    # (a W in 8 bits takes an A in 8 bits only)
    odd = bytes(structure(fmt=7))
    assert gemm(packed, odd) == FMT and gemm(odd, packed) == FMT     # and read as what they say
