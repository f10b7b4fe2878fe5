"""Q4_INT8_ROW on the host: sizes, and what its calls refuse before any launch."""
import ctypes

import pytest
import torch

import w4_gemm_amd as q4

OK, NULL, SHAPE, ALIGN, FMT = 0, -1, -2, -3, -4
A16 = 0x7F0000000000


def desc(rows=64, cols=512, fmt=q4.INT8_ROW, codes=A16, scales=A16, gs=None, layout=0):
    return q4._Q4TensorC(fmt, layout, rows, cols, codes, scales, gs)


def gemm(M, a, w, C=A16, ldc=4096, A=None):
    return q4.lib().q4_gemm(M, A, 512, ctypes.byref(a) if a else None, ctypes.byref(w), C, ldc, None)


def test_sizes():
    assert q4.q4_sizes("int8_row", 3, 1024) == (3 * 1024, 12)
    assert q4.q4_sizes("int8_row", 0, 16) == (0, 0)
    for rows, cols, layout in ((3, 1000, 0), (3, 1024, 1), (-1, 16, 0)):
        with pytest.raises(q4.Q4Error):
            q4.q4_sizes("int8_row", rows, cols, layout)
    t = q4.empty_q4("int8_row", 3, 32, device="cpu")
    assert t.codes.dtype == torch.int8 and t.codes.shape == (3, 32) and t.scales.shape == (3,)


def test_quantize_refuses():
    L = q4.lib()
    q = lambda d, src=A16, ld=512, gs=None: L.q4_quantize(src, ld, ctypes.byref(d), gs, None)  # noqa: E731
    assert q(desc(layout=1)) == FMT
    assert q(desc(gs=A16)) == FMT
    assert q(desc(), gs=A16) == FMT
    assert q(desc(cols=24)) == SHAPE
    assert q(desc(), ld=504) == SHAPE
    assert q(desc(), ld=516) == ALIGN
    assert q(desc(), src=A16 + 2) == ALIGN
    assert q(desc(codes=A16 + 8)) == ALIGN
    assert q(desc(scales=None)) == NULL
    assert q(desc(rows=1 << 22)) == SHAPE
    assert q(desc(rows=0)) == OK and q(desc(cols=0)) == OK


def test_gemm_refuses():
    a, w = desc(), desc(rows=256)
    assert gemm(64, None, w, A=A16) == FMT                         # bf16 activations with 8-bit weights
    assert gemm(64, desc(fmt=q4.FP8_ROW), w) == FMT
    assert gemm(64, desc(fmt=q4.MXFP4), w) == FMT
    assert gemm(64, a, desc(fmt=q4.MXFP4)) == FMT
    assert gemm(64, a, desc(fmt=q4.INT4_G128)) == FMT
    assert gemm(64, a, desc(fmt=q4.FP8_ROW)) == FMT
    assert gemm(63, a, w) == SHAPE
    assert gemm(64, desc(cols=528), w) == SHAPE
    assert gemm(64, desc(cols=1040), desc(rows=256, cols=1040)) == SHAPE     # K % 128
    assert gemm(64, desc(cols=1 << 17), desc(rows=256, cols=1 << 17)) == SHAPE
    assert gemm(64, desc(cols=0), desc(rows=256, cols=0)) == SHAPE
    assert gemm(64, a, desc(rows=1 << 27), ldc=1 << 27) == SHAPE
    assert gemm(64, a, w, ldc=255) == SHAPE
    assert gemm(64, a, w, C=None) == NULL
    assert gemm(64, a, w, C=A16 + 1) == ALIGN
    assert gemm(-1, a, w) == SHAPE
    assert gemm(0, desc(rows=0), w) == OK
    assert gemm(64, a, desc(rows=0)) == OK


def test_other_calls_refuse():
    L, d = q4.lib(), desc(rows=256)
    assert L.q4_gemv(ctypes.byref(d), A16, 1, 512, A16, 256, None) == FMT
    assert L.q4_relayout(ctypes.byref(d), ctypes.byref(d), None) == FMT
    assert L.q4_grouped_gemm(A16, 512, 8, A16, A16, 1, 8, ctypes.byref(d), 256, A16, 256, None) == FMT
    assert L.q4_gemm_dgrad(8, A16, 256, ctypes.byref(d), A16, 512, None, 0, None) == FMT
    assert L.q4_gemm_wgrad(256, A16, 64, None, 0, ctypes.byref(d), 64, 512, A16, 1, 512, 0, None, 0, None) == FMT


def test_binding_checks():
    A, W = q4.empty_q4("int8_row", 4, 256, device="cpu"), q4.empty_q4("int8_row", 8, 384, device="cpu")
    C = torch.empty(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="columns"):
        q4.q4_gemm(A, W, C)
    W = q4.empty_q4("int8_row", 8, 256, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        q4.q4_gemm(A, W, C)
    with pytest.raises(ValueError, match="hold"):
        q4.q4_gemm(q4.Q4Tensor(q4.INT8_ROW, 4, 256, A.codes[:3], A.scales), W, C)


def test_plan():
    L = q4.lib()
    a, b, c = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
    ref = [ctypes.byref(v) for v in (a, b, c)]
    assert L.q4_w8a8_plan(1, 1, 128, None, *ref[1:]) == NULL
    for M, N, K in ((-1, 1, 128), (1, -1, 128), (1, 1 << 27, 128), (1, 1, 64), (1, 1, 1 << 17), (65535 * 64 + 1, 1, 128)):
        assert L.q4_w8a8_plan(M, N, K, *ref) == SHAPE
    assert q4.q4_w8a8_plan(0, 5, 128) == (0, 0, 0) == q4.q4_w8a8_plan(5, 0, 128)
    # the smallest and the largest, and a launch that stays below 2^32 threads at the limits
    assert q4.q4_w8a8_plan(1, 1, 128)[2] == 1
    assert q4.q4_w8a8_plan(4096, 8192, 8192) == (256, 256, 512)
    for M in (1, 16, 17, 33, 64, 65, 128, 129, 160, 200, 256):
        assert q4.q4_w8a8_plan(M, (1 << 27) - 1, 128)[2] < 1 << 23
    assert q4.q4_w8a8_plan(65535 * 64, 1, 128)[2] < 1 << 22


def test_the_gpu_tests_reach_every_kind():
    """Every block with up to 256 workgroups and with more is among the sizes that the GPU tests run."""
    from test_gpu_w8a8 import SHAPES
    kinds = set()
    for M, N, K in SHAPES:
        r, c, n = q4.q4_w8a8_plan(M, N, K)
        kinds.add((r, c, n <= 256))
    blocks = [(16, 32), (32, 32), (48, 32), (32, 64), (64, 64), (128, 64), (128, 128), (256, 256)]
    # (48 x 32 and 32 x 32 have one variant)
    want = {(r, c, few) for r, c in blocks for few in (True, False)} - {(48, 32, False), (32, 32, False)}
    assert kinds >= want, want - kinds
