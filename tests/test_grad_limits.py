"""The largest sizes of the backward calls, on the host: a launch has fewer
than 2^32 threads, so what would need more is refused before it."""
import ctypes

import pytest

import w4_gemm_amd as q4

SHAPE = -2
A16 = 0x7F0000000000        # never dereferenced: every call below ends before a launch


@pytest.mark.parametrize("T", ((1 << 26) - 3, (1 << 26) - 1, 1 << 26))
def test_tokens_of_the_gates(T):
    """Workgroups of 4 tokens and 256 threads: 2^24 of them are 2^32 threads."""
    L = q4.lib()
    assert (T + 3) // 4 * 256 >= 1 << 32 > ((1 << 26) - 4 + 3) // 4 * 256
    assert L.q4_moe_topk(A16, 8, T, 8, 2, A16, A16, None) == SHAPE
    assert L.q4_moe_topk_backward(A16, 8, T, 8, 2, A16, A16, A16, 8, None) == SHAPE


def test_tokens_times_columns():
    """A workgroup per token, or of 128 threads per token and 1024 columns."""
    L = q4.lib()
    for T, K in ((1 << 23, 8), (1 << 22, 8 * 1024), ((1 << 25) // 7, 7 * 1024)):
        fits = T < 1 << 23 and T * ((K + 1023) // 1024) < 1 << 25
        if not fits:
            assert L.q4_moe_permute(A16, K, A16, T, 2, K, 8, A16, K, None) == SHAPE
            assert L.q4_moe_combine_backward(A16, K, A16, K, A16, A16, T, 2, K, 8, A16, K, A16, None) == SHAPE
        else:
            assert T * ((K + 1023) // 1024) * 128 < 1 << 32 and T * 512 < 1 << 32


def test_blocks_of_the_products():
    L = q4.lib()
    d = q4._Q4TensorC(q4.MXINT8, 0, 64, 256, A16, A16, None)
    assert L.q4_grouped_gemm_wgrad(A16, 1 << 21, None, 0, ctypes.byref(d), 64, A16, A16, 129, 8, 1 << 21, 256, A16, 1, 256,
                                   0, A16, 1 << 40, None) == SHAPE
