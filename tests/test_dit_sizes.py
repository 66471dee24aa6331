"""include/nvfp4_dit.h: the largest lengths, that kernels round up to tiles of
128 in 32 bits.  Every call holds a misaligned pointer, whose check comes after
that of the sizes: none reaches a device."""
import ctypes
import struct

import pytest

from nvfp4_w4a4_gemm_quantize_b200 import _lib, build

SHAPE, MISALIGNED = 2, 3
A, ODD = 0x10000, 0x10002                    # fake device addresses (never dereferenced)
MOST = 2 ** 31 - 128


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("K,want", [(MOST, MISALIGNED), (MOST + 64, SHAPE), (MOST + 128, SHAPE), (2 ** 32, SHAPE)])
def test_gemv_k(L, fmt, K, want):
    assert L.nvfp4_gemv_w4a16(ODD, K, A, A, A, fmt, None, 1, 1, K, A, 0, None) == want


@pytest.mark.parametrize("N,want", [(MOST - 1, MISALIGNED), (MOST, SHAPE), (2 ** 31 - 1, SHAPE), (2 ** 32, SHAPE)])
def test_gemv_n(L, N, want):
    assert L.nvfp4_gemv_w4a16(ODD, 128, A, A, A, 0, None, 1, N, 128, A, 0, None) == want


@pytest.mark.parametrize("Lq,Lk,want", [(1, MOST, MISALIGNED), (MOST, 1, MISALIGNED), (1, MOST + 1, SHAPE), (MOST + 1, 1, SHAPE),
                                        (16, 2 ** 31 - 2, SHAPE), (2 ** 31 - 2, 16, SHAPE), (0, MOST + 1, SHAPE)])
def test_attention_lengths(L, Lq, Lk, want):
    h, odd = struct.pack("Pqqq", A, 8, 8, 8), struct.pack("Pqqq", ODD, 8, 8, 8)
    if Lq > 0:
        assert L.nvfp4_cross_attention(odd, h, h, None, 0.5, 1, 1, 1, Lq, Lk, 8, h, None, None, None) == want
    assert L.nvfp4_cross_attention_backward(odd, h, odd, h, h, A, None, 0.5, 1, 1, 1, Lq, Lk, 8, h, h, h, A,
                                            ctypes.c_size_t(2 ** 50), None, None) == want
    assert (L.nvfp4_cross_attention_backward_workspace_bytes(1, 1, 1, Lq, Lk, 8) > 0) == (want != SHAPE)
