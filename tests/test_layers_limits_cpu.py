"""Sizes of the layer operators (include/dobb_layers.h) that a launch, of fewer than 2^32 threads, cannot hold are refused
on the host like any other, and not by the launch.  Every call below is such a size: nothing is enqueued.
"""
import ctypes

import pytest

from block_diagonal_eigenbasis_amd import _layers

SHAPE = -2
CODES, SCALES, CODES2, SCALES2, OUT = 1 << 40, 1 << 42, 1 << 43, 1 << 44, 1 << 45


def operand(rows, k, codes=CODES, scales=SCALES):
    return _layers._CFp8Operand(codes, scales, rows, k, 0)


@pytest.mark.parametrize("rows,k,transpose", [(1 << 17, 1 << 19, 0), (32, 1 << 31, 0), (1 << 24, 1 << 12, 0), ((1 << 24) - 31, 1 << 12, 0),
                                              (1 << 17, 1 << 20, 1), (128, 1 << 30, 1), (1 << 24, 1 << 13, 1)])
def test_read_back(rows, k, transpose):
    assert _layers._lib().dobb_fp8_dequantize(ctypes.byref(operand(rows, k)), transpose, OUT, 1, rows if transpose else k, None) == SHAPE


@pytest.mark.parametrize("N,n", [(1 << 19, 1 << 19), (1 << 24, 1 << 14), (1 << 31, 128), (1 << 14, 1 << 24)])
def test_quantize(N, n):
    L = _layers._lib()
    cols = ctypes.byref(operand(n, N))
    assert L.dobb_fp8_quantize(N, n, OUT, 1, n, 0, None, cols, None) == SHAPE
    if N <= 1 << 24:
        rows = ctypes.byref(operand(N, n, CODES2, SCALES2))
        assert L.dobb_fp8_quantize(N, n, OUT, 1, n, 0, rows, None, None) == SHAPE
        assert L.dobb_layer_norm_fp8(N, n, OUT, 1, n, None, None, 0, 1e-5, 1 << 30, 1 << 31, None, cols, None) == SHAPE
