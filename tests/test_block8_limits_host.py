"""Sizes whose launch would hold 2^32 threads or more are refused as shapes (no GPU needed: nothing is enqueued)."""
import ctypes as C

from mxfp8_precision_numerics_amd import _lib

P = 0x10000


def test_norm_rows():
    f = _lib.load().rmsnorm_mx_quantize
    for cols, threads in ((64, 64), (2048, 64), (2080, 256), (8192, 256), (8224, 512), (12288, 512), (12320, 1024), (32768, 1024)):
        rows = 2 ** 32 // threads
        for r in (rows, rows - 1024 // threads + 1, 2 * rows):
            assert f(P, P, P, r, cols, C.c_float(1e-6), P, P, P, P, None, None, None, None, 0, None) == 2, (r, cols)
    # the column orientation: 65535 tiles of 128 rows
    assert f(P, P, P, 128 * 65535 + 32, 64, C.c_float(1e-6), P, P, P, P, P, P, None, None, 0, None) == 2


def test_swiglu_values():
    f = _lib.load().swiglu_mx_quantize_checkpoint
    for rows, F in ((2 ** 26, 512), (2 ** 20, 2 ** 15), (1, 2 ** 35), (2 ** 40, 32), (2 ** 26 - 15, 512)):
        assert f(P, rows, F, P, P, P, P, 0, None) == 2, (rows, F)
