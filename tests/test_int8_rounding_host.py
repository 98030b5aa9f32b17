"""The arithmetic behind the int8 codes, on the host: how near 127 x / amax comes to a half between two codes, and the kernel's
sequence (fp32 quotient and product, 18 significant bits, the addition that rounds) against whole numbers."""
import numpy as np

SIG = np.arange(128, 256, dtype=np.int64)                                 # 8-bit significands


def _pairs():
    """(x, amax) as whole numbers, x <= amax, x up to 11 binades below."""
    for e in range(12):
        A, X = np.meshgrid(SIG << e, SIG, indexing="ij")
        ok = X <= A
        yield X[ok], A[ok]


def test_distance_from_a_half():
    nearest = 1.0
    for X, A in _pairs():
        # 127 X / A - (2c + 1) / 2 = (254 X - (2c + 1) A) / 2A, for the two halves around the quotient
        c = 127 * X // A
        for half in (2 * c - 1, 2 * c + 1, 2 * c + 3):
            off = np.abs(254 * X - half * A)
            assert (off[off > 0] * 255 * 254 >= 254 * X[off > 0]).all()   # off / 2A >= (127 X / A) / (254 * 255)
            nearest = min(nearest, (off[off > 0] / (254.0 * X[off > 0])).min())
    assert 2.0 ** -16 < nearest < 2.0 ** -15


def test_codes():
    f = np.float32
    for X, A in _pairs():
        t = X.astype(f) * (f(127.0) / A.astype(f))
        u = ((t.view(np.uint32) + np.uint32(0x20)) & ~np.uint32(0x3F)).view(f)
        code = (u + f(12582912.0)).view(np.uint32) & 0xFF
        c, rest = 127 * X // A, 127 * X % A                               # nearest whole number, ties to even
        want = c + ((2 * rest > A) | ((2 * rest == A) & (c % 2 == 1)))
        assert np.array_equal(code.astype(np.int64), want)
