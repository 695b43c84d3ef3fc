"""The 4-bit store's fp32 quotient, restated in integers: x times the correctly
rounded reciprocal of a step, corrected once by the exact remainder (Markstein's
method), is the correctly rounded x / step for steps of four significant bits
(and so for 7, of which it also divides)."""
from fractions import Fraction

import numpy as np
import pytest


def to24(v):
    """v (int64 > 0) rounded to nearest even at 24 significant bits: (mantissa, shift)."""
    s = np.maximum(np.floor(np.log2(v.astype(np.longdouble))).astype(np.int64) + 1 - 24, 0)
    q = v >> s
    rest, half = v - (q << s), np.where(s > 0, np.int64(1) << np.maximum(s - 1, 0), 1)
    return q + ((rest > half) | ((rest == half) & (q & 1 == 1))), s


@pytest.mark.parametrize("m", range(8, 16))
def test_corrected_quotient_is_correctly_rounded(m):
    x = np.concatenate([np.arange(1 << 23, 1 << 24, 13), np.arange((1 << 24) - 4096, 1 << 24),
                        np.arange(1 << 23, (1 << 23) + 4096)]).astype(np.int64)
    inv, e = Fraction(1, m), 0
    while inv < 1 << 23:
        inv, e = inv * 2, e + 1
    inv = round(inv)                                # 1 / m = inv 2^-e, to nearest even
    t, s = to24(x * inv)                            # t 2^(s - e) = x * (1 / m), rounded
    r = (x << (e - s)) - m * t                      # the remainder, exact, in units of 2^(s - e)
    q, s2 = to24((t << e) + r * inv)                # fma(r, 1 / m, t), rounded once
    whole = (x << 30) // m                          # x / m with the rest as a sticky bit
    want, s3 = to24((whole << 1) | ((whole * m) != (x << 30)))
    assert np.array_equal(np.ldexp(q.astype(float), s + s2 - 2 * e), np.ldexp(want.astype(float), s3 - 31))
