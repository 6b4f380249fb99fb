"""The Q8_0 scale top / 127 without a division, as lq_kv.cu takes it: q = top
rounded(1 / 127), then q + (top - 127 q) rounded(1 / 127) by two fused
multiply-adds. In integers, for every mantissa: the remainder is a float32
number, and the result is the quotient rounded to nearest."""
import numpy as np

BY_127 = int(np.float32(1.0 / 127.0) * 2.0**30)  # its 24-bit mantissa; the value is BY_127 / 2^30


def _round(x, shift):
    """x / 2^shift to the nearest integer, ties to even, in int64."""
    whole, rest, half = x >> shift, x & ((1 << shift) - 1), 1 << (shift - 1)
    return whole + ((rest > half) | ((rest == half) & (whole & 1 == 1)))


def test_every_mantissa():
    assert 1 << 23 <= BY_127 < 1 << 24
    for first in range(1 << 23, 1 << 24, 1 << 21):
        m = np.arange(first, first + (1 << 21), dtype=np.int64)  # top = m, an integer of 24 bits
        product = m * BY_127                                     # top / 127 2^30, about
        # q has 24 bits: quotients from 2^16 come in steps of 2^-7, from 2^17 in steps of 2^-6
        step = np.where(product >= 1 << 47, 6, 7)
        q = np.where(step == 6, _round(product, 24), _round(product, 23))
        remainder = (m << step) - 127 * q                        # exact, in steps
        assert np.abs(remainder).max() < 1 << 24
        total = (q << 30) + remainder * BY_127                   # the second fused multiply-add's sum, in steps / 2^30
        rounded = _round(total, 30)
        # the quotient itself: no tie, as 127 is odd
        wanted_step = np.where(m >= 127 << 17, 6, 7)
        wanted = (2 * (m << wanted_step) + 127) // 254
        assert np.array_equal(rounded << (7 - step), wanted << (7 - wanted_step))


def test_the_check_catches_a_quotient_without_its_correction():
    m = np.arange(1 << 23, 1 << 24, dtype=np.int64)
    q = np.where(m * BY_127 >= 1 << 47, _round(m * BY_127, 24) << 1, _round(m * BY_127, 23))
    step = np.where(m >= 127 << 17, 6, 7)
    wanted = (2 * (m << step) + 127) // 254
    assert (q != wanted << (7 - step)).any()
