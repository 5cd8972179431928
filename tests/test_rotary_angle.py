"""The rotary angle's arithmetic (whole numbers, so the same here as on the
device): position * inv_freq in turns, from the constants in the kernel's source,
against the exact product, and the error that include/extkv.h promises."""
import os
import re
import struct
from fractions import Fraction

import pytest

from packed_ref import _BITS, _INV_2PI

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV_2PI = Fraction(_INV_2PI, 1 << _BITS)


def constants():
    src = open(os.path.join(ROOT, "biased_gqa_attention_gb300", "csrc", "rotary_append.cu")).read()
    hi, lo = re.search(r"c_hi = (0x[0-9A-F]+)ull, c_lo = (0x[0-9A-F]+)ull", src).groups()
    return int(hi, 16), int(lo, 16)


def bits_of(f):
    return struct.unpack("<I", struct.pack("<f", f))[0]


def value_of(bits):
    return struct.unpack("<f", struct.pack("<I", bits))[0]


def turns(pos, f):
    """The upper 64 bits of the fraction, as cos_sin() forms it, for pos, f >= 0."""
    c_hi, c_lo = constants()
    u = bits_of(f) & 0x7FFFFFFF
    ex = u >> 23
    m = (u & 0x7FFFFF) | 0x800000 if ex else u & 0x7FFFFF
    p = (c_lo * m + ((c_hi * m) << 64)) & ((1 << 128) - 1)
    sh = (ex or 1) - 150 + 32
    F = (p << sh) & ((1 << 128) - 1) if sh >= 0 else p >> -sh
    return ((F >> 64) * pos + (((F & ((1 << 64) - 1)) * pos) >> 64)) & ((1 << 64) - 1)


def error(pos, f):
    """Turns by which the fraction is off, around the circle."""
    exact = pos * Fraction(f) * INV_2PI
    e = (Fraction(turns(pos, f), 1 << 64) - exact) % 1
    return min(e, 1 - e)


def promised(pos, f):
    return Fraction(1, 1 << 64) + Fraction(pos, 1 << 128) + pos * Fraction(f) / (1 << 96)


POSITIONS = (0, 1, 5, 4095, 10 ** 6, 2 ** 31, 2 ** 40 + 3, 2 ** 62 + 12345, 2 ** 63 - 1, 2 ** 63)
FREQS = [value_of(bits_of(x)) for x in (1.0, 1e-4, 1e-8, 1e-20, 1e-38, 3.7e4, 0.31622776, 4.2949e9)] + \
    [value_of(1), value_of(0x7FFFFF), value_of(bits_of(2.0 ** 32) - 1)]


def test_the_constant_is_one_over_two_pi():
    hi, lo = constants()
    assert (hi << 64 | lo) == (_INV_2PI << 96) >> _BITS


@pytest.mark.parametrize("f", FREQS)
def test_the_angle_errs_by_no_more_than_is_promised(f):
    for pos in POSITIONS:
        assert error(pos, f) <= promised(pos, f), (pos, f)


def test_each_part_of_the_promise_is_needed():
    """Without one of the three terms the bound does not hold."""
    small = value_of(bits_of(1e-4))
    assert error(1, small) > promised(1, small) - Fraction(1, 1 << 64)
    assert any(error(2 ** 63 - 1, f) > Fraction(1, 1 << 64) + 2 ** 63 * Fraction(f) / (1 << 96)
               for f in (value_of(bits_of(x)) for x in (1e-30, 3e-33, 7e-35, 2e-36)))
    fast = value_of(bits_of(2.0 ** 32) - 1)
    assert error(2 ** 63, fast) > Fraction(1, 1 << 64) + Fraction(2 ** 63, 1 << 128)


def test_the_header_names_the_bound():
    text = open(os.path.join(ROOT, "include", "extkv.h")).read()
    assert "2^-64 + |position| * 2^-128 + |position * inv_freq| * 2^-96 turns" in text
