"""The arithmetic that makes the 8-bit block cache's codes the same however a quotient is computed: with
scales of 8 significant bits, the kernel's roundings (product with the rounded 1 / s, then a grid that has
every middle between two codes on it) give the code of the exact quotient, for every pair of significands
and every exponent that can occur.  CPU only."""
from fractions import Fraction

import numpy as np
import pytest


def half_even(q):
    """Nearest whole number of an array of exact quotients a / b, ties to even."""
    a, b = q
    two = 2 * a
    k = two // (2 * b)                       # floor
    rest = two - 2 * b * k                   # in [0, 2b)
    return np.where(rest > b, k + 1, np.where(rest < b, k, k + (k & 1)))


def significands():
    a, b = np.meshgrid(np.arange(128, 256, dtype=np.int64), np.arange(128, 256, dtype=np.int64), indexing="ij")
    return a.ravel(), b.ravel()


def quotient(a, b, j):
    """x times the rounded 1 / s for x = a 2^j, s = b, before any rounding of the product (it is exact in 64 bits)."""
    inv = (np.float32(1.0) / b.astype(np.float32)).astype(np.float64)
    return a * 2.0 ** j * inv


@pytest.mark.parametrize("j", range(-12, 8))
def test_int8_codes(j):
    a, b = significands()
    keep = a * 2.0 ** j <= 127 * b
    a, b = a[keep], b[keep]
    y = np.rint(quotient(a, b, j) * 1024) / 1024               # 12288 + y in fp32: multiples of 2^-10
    got = np.rint(y)
    exact = half_even((a << j, b) if j >= 0 else (a, b << -j))
    assert (got == exact).all()


def e4m3(y):
    """Nearest E4M3 number, ties to even, of values that fp32 or 64 bits hold."""
    e = np.maximum(np.frexp(y)[1] - 1, -6)
    unit = np.ldexp(1.0, e - 3)
    return np.rint(y / unit) * unit


@pytest.mark.parametrize("j", range(-14, 10))
def test_e4m3_codes(j):
    a, b = significands()
    keep = a * 2.0 ** j <= 448 * b
    a, b = a[keep], b[keep]
    y = quotient(a, b, j).astype(np.float32)
    snapped = ((y.view(np.uint32) + np.uint32(0x80)) & np.uint32(0xFFFFFF00)).view(np.float32).astype(np.float64)
    got = e4m3(snapped)
    unit = np.ldexp(1.0, np.maximum(np.frexp(a * 2.0 ** j / b)[1] - 1, -6) - 3)
    k = np.log2(unit).astype(np.int64)                          # quotient / unit = a 2^(j - k) / b
    exact = np.array([float(round(Fraction(int(p)) * Fraction(2) ** int(j - x) / int(q))) for p, q, x in zip(a, b, k)])
    assert (got == exact * unit).all()


@pytest.mark.parametrize("top", [127, 448])
def test_scales_hold_every_value_and_are_the_smallest(top):
    amax = (np.arange(0x2B80, 0x7100, dtype=np.uint32) << 16).view(np.float32)  # bf16 numbers, 2^-40 to 2^99
    t = amax / np.float32(top)
    s = ((t.view(np.uint32) + np.uint32(0xFFFF)) & np.uint32(0xFFFF0000)).view(np.float32)
    below = (s.view(np.uint32) - np.uint32(0x10000)).view(np.float32)
    assert (s.astype(np.float64) * top >= amax).all() and (below.astype(np.float64) * top < amax).all()
