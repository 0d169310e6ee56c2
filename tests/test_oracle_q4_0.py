"""Pins for the oracle's q4_0 quantiser (no GPU): none of these re-runs its formula."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import q4_0


def test_codes_by_rational_numbers():
    # the nearest code by exact arithmetic, ties away from zero, the eighth step up cut off at 7
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((300, 32)) * rng.choice([1e-30, 1e-3, 1.0, 1e4], size=(300, 1))).astype(np.float32)
    x[:150] = np.round(x[:150] / np.abs(x[:150]).max(1, keepdims=True) * 16) / 16   # many ties
    x[0] = 0
    d, q = q4_0.quantize_blocks(x)
    for b, dd, qq in zip(x, d[:, 0], q):
        a = [Fraction(float(v)) for v in b]
        most = max(abs(v) for v in a)
        m = -most if -most in a else most
        for v, c in zip(a, qq):
            if m == 0:
                assert c == 0
                continue
            err = lambda k: abs(v + m * k / 8)
            best = min(err(k) for k in range(-9, 10))
            want = max((k for k in range(-9, 10) if err(k) == best), key=abs)
            assert c == min(want, 7)
        assert dd == np.float16(float(-m / 8)) and (m != 0 or not np.signbit(dd))


def test_hand_made_block():
    x = np.zeros(32, np.float32)
    x[:8] = [8, -8, 7.5, -7.5, 0.5, -0.5, 0.49, 1.5]
    d, q = q4_0.quantize_blocks(x)
    assert d[0] == 1.0     # the negative one of the two greatest: -m / 8 = 1
    assert list(q[:8]) == [7, -8, 7, -8, 1, -1, 0, 2]
    d, q = q4_0.quantize_blocks(-x[None, :] + np.eye(1, 32, 31, dtype=np.float32) * 9)
    assert d[0, 0] == -1.125 and q[0, 31] == -8
    # values 0 .. 7 of a word in the order 0 2 4 6 | 1 3 5 7 from its low bits
    p = q4_0.pack(np.array([0, 1, 2, 3, 4, 5, 6, 7], np.int8))
    assert list(p) == [0xA8, 0xEC, 0xB9, 0xFD]


def test_round_trip_and_error():
    rng = np.random.default_rng(5)
    q = rng.integers(-8, 8, (20, 64)).astype(np.int8)
    assert np.array_equal(q4_0.unpack(q4_0.pack(q)), q)
    x = rng.standard_normal((500, 96)).astype(np.float32)
    d, q = q4_0.quantize_blocks(x)
    y = q4_0.dequantize_blocks(d, q)
    step = np.abs(d.astype(np.float32)).repeat(32, -1)
    # half a step, a whole one at the cut-off code, and the scale's own rounding of 8 steps
    assert (np.abs(x - y) <= step * np.where(q == 7, 1.0, 0.5) * (1 + 1e-6) + 8 * step * 2.0 ** -11).all()


def test_refuses_what_it_does_not_define():
    with pytest.raises(ValueError):
        q4_0.quantize_blocks(np.full(32, np.nan, np.float32))
    with pytest.raises(ValueError):
        q4_0.quantize_blocks(np.zeros(33, np.float32))
