"""Codes of 8 bits by oracle/rows.py where products have up to 48 bits: float32
rows with float32 weights, against rational arithmetic (CPU)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import rows as orows


def rational_codes(v):
    """127 v / max|v| to the nearest whole number, ties to the even one, of the
    Fractions in v (round of a Fraction goes to the even one)."""
    top = max(abs(x) for x in v)
    return [round(127 * x / top) if top else 0 for x in v]


def halves(rows, H, seed):
    """(h [rows, H], w [H]) float32 with 24 random bits each, in pairs of equal
    weights: in the pair that holds a row's maximum the other element is half of
    it, or (2 k + 1) / 254 of it where the maximum's h is a multiple of 127."""
    rng = np.random.default_rng(seed)
    w = np.repeat(1.0 + rng.random(H // 2), 2).astype(np.float32)
    h = rng.uniform(-0.25, 0.25, size=(rows, H)).astype(np.float32)
    for r in range(rows):
        c = 2 * int(rng.integers(0, H // 2))
        if r % 2:
            j = int(rng.integers(1 << 15, 1 << 16))
            h[r, c], h[r, c + 1] = 127 * j * 2.0 ** -21, (2 * (r % 127) + 1) * j * 2.0 ** -22
        else:
            h[r, c] = 4.0 + 4.0 * rng.random()
            h[r, c + 1] = -h[r, c] / 2
    return h, w


def test_products_of_48_bits():
    h, w = halves(64, 40, 1)
    ties = 0
    q, _ = orows.quantize(h.astype(np.float64) * w.astype(np.float64))
    for r in range(len(h)):
        v = [Fraction(float(a)) * Fraction(float(b)) for a, b in zip(h[r], w)]
        top = max(abs(x) for x in v)
        ties += sum((254 * x / top).denominator == 1 and (254 * x / top) % 2 == 1 for x in v)
        assert q[r].tolist() == rational_codes(v)
    assert ties >= 60


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_quotient_just_above_a_half(sign):
    # 254 a - 253 top = 1
    v = np.array([[sign * 12523703.0 * 12164073.0, 10823765.0 * 14130145.0, 0.0]])
    assert orows.quantize(v)[0].tolist() == [[127 * int(sign), 127, 0]]
