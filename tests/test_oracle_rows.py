"""Pins of oracle/rows.py: rational arithmetic, differences, moe_align's definition (CPU)."""
from fractions import Fraction

import numpy as np

from oracle import rows as orows


def test_codes_against_rational_arithmetic():
    rng = np.random.default_rng(1)
    # few significant bits: many quotients lie exactly between two codes
    v = rng.integers(-64, 65, size=(40, 24)) * 2.0 ** rng.integers(-3, 4, size=(40, 1))
    v[0] = 0.0
    q, top = orows.quantize(v)
    ties = 0
    for r in range(v.shape[0]):
        m = max(abs(Fraction(x)) for x in v[r])
        assert m == Fraction(top[r])
        for x, c in zip(v[r], q[r]):
            want = round(127 * Fraction(x) / m) if m else 0     # (round of a Fraction: ties to even)
            ties += bool(m) and (2 * 127 * Fraction(x) / m).denominator == 1 and (254 * Fraction(x) / m) % 2 == 1
            assert c == want
    assert ties > 0     # (the rule is met)


def test_norm_of_a_row_by_hand():
    y, q, s = orows.rms_norm([[3.0, -4.0, 0.0, 0.0]], [1.0, 2.0, 1.0, 1.0], 0.0)
    assert np.allclose(y, [[1.2, -3.2, 0.0, 0.0]])          # rms 2.5
    assert q.tolist() == [[48, -127, 0, 0]]                  # 127 * 3 / 8 = 47.6
    assert np.allclose(s, 3.2 / 127)


def test_rows_by_expert():
    ids = np.array([[2, 0], [0, 5], [2, 2]])
    offsets, inv = orows.align(ids, 4, 1)
    assert offsets.tolist() == [0, 2, 2, 5, 5, 8]
    assert inv.tolist() == [2, 0, 1, -1, 3, 4, 5, 6, 7]
    x = np.arange(6.0).reshape(3, 2)
    rows = orows.permute(x, inv, 2, 1, np.zeros((9, 2)))
    assert rows[:, 0].tolist() == [0, 2, 0, 4, 4, 0, 2, 4, 0]


def test_gradients_against_differences():
    rng = np.random.default_rng(2)
    T, k, E = 5, 3, 4
    ids = rng.integers(-1, E, size=(T, k))
    _, inv = orows.align(ids, E, 1)
    P = T * (k + 1)
    rows, w, d = rng.normal(size=(P, 6)), rng.normal(size=(T, k)), rng.normal(size=(T, 6))
    f = lambda r, v: float((orows.unpermute(r, inv, T, k, 1, v)[0] * d).sum())
    d_rows, d_w, _ = orows.unpermute_backward(d, rows, inv, k, 1, w)
    for p in range(P):
        for i in range(6):
            e = np.zeros_like(rows)
            e[p, i] = 0.5
            assert abs(f(rows + e, w) - f(rows - e, w) - d_rows[p, i]) < 1e-9   # (linear)
    for t in range(T):
        for j in range(k):
            e = np.zeros_like(w)
            e[t, j] = 0.5
            assert abs(f(rows, w + e) - f(rows, w - e) - d_w[t, j]) < 1e-9
