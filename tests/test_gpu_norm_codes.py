"""Codes of rms_norm where float32 rows meet float32 weights (products of up to
48 bits), against rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_03_amd import ops

from parity import device, to_np
from test_oracle_codes import halves, rational_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def _fractions(a):
    return [Fraction(float(x)) for x in a]


# one wavefront a row, several, and several pieces a thread
@pytest.mark.parametrize("T,H", [(64, 264), (12, 2056), (6, 8200)])
@pytest.mark.parametrize("residual", [False, True])
def test_ties_of_float32_rows_and_weights(dev, T, H, residual):
    h, w = halves(T, H, H + T)
    x = torch.from_numpy(h).to(dev)
    if residual:      # (the two halves of h: an exact sum)
        n = ops.rms_norm(x / 2, torch.from_numpy(w).to(dev), residual=x / 2, outputs="both")
        assert torch.equal(n.h, x)
    else:
        n = ops.rms_norm(x, torch.from_numpy(w).to(dev), outputs="both")
    q, wf = to_np(n.q), _fractions(w)
    for r in range(T):
        assert q[r].tolist() == rational_codes([a * b for a, b in zip(_fractions(h[r]), wf)])


@pytest.mark.parametrize("exponent", [-70, -24, 0, 60])
def test_a_quotient_just_above_a_half(dev, exponent):
    # 254 a - 253 top = 1 in whole numbers
    h = torch.zeros(2, 8)
    h[0, :2] = torch.tensor([12523703.0, 10823765.0])
    h[1, :2] = torch.tensor([-12523703.0, -10823765.0])
    w = torch.tensor([12164073.0, 14130145.0] + [1.0] * 6)
    n = ops.rms_norm((h * 2.0 ** exponent).to(dev), w.to(dev), outputs="int8")
    want = np.zeros((2, 8), dtype=np.int8)
    want[0, :2], want[1, :2] = 127, -127
    assert np.array_equal(to_np(n.q), want)
