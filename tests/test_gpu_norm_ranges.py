"""Rows whose magnitudes leave what FP32 holds exactly, in every layout of the
norm: one wavefront a row or several, one piece a thread or more, many rows."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_03_amd import ops
from oracle import rows as orows

from parity import device
from test_gpu_norm import HALF, _check, _f64, _gen, _sum
from parity import to_np

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EXPONENTS = (120, 100, 64, 30, 0, -30, -58, -62, -90, -110, -120, -126)


@pytest.fixture(scope="module")
def dev():
    return device()


def _rows(dev, T, H, dt):
    x = torch.randn(T, H, generator=_gen(dev, T + H), device=dev)
    e = torch.tensor([2.0 ** v for v in EXPONENTS], device=dev)
    return (x * e[torch.arange(T, device=dev) % len(EXPONENTS)].unsqueeze(1)).to(dt)


# wavefronts a row x pieces a thread: 1 x 1, 4 x 1, 8 x 1, 16 x 1, 16 x 2, 16 x 3, 8 x 4, 8 x 5, 8 x 8; many rows 1 x 2, 4 x 3
@pytest.mark.parametrize("T,H", [(12, 264), (12, 2040), (12, 4088), (12, 8184), (12, 8200), (12, 20488), (264, 16376),
                                 (264, 20472), (12, 32760), (4104, 1000), (4104, 6136)])
@pytest.mark.parametrize("xt,rt,wt", [(BF, None, BF), (BF, BF, BF), (F32, None, F32), (BF, None, F32), (F32, BF, BF)])
def test_rows_at_the_ends_of_fp32(dev, T, H, xt, rt, wt):
    x = _rows(dev, T, H, xt)
    r = _rows(dev, T, H, rt).roll(12, 0) if rt else None
    w = (2.0 ** -3 * torch.randn(H, generator=_gen(dev, H), device=dev)).to(wt)
    rows = slice(None) if T < 1000 else slice(T - 24, T)
    for eps in (0.0, 1e-6):
        n = ops.rms_norm(x, w, eps, residual=r, outputs="both", out_dtype=F32)
        h = _sum(x, r)
        if r is not None:
            assert torch.equal(n.h.cpu(), h)
        _check(n, h, w, eps, rows)


# the quantiser's own layouts: 1 x 1, 1 x 2, 1 x 4, 4 x 2, 4 x 4, 4 x 3, then as above
@pytest.mark.parametrize("T,K", [(12, 264), (1032, 1000), (1032, 2040), (1032, 4088), (1032, 8184), (1032, 6136),
                                 (12, 8184), (12, 20488), (264, 16376), (264, 20472), (264, 32760)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_quantised_rows_at_the_ends_of_fp32(dev, T, K, dt):
    x = _rows(dev, T, K, dt)
    q, s = ops.int8_quantize(x)
    want, ws = orows.int8_quantize(_f64(x))
    assert np.array_equal(to_np(q), want)
    assert (np.abs(_f64(s) - ws) <= 1.001 * HALF * ws + 2.0 ** -150).all()
