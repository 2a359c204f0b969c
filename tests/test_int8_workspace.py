"""The workspace that int8_linear_workspace makes: for every call it promises,
or refused.  Sizes on the CPU; calls with it on the GPU."""
import os

import pytest
import torch

from nvfp4_block_scaled_03_amd import _lib, ops


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


# around the 32768 from which on bfloat16 rows are not taken
@pytest.mark.parametrize("K", [16, 1040, 32768, 32784, 40960, 65536, 131056])
@pytest.mark.parametrize("M,N", [(1, 4), (40, 520), (300, 1032), (4096, 5120)])
def test_as_large_as_every_call_demands(lib, M, N, K):
    have = ops.int8_linear_workspace(M, N, K, "cpu").numel()
    for x_dtype in (_lib.NVFP4_BF16, _lib.NVFP4_I8):
        for m in {1, M // 2, M}:
            assert have >= lib.int8_linear_workspace_size(m, N, K, x_dtype)
    assert lib.int8_linear_workspace_size(M, N, K, _lib.NVFP4_I8) > 0


@pytest.mark.parametrize("M,N,K", [(4, 66, 128), (4, 64, 24), (4, 64, 131072), (-1, 64, 128), (4, 0, 128), (4, 1 << 21, 128),
                                   ((1 << 24) + 1, 64, 128), (1 << 24, 1 << 20, 128), (0, 66, 128)])
def test_refused(lib, M, N, K):
    with pytest.raises(ValueError, match="int8"):
        ops.int8_linear_workspace(M, N, K, "cpu")


def test_no_rows(lib):
    assert ops.int8_linear_workspace(0, 64, 128, "cpu").numel() >= 256


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(40, 520, 40960), (300, 1032, 65536), (3, 264, 131056)])
@pytest.mark.parametrize("gated", [False, True])
def test_long_rows_with_it(M, N, K, gated):
    """Codes past 32768 columns, with K in parts: against exact sums."""
    from parity import device
    dev = device()
    g = torch.Generator(device=dev).manual_seed(M)
    codes = lambda rows: torch.randint(-128, 128, (rows, K), generator=g, device=dev, dtype=torch.int8)
    xq, wq = codes(M), codes(N)
    sx = 0.5 + torch.rand(M, generator=g, device=dev)
    sw = torch.exp2(torch.randint(-30, -20, (N,), generator=g, device=dev).float())
    w = ops.prepare_int8_weight(wq, sw, gated)
    got = ops.int8_linear(xq, w, sx, out_dtype=torch.float32, ws=ops.int8_linear_workspace(M, N, K, dev))
    v = (xq.double() @ wq.double().t()) * sx.double()[:, None] * sw.double()[None]      # (sums below 2^53)
    # the sum's conversion to float32, the scales' product and theirs: three roundings
    err = 3.01 * 2.0 ** -24 * v.abs()
    if gated:
        a, u, da, du = v[:, :N // 2], v[:, N // 2:], err[:, :N // 2], err[:, N // 2:]
        v, err = a * u, da * u.abs() + du * a.abs() + da * du + 2.0 ** -24 * (a * u).abs() * (1 + 2.0 ** -20)
    assert ((got.double() - v).abs() <= err).all()
