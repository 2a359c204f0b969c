"""Which kernels int8_linear's shapes reach: the tests' shapes cover every tile
size, with K whole and in parts, for whole layers and for the columns left over
by whole rounds of 256 x 256 tiles (CPU); and the layers with left-over columns
against FP64 (GPU)."""
import ctypes
import itertools
import os

import pytest

import test_gpu_int8
from nvfp4_block_scaled_03_amd import _lib

TILES = [(16, 64), (32, 64), (64, 64), (128, 64), (64, 256), (128, 256), (256, 128), (256, 256)]

# columns left over for every tile size, K whole and in parts, and a prompt's projection
LEFT_OVER = [(3833, 4416, 624), (389, 32848, 5072), (5761, 2848, 576), (2706, 5928, 4512), (3635, 4592, 544),
             (2956, 5432, 4896), (948, 24712, 784), (387, 35368, 8224), (5521, 3000, 656), (1256, 13480, 6768),
             (6237, 3216, 2320), (1602, 10472, 5472), (7088, 3456, 720), (6105, 2944, 6928), (4147, 4832, 13616),
             (4096, 5120, 17408)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


def _plan(lib, M, N, K, gated):
    """[(tile rows, tile columns, parts of K, first column)] of a call's launches."""
    p = (ctypes.c_int32 * 9)()
    assert lib.int8_linear_plan(M, N, K, int(gated), p) == 0
    return [tuple(p[1 + 4 * i:5 + 4 * i]) for i in range(p[0])]


def _shapes(test):
    """(M, N, K) of a parametrised test."""
    lists = {m.args[0]: m.args[1] for m in test.pytestmark if m.name == "parametrize"}
    return lists["M,N,K"] if "M,N,K" in lists else [(M, *nk) for M, nk in itertools.product(lists["M"], lists["N,K"])]


@pytest.mark.parametrize("gated", [False, True])
def test_whole_layers_cover_every_kernel(lib, gated):
    reached = set()
    for test in (test_gpu_int8.test_larger_layers, test_gpu_int8.test_a_handful_of_rows, test_gpu_int8.test_tile_sizes):
        for shape in _shapes(test):
            plan = _plan(lib, *shape, gated)
            if len(plan) == 1:
                reached.add((*plan[0][:2], plan[0][2] > 1))
    assert reached == {(0, 0, False), *((*t, s) for t in TILES for s in (False, True))}


@pytest.mark.parametrize("gated", [False, True])
def test_left_over_columns_cover_every_kernel(lib, gated):
    reached = set()
    for M, N, K in LEFT_OVER:
        plan = _plan(lib, M, N, K, gated)
        assert len(plan) == 2 and plan[0] == (256, 256, 1, 0), (M, N, K)
        assert plan[1][3] > 0 and plan[1][3] % 256 == 0
        reached.add((*plan[1][:2], plan[1][2] > 1))
    # (a remainder of 256 x 256 tiles with K whole would be part of the rounds)
    assert reached == {(*t, s) for t in TILES for s in (False, True)} - {(256, 256, False)}


def test_plans_refused(lib):
    p = (ctypes.c_int32 * 9)()
    assert lib.int8_linear_plan(4, 64, 128, 0, None) == _lib.NVFP4_EINVAL
    for bad in ((0, 64, 128, 0), (4, 66, 128, 0), (4, 68, 128, 1), (4, 64, 24, 0), (4, 64, 131072, 0), (4, 64, 128, 2)):
        assert lib.int8_linear_plan(*bad, p) == _lib.NVFP4_ESHAPE, bad


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", LEFT_OVER)
@pytest.mark.parametrize("cfg", [test_gpu_int8.CONFIGS[1], test_gpu_int8.CONFIGS[5]], ids=["plain", "gated"])
def test_left_over_columns(M, N, K, cfg):
    got = test_gpu_int8._rows_of_large(test_gpu_int8.device(), M, N, K, cfg)
    assert got.shape == (M, N // 2 if cfg[1] else N)
