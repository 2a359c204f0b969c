"""Refusals and size queries of the norm, the int8 layers and the movement of
rows by expert (CPU only: no kernel is launched)."""
import ctypes
import os

import pytest

from nvfp4_block_scaled_03_amd import _lib

P = 1 << 20      # a pointer that no refused call follows


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


def _fails(lib, rc, code, frag):
    assert rc == code, (rc, lib.nvfp4_last_error())
    assert frag in lib.nvfp4_last_error().decode()


def _norm(**kw):
    a = dict(x=P, ldx=64, residual=2 * P, ld_residual=64, weight=3 * P, h=4 * P, ld_h=64, y=5 * P, ld_y=64, q=6 * P,
             s=7 * P, x_dtype=0, residual_dtype=0, w_dtype=0, y_dtype=0, eps=1e-6)
    a.update(kw)
    return _lib.RmsNormArgs(**a)


@pytest.mark.parametrize("args,rows,H,code,frag", [
    (dict(x_dtype=2), 4, 64, _lib.NVFP4_EINVAL, "x_dtype=2"),
    (dict(y_dtype=-1), 4, 64, _lib.NVFP4_EINVAL, "y_dtype=-1"),
    (dict(eps=-1.0), 4, 64, _lib.NVFP4_EINVAL, "eps"),
    (dict(eps=float("nan")), 4, 64, _lib.NVFP4_EINVAL, "eps"),
    (dict(), -1, 64, _lib.NVFP4_ESHAPE, "rows=-1"),
    (dict(), 1 << 31, 64, _lib.NVFP4_ESHAPE, "rows < 2^31"),
    (dict(), 4, 60, _lib.NVFP4_ESHAPE, "H=60"),
    (dict(), 4, 0, _lib.NVFP4_ESHAPE, "H=0"),
    (dict(ldx=32776), 4, 32776, _lib.NVFP4_ESHAPE, "at most 32768"),
    (dict(ldx=56), 4, 64, _lib.NVFP4_ESHAPE, "ldx=56"),
    (dict(ld_residual=68), 4, 64, _lib.NVFP4_ESHAPE, "ld_residual=68"),
    (dict(ld_h=0), 4, 64, _lib.NVFP4_ESHAPE, "ld_h=0"),
    (dict(ld_y=65), 4, 64, _lib.NVFP4_ESHAPE, "ld_y=65"),
    (dict(x=None), 4, 64, _lib.NVFP4_EINVAL, "null"),
    (dict(weight=None), 4, 64, _lib.NVFP4_EINVAL, "null"),
    (dict(y=None, q=None), 4, 64, _lib.NVFP4_EINVAL, "null"),
    (dict(s=None), 4, 64, _lib.NVFP4_EINVAL, "null"),
    (dict(residual=None), 4, 64, _lib.NVFP4_EINVAL, "h only with a residual"),
    (dict(x=P + 8), 4, 64, _lib.NVFP4_EINVAL, "misaligned"),
    (dict(q=P + 4), 4, 64, _lib.NVFP4_EINVAL, "misaligned"),
    (dict(h=2 * P, ld_h=72), 4, 64, _lib.NVFP4_EINVAL, "in place"),
    (dict(h=P, x_dtype=1), 4, 64, _lib.NVFP4_EINVAL, "in place"),
    (dict(y=4 * P), 4, 64, _lib.NVFP4_EINVAL, "y is h"),
    (dict(y=2 * P), 4, 64, _lib.NVFP4_EINVAL, "residual"),
    (dict(y=P, y_dtype=1), 4, 64, _lib.NVFP4_EINVAL, "in place"),
])
def test_rms_norm_refuses(lib, args, rows, H, code, frag):
    _fails(lib, lib.rms_norm(_norm(**args), rows, H, None), code, frag)


def test_rms_norm_of_no_rows_and_no_args(lib):
    assert lib.rms_norm(_norm(x=None, weight=None, y=None, q=None, s=None, h=None, residual=None), 0, 64, None) == 0
    _fails(lib, lib.rms_norm(None, 4, 64, None), _lib.NVFP4_EINVAL, "NULL")


@pytest.mark.parametrize("args,code,frag", [
    ((P, 2, 4, 64, 64, P, P, None), _lib.NVFP4_EINVAL, "dtype=2"),
    ((P, 0, 4, 60, 64, P, P, None), _lib.NVFP4_ESHAPE, "K=60"),
    ((P, 0, 4, 64, 56, P, P, None), _lib.NVFP4_ESHAPE, "ldx=56"),
    ((P, 0, -4, 64, 64, P, P, None), _lib.NVFP4_ESHAPE, "rows=-4"),
    ((P, 0, 4, 65536, 65536, P, P, None), _lib.NVFP4_ESHAPE, "at most 32768"),
    ((None, 0, 4, 64, 64, P, P, None), _lib.NVFP4_EINVAL, "null"),
    ((P, 0, 4, 64, 64, P, None, None), _lib.NVFP4_EINVAL, "null"),
    ((P + 2, 0, 4, 64, 64, P, P, None), _lib.NVFP4_EINVAL, "misaligned"),
])
def test_int8_quantize_refuses(lib, args, code, frag):
    _fails(lib, lib.int8_quantize(*args), code, frag)
    assert lib.int8_quantize(None, 0, 0, 64, 64, None, None, None) == 0


def test_int8_sizes(lib):
    assert lib.int8_prep_weights_size(64, 128, 0) == 64 * 128
    assert lib.int8_prep_weights_size(4, 16, 0) == 64 * 128          # whole fours of tiles, pairs of chunks
    assert lib.int8_prep_weights_size(72, 144, 1) == 128 * 256       # 36 gate columns: 3 pairs of tiles, in fours
    for bad in ((6, 128, 0), (4, 128, 1), (64, 24, 0), (64, 131072, 0), (0, 128, 0), (64, 128, 2), (1 << 21, 128, 0),
                (1 << 20, (1 << 15) + 16, 0)):
        assert lib.int8_prep_weights_size(*bad) == 0, bad
    assert lib.int8_linear_workspace_size(3, 64, 128, 0) >= 3 * 128 + 3 * 4
    assert lib.int8_linear_workspace_size(3, 64, 128, 1) == 0
    for x_dtype in (0, 2):
        sizes = [lib.int8_linear_workspace_size(M, 4096, 1024, x_dtype) for M in range(0, 700, 7)]
        assert sizes == sorted(sizes)
    for M in (1, 100, 5000):
        assert lib.int8_linear_workspace_size(M, 4096, 1024, 0) >= lib.int8_linear_workspace_size(M, 4096, 1024, 2)


def _linear(lib, x=P, x_dtype=2, ldx=128, sx=2 * P, M=4, N=64, K=128, w=3 * P, sw=4 * P, epi=None, out=5 * P, out_dtype=0,
            ws=6 * P, ws_bytes=1 << 30):
    e = None if epi is None else _lib.Epilogue(**{**dict(act=0, gated=0, ld_out=N), **epi})
    return lib.int8_linear(x, x_dtype, ldx, sx, M, N, K, w, sw, e, out, out_dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("args,code,frag", [
    (dict(x_dtype=1), _lib.NVFP4_EINVAL, "x_dtype=1"),
    (dict(M=-1), _lib.NVFP4_ESHAPE, "M=-1"),
    (dict(M=(1 << 24) + 1), _lib.NVFP4_ESHAPE, "M <= 2^24"),
    (dict(N=66), _lib.NVFP4_ESHAPE, "N=66"),
    (dict(N=0), _lib.NVFP4_ESHAPE, "N=0"),
    (dict(N=68, epi=dict(gated=1, ld_out=36)), _lib.NVFP4_ESHAPE, "N=68"),
    (dict(K=120), _lib.NVFP4_ESHAPE, "K=120"),
    (dict(K=131072, ldx=131072), _lib.NVFP4_ESHAPE, "K=131072"),
    (dict(K=32784, ldx=32784, x_dtype=0), _lib.NVFP4_ESHAPE, "at most 32768"),
    (dict(ldx=112), _lib.NVFP4_ESHAPE, "ldx=112"),
    (dict(ldx=136), _lib.NVFP4_ESHAPE, "ldx=136"),
    (dict(ldx=(1 << 22) + 16), _lib.NVFP4_ESHAPE, "at most 2^22"),
    (dict(N=1 << 20, K=(1 << 15) + 16, ldx=(1 << 15) + 16), _lib.NVFP4_ESHAPE, "N K <= 2^35"),
    (dict(out_dtype=2), _lib.NVFP4_EINVAL, "out_dtype=2"),
    (dict(epi=dict(act=5)), _lib.NVFP4_EINVAL, "act=5"),
    (dict(epi=dict(gated=2)), _lib.NVFP4_ESHAPE, "gated=2"),
    (dict(epi=dict(ld_out=62)), _lib.NVFP4_ESHAPE, "ld_out=62"),
    (dict(epi=dict(residual=P, residual_dtype=2, ld_residual=64)), _lib.NVFP4_EINVAL, "residual_dtype=2"),
    (dict(epi=dict(residual=5 * P, residual_dtype=1, ld_residual=64)), _lib.NVFP4_EINVAL, "in place of out"),
    (dict(x=None), _lib.NVFP4_EINVAL, "null"),
    (dict(sx=None), _lib.NVFP4_EINVAL, "null"),
    (dict(w=None), _lib.NVFP4_EINVAL, "null"),
    (dict(sw=None), _lib.NVFP4_EINVAL, "null"),
    (dict(out=None), _lib.NVFP4_EINVAL, "null"),
    (dict(x=P + 8), _lib.NVFP4_EINVAL, "aligned"),
    (dict(sw=P + 2), _lib.NVFP4_EINVAL, "aligned"),
    (dict(out=P + 4), _lib.NVFP4_EINVAL, "aligned"),
    (dict(out=P), _lib.NVFP4_EINVAL, "out is x"),
    (dict(x_dtype=0, ws_bytes=256), _lib.NVFP4_EWORKSPACE, "needed"),
    (dict(x_dtype=0, ws=None), _lib.NVFP4_EWORKSPACE, "needed"),
    (dict(x_dtype=0, ws=P + 128), _lib.NVFP4_EINVAL, "aligned"),
])
def test_int8_linear_refuses(lib, args, code, frag):
    _fails(lib, _linear(lib, **args), code, frag)


def test_int8_linear_of_no_rows(lib):
    assert _linear(lib, M=0, x=None, sx=None, w=None, sw=None, out=None, ws=None, ws_bytes=0) == 0
    _fails(lib, lib.int8_prep_weights(64, 128, 0, None, P, None), _lib.NVFP4_EINVAL, "null")
    _fails(lib, lib.int8_prep_weights(64, 128, 0, P + 8, P, None), _lib.NVFP4_EINVAL, "aligned")
    _fails(lib, lib.int8_prep_weights(66, 128, 0, P, P, None), _lib.NVFP4_ESHAPE, "N=66")


def _d(T=4, topk=2, E=8, H=1, I=1, shared=1):
    return _lib.Dims(T, topk, E, H, I, shared)


def _permute(lib, d=None, x=P, dtype=0, width=64, ldx=64, off=2 * P, inv=3 * P, rows=4 * P):
    return lib.moe_permute(d or _d(), x, dtype, width, ldx, off, inv, rows, 1, None)


def _unpermute(lib, d=None, rows=P, dtype=0, width=64, off=2 * P, inv=3 * P, w=4 * P, out=5 * P, out_dtype=0):
    return lib.moe_unpermute(d or _d(), rows, dtype, width, off, inv, w, out, out_dtype, None)


def _backward(lib, d=None, d_out=P, out_dtype=0, rows=2 * P, dtype=0, width=64, off=3 * P, inv=4 * P, w=5 * P,
              d_rows=6 * P, d_w=7 * P):
    return lib.moe_unpermute_backward(d or _d(), d_out, out_dtype, rows, dtype, width, off, inv, w, d_rows, d_w, 1, None)


@pytest.mark.parametrize("fn,args,code,frag", [
    (_permute, dict(d=_d(topk=9)), _lib.NVFP4_ESHAPE, "topk=9"),
    (_permute, dict(d=_d(T=-1)), _lib.NVFP4_ESHAPE, "T=-1"),
    (_permute, dict(d=_d(T=1 << 23)), _lib.NVFP4_ESHAPE, "exceeds 2^24"),
    (_permute, dict(d=_d(E=1024)), _lib.NVFP4_ESHAPE, "exceeds 1024"),
    (_permute, dict(width=60), _lib.NVFP4_ESHAPE, "width=60"),
    (_permute, dict(width=(1 << 20) + 8), _lib.NVFP4_ESHAPE, "width"),
    (_permute, dict(d=_d(T=1 << 22, topk=2), width=1 << 20, ldx=1 << 20), _lib.NVFP4_ESHAPE, "2^40"),
    (_permute, dict(d=_d(T=1 << 22, topk=1), width=8192, ldx=8192), _lib.NVFP4_ESHAPE, "64 GiB"),
    (_unpermute, dict(d=_d(T=1 << 22, topk=1), width=4096, dtype=1), _lib.NVFP4_ESHAPE, "64 GiB"),
    (_permute, dict(ldx=56), _lib.NVFP4_ESHAPE, "ldx=56"),
    (_permute, dict(dtype=2), _lib.NVFP4_EINVAL, "dtype=2"),
    (_permute, dict(x=None), _lib.NVFP4_EINVAL, "null"),
    (_permute, dict(inv=None), _lib.NVFP4_EINVAL, "null"),
    (_permute, dict(x=P + 8), _lib.NVFP4_EINVAL, "aligned"),
    (_permute, dict(rows=P), _lib.NVFP4_EINVAL, "rows is x"),
    (_unpermute, dict(width=4), _lib.NVFP4_ESHAPE, "width=4"),
    (_unpermute, dict(out_dtype=2), _lib.NVFP4_EINVAL, "out_dtype=2"),
    (_unpermute, dict(out=None), _lib.NVFP4_EINVAL, "null"),
    (_unpermute, dict(rows=P + 4), _lib.NVFP4_EINVAL, "aligned"),
    (_unpermute, dict(out=P), _lib.NVFP4_EINVAL, "out is rows"),
    (_backward, dict(d_rows=None, d_w=None), _lib.NVFP4_EINVAL, "null"),
    (_backward, dict(rows=None), _lib.NVFP4_EINVAL, "null"),
    (_backward, dict(d_w=P + 2), _lib.NVFP4_EINVAL, "aligned"),
    (_backward, dict(d_rows=2 * P), _lib.NVFP4_EINVAL, "d_rows is rows"),
    (_backward, dict(dtype=3), _lib.NVFP4_EINVAL, "dtype=3"),
])
def test_rows_by_expert_refuse(lib, fn, args, code, frag):
    _fails(lib, fn(lib, **args), code, frag)


def test_rows_by_expert_of_no_tokens(lib):
    d = _d(T=0)
    none = dict(d=d, off=None, inv=None)
    assert _permute(lib, x=None, rows=None, **none) == 0
    assert _unpermute(lib, rows=None, out=None, **none) == 0
    assert _backward(lib, d_out=None, rows=None, d_rows=None, d_w=None, **none) == 0
    assert lib.moe_permute(None, P, 0, 64, 64, P, P, P, 0, None) == _lib.NVFP4_EINVAL


def test_struct_layout_matches_the_header():
    assert ctypes.sizeof(_lib.RmsNormArgs) == 11 * 8 + 5 * 4 + 4
