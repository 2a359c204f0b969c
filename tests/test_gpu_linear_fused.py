"""GPU parity of the dense layers with an epilogue (nvfp4_linear_fused,
nvfp4_linear_w4a16_fused, mxfp4_linear_fused) against oracle/linear.py and
oracle/mxfp4.py in FP64.

The operands are exact, so the product v carries FP32 accumulation alone:
dv = K 2^-23 (|x_hat| |W_hat|^T), as for the layers without an epilogue; the
scale and the bias round it by 2 half steps more.  The activation passes an
error on with its largest slope (1.13) and adds its own: the exponential of an
FP32 argument a is off by |a| half steps, the reciprocal, the products and the
sum by a few; GELU's erfc by twice the square of its argument.  A gated value
is a product of two such values.  The residual adds half a step of the sum,
and a bfloat16 output half a step of its own (2^-8).
"""
import functools

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_03_amd import _lib, ops
from oracle import linear as olin
from oracle import mxfp4 as omx
from oracle import nvfp4 as onv

from parity import device, to_np

pytestmark = pytest.mark.gpu

FORMATS = ("w4a4", "w4a16", "mxfp4")
HALF = 2.0 ** -24    # half a step of FP32, relative


@pytest.fixture(scope="module")
def dev():
    return device()


def _gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


@functools.lru_cache(maxsize=8)
def _weight(fmt, N, K, gated, seed=3):
    """(prepared weight, FP64 dequantised weight)"""
    dev = torch.device("cuda")
    w = 0.05 * torch.randn(N, K, generator=_gen(dev, seed), device=dev)
    if fmt == "mxfp4":
        q, ex = omx.quantize(to_np(w).astype(np.float64))
        return ops.quantize_mx_weight(w, gated), omx.dequantize(q, ex)
    c, s, g = olin.quantize_weight(to_np(w))
    return ops.quantize_linear_weight(w, gated), onv.dequantize(c, s, g)


def _x(dev, M, K, seed):
    x = torch.randn(M, K, generator=_gen(dev, seed), device=dev)
    x[:, ::97] *= 20.0
    return x.to(torch.bfloat16)


def _operand(fmt, x):
    xf = to_np(x.float()).astype(np.float64)
    if fmt == "w4a16":
        return xf
    if fmt == "mxfp4":
        return omx.dequantize(*omx.quantize(xf))
    g = onv.global_scale(xf)
    return onv.dequantize(*onv.quantize(xf, g), g)


def _act_error(z, dz, act):
    """Bound of the activation's error for an argument off by dz."""
    a = np.abs(olin.activation(z, act))
    if act in ("none", "relu"):
        return dz
    if act == "silu":
        own = 8 + 4 * np.abs(z)
    elif act == "gelu":
        own = 16 + 4 * z * z
    else:
        own = 16 + 16 * np.abs(1.6 * z * (1 + 0.044715 * z * z))
    return 1.13 * dz + own * HALF * a + 2.0 ** -120


def _reference(fmt, x, w_hat, bias, act, gated, residual, out_dtype, x_hat=None):
    """(FP64 result, bound of the error)"""
    x_hat = _operand(fmt, x) if x_hat is None else x_hat
    v = x_hat @ w_hat.T
    dv = x.shape[1] * 2 * HALF * (np.abs(x_hat) @ np.abs(w_hat).T) + 2 * HALF * np.abs(v)
    b = None if bias is None else to_np(bias).astype(np.float64)
    r = None if residual is None else to_np(residual.float()).astype(np.float64)
    ref = olin.epilogue(v, b, act, gated, r)
    if b is not None:
        v = v + b
        dv = dv + HALF * np.abs(v)
    if gated:
        h = v.shape[1] // 2
        a, u = np.abs(olin.activation(v[:, :h], act)), np.abs(v[:, h:])
        da, du = _act_error(v[:, :h], dv[:, :h], act), dv[:, h:]
        err = da * u + a * du + da * du + HALF * a * u
    else:
        err = _act_error(v, dv, act)
    if r is not None:
        err = err + HALF * (np.abs(ref) + err)
    if out_dtype == torch.bfloat16:
        err = err + 2.0 ** -8 * (np.abs(ref) + err)
    return ref, err + 2.0 ** -125


def _call(fmt, x, w, **kw):
    return ops.mx_linear(x, w, **kw) if fmt == "mxfp4" else ops.linear(x, w, fmt, **kw)


def _check(fmt, x, wt, bias, act, gated, residual, got):
    ref, bound = _reference(fmt, x, wt[1], bias, act, gated, residual, got.dtype)
    err = np.abs(to_np(got.float()).astype(np.float64) - ref)
    assert err.shape == bound.shape
    assert (err <= bound).all(), f"{float((err / bound).max())} times the bound"


# (act, gated, bias, residual type, output type)
CONFIGS = [
    ("none", False, True, None, torch.bfloat16),
    ("none", False, False, torch.bfloat16, torch.bfloat16),
    ("relu", False, True, torch.float32, torch.float32),
    ("silu", True, False, None, torch.bfloat16),
    ("gelu", False, True, torch.bfloat16, torch.float32),
    ("gelu_tanh", True, True, torch.float32, torch.float32),
]


def _case(dev, fmt, M, N, K, cfg, seed=0):
    act, gated, with_bias, rdt, odt = cfg
    wt = _weight(fmt, N, K, gated)
    x = _x(dev, M, K, 100 + M + seed)
    g = _gen(dev, 200 + M + seed)
    bias = 0.5 * torch.randn(N, generator=g, device=dev) if with_bias else None
    n_out = N // 2 if gated else N
    res = torch.randn(M, n_out, generator=g, device=dev).to(rdt) if rdt else None
    got = _call(fmt, x, wt[0], bias=bias, act=act, residual=res, out_dtype=odt)
    assert got.shape == (M, n_out) and got.dtype == odt
    _check(fmt, x, wt, bias, act, gated, res, got)


@pytest.mark.parametrize("cfg", range(len(CONFIGS)))
@pytest.mark.parametrize("M", [1, 2, 4, 5, 16, 17, 32, 33, 40, 41, 64, 65, 100, 128, 129, 203, 300])
@pytest.mark.parametrize("fmt", FORMATS)
def test_fused(dev, fmt, M, cfg):
    _case(dev, fmt, M, 512, 384, CONFIGS[cfg])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 256, 128), (3, 128, 256), (7, 768, 1408), (19, 384, 640), (50, 1280, 128),
                                   (70, 128, 512), (260, 896, 2048), (1000, 256, 896), (515, 640, 128),
                                   # few tiles and a long contraction: split along K and joined
                                   (1, 128, 16384), (16, 256, 17408), (33, 768, 5120), (64, 640, 8192),
                                   (100, 1280, 4096), (48, 2560, 6144)])
def test_fused_sizes(dev, fmt, M, N, K):
    for cfg in (CONFIGS[3], CONFIGS[4]):
        if not (cfg[1] and N % 256):
            _case(dev, fmt, M, N, K, cfg, 7)


def _coded_weight(fmt, N, K, gated):
    """A weight of random codes and scales: (prepared, FP64 dequantised)."""
    rng = np.random.default_rng(N + K)
    codes = rng.integers(0, 16, (N, K), dtype=np.uint8)
    q = torch.from_numpy(codes[:, 0::2] | (codes[:, 1::2] << 4)).cuda()
    if fmt == "mxfp4":
        ex = rng.integers(117, 123, (N, K // 32), dtype=np.uint8)
        return ops.prepare_mx_weight(q, torch.from_numpy(ex).cuda(), gated), omx.dequantize(codes, ex)
    sf, g = rng.integers(0, 127, (N, K // 16), dtype=np.uint8), np.float32(2.0 ** -14)
    return (ops.prepare_linear_weight(q, torch.from_numpy(sf).cuda(), torch.tensor([float(g)]).cuda(), gated),
            onv.dequantize(codes, sf, g))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [
    # many columns: 64-column workgroups for few rows
    (1, 32768, 128), (3, 33280, 256), (8, 32768, 256), (16, 32768, 384), (29, 33024, 256),
    # row blocks of 48 and 64 rows, 128 and 256 columns a tile, N not a multiple of 256
    (40, 8448, 256), (100, 8192, 384), (37, 8448, 2304), (70, 8320, 2304),
    # long contractions: chunks dealt out and joined, also with whole rounds before
    (100, 8320, 4224), (45, 8448, 6144), (333, 8320, 2560),
    # tiles that fill the device
    (1024, 8192, 128), (4100, 2048, 256), (515, 13312, 128)])
def test_fused_large(dev, fmt, M, N, K):
    gated = N % 256 == 0 and M % 2 == 0
    wt = _coded_weight(fmt, N, K, gated)
    x = _x(dev, M, K, M)
    g = _gen(dev, N)
    bias = torch.randn(N, generator=g, device=dev)
    res = torch.randn(M, N // 2 if gated else N, generator=g, device=dev).to(torch.bfloat16)
    got = _call(fmt, x, wt[0], bias=bias, act="silu", residual=res, out_dtype=torch.float32)
    rows = np.unique(np.r_[0:min(M, 40), M // 2, max(0, M - 40):M])
    _check_rows(fmt, x, wt, bias, "silu", gated, res, got, rows)
    again = _call(fmt, x, wt[0], bias=bias, act="silu", residual=res, out_dtype=torch.float32)
    assert torch.equal(got, again)


@pytest.mark.parametrize("M,N,K,gated", [
    # 160 .. 639 pieces of 64 x 64: each width and count of wavefronts
    (130, 4096, 128, False), (250, 5120, 384, True), (330, 5120, 128, False), (333, 8192, 256, True),
    # a whole round of 256 x 256 tiles, the columns left over in 64-row blocks ...
    (300, 33024, 128, False), (300, 33024, 256, True), (512, 34816, 128, False),
    # ... in 128-row tiles, N not a multiple of 256 in the last column tile
    (260, 60032, 128, False), (500, 60160, 128, True),
    # 128-row and 256-row tiles alone
    (1000, 8192, 256, True), (1900, 8320, 128, False), (2100, 8448, 256, True)])
def test_mx_rounds(dev, M, N, K, gated):
    wt = _coded_weight("mxfp4", N, K, gated)
    x = _x(dev, M, K, M)
    g = _gen(dev, N)
    bias = torch.randn(N, generator=g, device=dev)
    res = torch.randn(M, N // 2 if gated else N, generator=g, device=dev).to(torch.bfloat16)
    got = _call("mxfp4", x, wt[0], bias=bias, act="silu", residual=res, out_dtype=torch.float32)
    rows = np.unique(np.r_[0:20, 60:70, 120:135, 250:262, M // 2, M - 40:M])
    _check_rows("mxfp4", x, wt, bias, "silu", gated, res, got, rows[rows < M])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [
    # the widest layers: each activation form, one and two row tiles
    (2, 65536, 128), (6, 65792, 256), (16, 65536, 256), (16, 65536, 6272), (27, 65664, 256),
    # more tiles than the narrow form of the wide kernel takes
    (1100, 16384, 128)])
def test_fused_wide(dev, fmt, M, N, K):
    test_fused_large(dev, fmt, M, N, K)


@pytest.mark.parametrize("fmt", ["w4a4", "w4a16"])
@pytest.mark.parametrize("M,N,K", [(4100, 4352, 128), (4100, 4224, 384), (4099, 4352, 256), (2000, 9600, 128)])
def test_fused_columns_left_over(dev, fmt, M, N, K):
    """More than a round of tiles: the last columns in narrower ones."""
    test_fused_large(dev, fmt, M, N, K)


@pytest.mark.parametrize("fmt", ["w4a4", "w4a16"])
@pytest.mark.parametrize("M,N,K", [(100, 32896, 2432), (250, 16640, 2432), (150, 22016, 2560)])
def test_fused_runs_of_a_chunk(dev, fmt, M, N, K):
    """A few tiles more than workgroups (258 and 260): those left over are dealt
    out in runs of a chunk or none."""
    test_fused_large(dev, fmt, M, N, K)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N", [(65552, 33024), (17, 1 << 20)])
def test_fused_large_output(dev, fmt, M, N):
    """An output of more than 2^31 elements; the widest weight."""
    test_fused_large(dev, fmt, M, N, 128)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", ["w4a4", "w4a16"])
@pytest.mark.parametrize("M,N,K,gated", [
    # operands of more than 2^31 bytes: on 128-row tiles, and on few columns
    (65552, 256, 16512, True), (65552, 256, 16512, False), (66000, 128, 16384, False)])
def test_fused_past_32_bits(dev, fmt, M, N, K, gated):
    wt = _coded_weight(fmt, N, K, gated)
    x = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    x.view(-1)[:1 << 20] = _x(dev, 1, 1 << 20, 7)[0]
    block = x.view(-1)[:1 << 20].clone()
    for at in range(0, M * K, 1 << 20):
        n = min(1 << 20, M * K - at)
        x.view(-1)[at:at + n] = block[:n]
    res = torch.randn(M, N // 2 if gated else N, generator=_gen(dev, N), device=dev).to(torch.bfloat16)
    got = _call(fmt, x, wt[0], act="silu", residual=res, out_dtype=torch.float32)
    rows = np.r_[0:8, M // 2, M - 24:M]
    at = torch.from_numpy(rows).to(dev)
    xs = x[at]
    xf = to_np(xs.float()).astype(np.float64)
    if fmt == "w4a4":
        gs = onv.global_scale(np.array([[float(x.abs().max())]]))
        x_hat = onv.dequantize(*onv.quantize(xf, gs), gs)
    else:
        x_hat = _operand(fmt, xs)
    ref, bound = _reference(fmt, xs, wt[1], None, "silu", gated, res[at], got.dtype, x_hat)
    err = np.abs(to_np(got[at].float()).astype(np.float64) - ref)
    assert (err <= bound).all(), f"{float((err / bound).max())} times the bound"


def _check_rows(fmt, x, wt, bias, act, gated, residual, got, rows):
    """_check on some rows (the activations' global scale is that of all)."""
    at = torch.from_numpy(rows).to(x.device)
    xs = x[at]
    if fmt == "w4a4":
        xf = to_np(x.float()).astype(np.float64)
        gs = onv.global_scale(xf)
        x_hat = onv.dequantize(*onv.quantize(xf[rows], gs), gs)
    else:
        x_hat = _operand(fmt, xs)
    ref, bound = _reference(fmt, xs, wt[1], bias, act, gated, residual[at], got.dtype, x_hat)
    err = np.abs(to_np(got[at].float()).astype(np.float64) - ref)
    assert (err <= bound).all(), f"{float((err / bound).max())} times the bound"


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
def test_activations_far_out(dev, act, gated):
    """Arguments from deep in the left tail to far right: the bias carries
    the argument from -200 to 200."""
    N, K, M = 512, 128, 9
    wt = _weight("w4a16", N, K, gated)
    x = _x(dev, M, K, 5)
    bias = torch.linspace(-200, 200, N, device=dev)
    if gated:
        bias = torch.cat([bias[::2], bias[:N // 2]])
    got = ops.linear(x, wt[0], "w4a16", bias=bias, act=act, out_dtype=torch.float32)
    assert torch.isfinite(got).all()
    _check("w4a16", x, wt, bias, act, gated, None, got)


@pytest.mark.parametrize("lo,hi", [(-0.01, 0.01), (-1, 0), (0, 1), (-3, -1), (1, 3), (-6, -3), (-14, -6), (3, 14)])
def test_gelu_steps(dev, lo, hi):
    """GELU over 2^20 arguments a stretch (the bias, on a product of zero).

    z Phi(z) = max(z, 0) - z q e, with H half a step, relative: the reciprocal
    of a rounded sum is off by 3 H, w r by 4; the polynomial's argument by
    (1 - u) 3 H + H, 7 at most, times its slope over its value, at most 1.04;
    its own roundings add 3 and the fit 1 (1.5e-8 of 0.4 or more); the exponential's
    argument w^2 / 2 is off by 2.5 H and the exponential by 2; two products add
    2.  In all 20 + 1.25 z^2 half steps of z q e, and one of the sum."""
    N, K = 1 << 20, 128
    w = ops.prepare_linear_weight(torch.zeros(N, K // 2, dtype=torch.uint8, device=dev),
                                  torch.full((N, K // 16), 56, dtype=torch.uint8, device=dev),
                                  torch.ones(1, device=dev))
    z = torch.empty(N, device=dev).uniform_(lo, hi, generator=_gen(dev, 3))
    got = ops.linear(torch.zeros(1, K, dtype=torch.bfloat16, device=dev), w, "w4a16", bias=z, act="gelu",
                     out_dtype=torch.float32)[0].double()
    z = z.double()
    ref = 0.5 * z * torch.special.erfc(-z / 2.0 ** 0.5)
    tail = 0.5 * z.abs() * torch.special.erfc(z.abs() / 2.0 ** 0.5)
    bound = HALF * ((20 + 1.25 * z * z) * tail + ref.abs()) + 2.0 ** -120
    err = (got - ref).abs()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 3, 30, 70, 200])
def test_nothing_added_is_the_plain_layer(dev, fmt, M):
    """A zero bias and residual give the layer without an epilogue, within
    its bound (the two may sum K in different orders)."""
    wt = _weight(fmt, 512, 384, False)
    x = _x(dev, M, 384, 9)
    for dt in (torch.float32, torch.bfloat16):
        ref, bound = _reference(fmt, x, wt[1], None, "none", False, None, dt)
        zero = dict(bias=torch.zeros(512, device=dev), residual=torch.zeros(M, 512, device=dev))
        for kw in ({}, zero):
            got = _call(fmt, x, wt[0], out_dtype=dt, **kw)
            assert (np.abs(to_np(got.float()) - ref) <= bound).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M", [1, 13, 37, 90, 150])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_strides_and_neighbours(dev, fmt, gated, M, dt):
    """Output and residual inside wider buffers: nothing beside the output's
    rows and columns is written; then the residual in place."""
    N, K = 512, 256
    n_out = N // 2 if gated else N
    wt = _weight(fmt, N, K, gated)
    x = _x(dev, M, K, 31)
    buf = torch.full((M + 2, n_out + 24), 7.0, dtype=dt, device=dev)
    res = torch.randn(M, n_out + 8, generator=_gen(dev, 8), device=dev).to(dt)[:, 4:4 + n_out]
    out = buf[1:M + 1, 8:8 + n_out]
    got = _call(fmt, x, wt[0], act="silu", residual=res, out=out)
    assert got.data_ptr() == out.data_ptr()
    _check(fmt, x, wt, None, "silu", gated, res, got)
    edge = buf.clone()
    edge[1:M + 1, 8:8 + n_out] = 7
    assert (edge == 7).all()
    first = got.clone()
    out.copy_(res)
    again = _call(fmt, x, wt[0], act="silu", residual=out, out=out)
    assert torch.equal(again, first)
    # a residual of odd stride is taken by copying
    odd = torch.randn(M, n_out + 1, generator=_gen(dev, 8), device=dev).to(dt)[:, 1:]
    _check(fmt, x, wt, None, "silu", gated, odd, _call(fmt, x, wt[0], act="silu", residual=odd, out_dtype=dt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 20, 64, 140])
def test_rows_and_zeros(dev, fmt, M):
    """All-zero activations leave act(bias) + residual, exactly for ReLU."""
    N, K = 256, 256
    wt = _weight(fmt, N, K, False)
    bias = torch.randn(N, generator=_gen(dev, 1), device=dev)
    res = torch.randn(M, N, generator=_gen(dev, 2), device=dev)
    got = _call(fmt, torch.zeros(M, K, dtype=torch.bfloat16, device=dev), wt[0], bias=bias, act="relu",
                residual=res, out_dtype=torch.float32)
    assert torch.equal(got, bias.clamp(min=0) + res)


def test_no_rows(dev):
    for fmt in FORMATS:
        w = _weight(fmt, 512, 256, True)[0]
        assert _call(fmt, torch.empty(0, 256, dtype=torch.bfloat16, device=dev), w, act="silu").shape == (0, 256)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [2, 24, 48, 160])
def test_captured_and_replayed(dev, fmt, M):
    """Two layers in a row (gated, then with the input as residual) captured
    once: every replay on new inputs equals the eager run, with eager work of
    the same buffers in between."""
    H, I = 256, 384
    g = _gen(dev, M)
    up = _weight(fmt, 2 * I, H, True)[0]
    down = _weight(fmt, H, I, False)[0]
    x = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    h = torch.empty(M, I, dtype=torch.bfloat16, device=dev)
    y = torch.empty(M, H, dtype=torch.bfloat16, device=dev)
    if fmt == "mxfp4":
        ws = [ops.mx_linear_workspace(M, 2 * I, H, dev), ops.mx_linear_workspace(M, H, I, dev)]
    else:
        ws = [ops.linear_workspace(M, 2 * I, H, fmt == "w4a4", dev), ops.linear_workspace(M, H, I, fmt == "w4a4", dev)]

    def step():
        _call(fmt, x, up, act="silu", out=h, ws=ws[0])
        _call(fmt, h, down, residual=x, out=y, ws=ws[1])

    x.normal_(generator=g)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        x.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, y)


def _workspace(fmt, sizes, dev):
    """One workspace that is large enough for each of ``sizes`` (M, N, K)."""
    make = ((lambda *a: ops.mx_linear_workspace(*a, dev)) if fmt == "mxfp4"
            else (lambda *a: ops.linear_workspace(*a, fmt == "w4a4", dev)))
    return max((make(*s) for s in sizes), key=lambda t: t.numel())


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_workspace_for_all(dev, fmt):
    """Calls with and without an epilogue, of every size class, one after the
    other in one workspace, equal those in fresh ones; then two captured
    graphs that share it, replayed in turn."""
    N, K = 8192, 128
    w, plain = _weight(fmt, N, K, True)[0], _weight(fmt, N, K, False)[0]
    Ms = (1100, 3, 80, 20, 300, 1)
    xs = {M: _x(dev, M, K, M) for M in Ms}
    res = {M: torch.randn(M, N // 2, generator=_gen(dev, M), device=dev).to(torch.bfloat16) for M in Ms}
    ws = _workspace(fmt, [(M, N, K) for M in Ms], dev)

    def run(M, ws=None):
        return (_call(fmt, xs[M], w, act="silu", residual=res[M], ws=ws), _call(fmt, xs[M], plain, ws=ws))

    fresh = {M: run(M) for M in Ms}
    for _ in range(2):
        for M in Ms:
            for got, want in zip(run(M, ws), fresh[M]):
                assert torch.equal(got, want), M
    torch.cuda.synchronize()
    graphs = {}
    for M in (80, 1100):
        graphs[M] = torch.cuda.CUDAGraph(), [torch.empty_like(t) for t in fresh[M]]
        with torch.cuda.graph(graphs[M][0]):
            for to, t in zip(graphs[M][1], run(M, ws)):
                to.copy_(t)
    for i in range(6):
        M = (80, 1100)[i & 1]
        for t in graphs[M][1]:
            t.zero_()
        graphs[M][0].replay()
        torch.cuda.synchronize()
        for got, want in zip(graphs[M][1], fresh[M]):
            assert torch.equal(got, want), (i, M)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 24, 64, 200])
def test_two_streams(dev, fmt, M):
    """Two calls at once, each on its own stream in its own workspace, equal
    the same calls alone."""
    N, K = 4096, 1024
    w = _weight(fmt, N, K, False)[0]
    xs = [_x(dev, M, K, s) for s in (1, 2)]
    want = [_call(fmt, x, w, act="gelu") for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [_workspace(fmt, [(M, N, K)], dev) for _ in xs]
    out = [torch.empty_like(t) for t in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, o, b in zip(streams, xs, out, ws):
            with torch.cuda.stream(s):
                _call(fmt, x, w, act="gelu", out=o, ws=b)
    torch.cuda.synchronize()
    for o, t in zip(out, want):
        assert torch.equal(o, t)


def test_guard_bands(dev):
    """Output, residual and workspace between known bytes that stay."""
    band = 4096
    for fmt in FORMATS:
        for M in (1, 9, 37, 100, 257):
            for gated in (False, True):
                N, K = 512, 384
                w = _weight(fmt, N, K, gated)[0]
                n_out = N // 2 if gated else N
                wsn = (ops.mx_linear_workspace(M, N, K, dev) if fmt == "mxfp4"
                       else ops.linear_workspace(M, N, K, fmt == "w4a4", dev)).numel()
                full = torch.full((2 * band + wsn,), 0xA5, dtype=torch.uint8, device=dev)
                full[band:band + wsn] = 0
                o = torch.full((2 * band + M * n_out * 2,), 0xA5, dtype=torch.uint8, device=dev)
                out = o[band:band + M * n_out * 2].view(torch.bfloat16).view(M, n_out)
                _call(fmt, _x(dev, M, K, 1), w, act="gelu", bias=torch.zeros(N, device=dev), out=out,
                      ws=full[band:band + wsn])
                for t, n in ((full, wsn), (o, M * n_out * 2)):
                    assert (t[:band] == 0xA5).all() and (t[band + n:] == 0xA5).all(), (fmt, M, gated)


def test_refusals(dev):
    w = _weight("w4a16", 512, 256, True)[0]
    x = _x(dev, 4, 256, 1)
    for bad in (dict(act="tanh"), dict(bias=torch.zeros(256, device=dev)),
                dict(bias=torch.zeros(512, dtype=torch.bfloat16, device=dev)),
                dict(residual=torch.zeros(4, 512, device=dev)), dict(residual=torch.zeros(4, 256)),
                dict(out=torch.zeros(4, 512, dtype=torch.bfloat16, device=dev)),
                dict(out=torch.zeros(4, 257, dtype=torch.bfloat16, device=dev)[:, 1:])):
        with pytest.raises(ValueError):
            ops.linear(x, w, "w4a16", **bad)
    with pytest.raises(ValueError):
        ops.linear(x, w, "w8a8", act="silu")
    with pytest.raises(ValueError):
        ops.linear(x[:, :128], w, "w4a16", act="silu")
    with pytest.raises(ValueError):
        ops.linear(x.float(), w, "w4a16", act="silu")
    with pytest.raises(TypeError):
        ops.linear(x, w, "w4a16", residual=torch.zeros(4, 256, dtype=torch.float16, device=dev))
    with pytest.raises(ValueError):
        ops.quantize_linear_weight(torch.zeros(384, 256, device=dev), gated=True)
    with pytest.raises(_lib.Nvfp4Error):
        ops.linear(x, w, "w4a16", act="silu", ws=torch.zeros(256, dtype=torch.uint8, device=dev)[:0])


def test_refuses_a_scale_elsewhere(dev):
    w = _weight("w4a16", 512, 256, False)[0]
    moved = ops.LinearWeight(w.prep, w.g.cpu(), w.N, w.K)
    with pytest.raises(ValueError):
        ops.linear(_x(dev, 4, 256, 1), moved, "w4a16", act="silu")


def test_refuses_x_as_output(dev):
    for fmt in FORMATS:
        w, x = _weight(fmt, 256, 256, False)[0], _x(dev, 4, 256, 1)
        with pytest.raises(_lib.Nvfp4Error):
            _call(fmt, x, w, residual=x, out=x)


@pytest.mark.parametrize("fmt", ["w4a4", "w4a16"])
@pytest.mark.parametrize("M", [1, 8, 9, 16, 64, 200, 300, 1100])
def test_default_workspace(dev, fmt, M, monkeypatch):
    """Calls without a workspace allocate what they demand, clear no more of it
    than the counter words (or 1 MiB), and equal those in a cleared one, bit for
    bit, whatever the memory held before."""
    N, K = 8192, 2304
    wt = [_coded_weight(fmt, N, K, gated)[0] for gated in (False, True)]
    x, res = _x(dev, M, K, M), torch.randn(M, N // 2, generator=_gen(dev, M), device=dev)
    ws = ops.linear_workspace(M, N, K, fmt == "w4a4", dev)
    calls = [(False, N, lambda ws=None: ops.linear(x, wt[0], fmt, ws=ws)),
             (True, N // 2, lambda ws=None: ops.linear(x, wt[1], fmt, act="silu", residual=res, ws=ws))]
    cleared = []
    zeros, zero_ = torch.zeros, torch.Tensor.zero_
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: cleared.append(zeros(*a, **kw)) or cleared[-1])
    monkeypatch.setattr(torch.Tensor, "zero_", lambda t: cleared.append(t) or zero_(t))
    for fused, cols, run in calls:
        want = run(ws)
        cleared.clear()
        poison = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=dev)
        del poison
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        got = run()
        torch.cuda.synchronize()
        n = _lib.load().nvfp4_linear_call_workspace_size(M, N, K, int(fmt == "w4a4"), int(fused))
        # (the allocator hands out up to 1 MiB more than asked for)
        assert torch.cuda.max_memory_allocated() - before <= n + 2 * M * cols + (2 << 20)
        assert sum(t.numel() for t in cleared) <= (max(512, n * (n <= 1 << 20)) if fmt == "w4a4" else 0)
        assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["w4a4", "w4a16"])
@pytest.mark.parametrize("M,N,K", [
    # every form of the few-row kernel, tiles with and without K dealt out, the grouped kernels
    (1, 512, 384), (8, 512, 384), (9, 512, 384), (16, 8192, 8192), (100, 512, 384), (200, 4096, 1024),
    (64, 8192, 2304), (100, 8320, 4224), (45, 8448, 6144), (1100, 8192, 128)])
def test_demanded_workspace_is_enough(dev, fmt, M, N, K):
    """In exactly the bytes a call demands, between known bytes that stay."""
    band = 4096
    w, x = _coded_weight(fmt, N, K, False)[0], _x(dev, M, K, 1)
    for kw in ({}, dict(act="silu", bias=torch.zeros(N, device=dev))):
        n = _lib.load().nvfp4_linear_call_workspace_size(M, N, K, int(fmt == "w4a4"), int(bool(kw)))
        full = torch.full((2 * band + n,), 0xA5, dtype=torch.uint8, device=dev)
        if fmt == "w4a4":
            full[band:band + 512] = 0
        got = ops.linear(x, w, fmt, ws=full[band:band + n], **kw)
        assert (full[:band] == 0xA5).all() and (full[band + n:] == 0xA5).all()
        assert torch.equal(got, ops.linear(x, w, fmt, **kw))
        with pytest.raises(_lib.Nvfp4Error):
            ops.linear(x, w, fmt, ws=full[band:band + n - 1], **kw)


# One size for each kernel: few rows in each form, tiles, tiles with K dealt out, what fills the device.
KERNELS = [(3, 512, 384), (12, 512, 384), (100, 512, 384), (70, 768, 5120), (1100, 8192, 128)]


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", KERNELS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_and_infinity_go_through(dev, fmt, M, N, K, act):
    """NaN and infinity in bias, residual and (W4A16) x come out where the
    definition has them, of every activation, plain and gated."""
    for gated in (False, True):
        wt = _coded_weight(fmt, N, K, gated)
        n_out = N // 2 if gated else N
        x = _x(dev, M, K, 3)
        if fmt == "w4a16":
            x[M // 2, 5] = float("nan")
            x[M - 1, K - 1] = float("inf")
        bias = torch.randn(N, generator=_gen(dev, 4), device=dev)
        bias[3], bias[64], bias[n_out - 1] = float("nan"), float("inf"), float("-inf")
        if gated:
            bias[n_out + 7] = float("nan")
            bias[n_out + 65:n_out + 68] = torch.tensor([float("inf"), float("-inf"), 0.0], device=dev)
        res = torch.randn(M, n_out, generator=_gen(dev, 5), device=dev)
        res[0, 9], res[M - 1, 10], res[1, 11] = float("nan"), float("inf"), float("-inf")
        got = to_np(_call(fmt, x, wt[0], bias=bias, act=act, residual=res, out_dtype=torch.float32)).astype(np.float64)
        rows = np.unique(np.r_[0:min(M, 12), M // 2, M - 1])
        at = torch.from_numpy(rows).to(dev)
        if fmt == "w4a4":
            xf = to_np(x.float()).astype(np.float64)
            gs = onv.global_scale(xf)
            x_hat = onv.dequantize(*onv.quantize(xf[rows], gs), gs)
        else:
            x_hat = _operand(fmt, x[at])
        with np.errstate(all="ignore"):
            ref, bound = _reference(fmt, x[at], wt[1], bias, act, gated, res[at], torch.float32, x_hat)
            got = got[rows]
            # An activation below 2^-120 may come out as zero in FP32 (_act_error: e^-z past the largest float
            # makes the quotient 0), and zero times an infinite up projection is NaN where the definition has an
            # infinity.
            lost = np.zeros(ref.shape, bool)
            if gated:
                v = x_hat @ wt[1].T + to_np(bias).astype(np.float64)
                lost = np.isinf(v[:, n_out:]) & (np.abs(olin.activation(v[:, :n_out], act)) < 2.0 ** -120)
            assert (lost | (np.isnan(got) == np.isnan(ref))).all()
            assert (lost | (got == ref) | ~np.isinf(ref)).all()
            fin = np.isfinite(ref)
            assert fin.any() and np.isnan(ref).any() and np.isinf(ref).any()
            assert (np.abs(got - ref)[fin] <= bound[fin]).all()


@pytest.mark.parametrize("M,N,K", KERNELS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_every_float_rounds_to_bfloat16(dev, fmt, M, N, K):
    """All-zero activations: the bf16 output is the float32 residual rounded to
    the nearest, ties to even, for any bits: subnormal, largest, infinite, and
    NaN of any payload (which stays NaN)."""
    w = _coded_weight(fmt, N, K, False)[0]
    bits = torch.randint(-2 ** 31, 2 ** 31, (M, N), generator=_gen(dev, 6), dtype=torch.int64, device=dev)
    bits[:, ::7] &= ~0xFFFF                      # on a step, and halfway between two
    bits[:, ::14] |= 0x8000
    bits[:, 1::32] &= ~0x7F800000                # subnormal
    for i, b in enumerate((0x7FFFFFFF, -1, 0x7F800001, 0x7FC00000, 0x7F80FFFF, 0x7F7FFFFF, 0x7F7F7FFF, 0x7F800000,
                           -0x00800000, 1, 0x8000, 0x7FFF)):
        bits[i % M, 2 + 16 * i] = b
    res = bits.to(torch.int32).view(torch.float32)
    got = _call(fmt, torch.zeros(M, K, dtype=torch.bfloat16, device=dev), w, residual=res).cpu()
    want = res.cpu().to(torch.bfloat16)
    nan = torch.isnan(res.cpu())
    assert nan.any() and torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


def test_one_workspace_for_both_kinds(dev):
    """W4A4 and W4A16 calls, with and without an epilogue, in turn in one
    workspace; what W4A4 counts in (64 bytes in) is zero after each."""
    N, K = 512, 8192                                # (M K > 2^18 from 33 rows on: the scale is counted together)
    w = _coded_weight("w4a16", N, K, False)[0]
    Ms = (40, 1, 1100, 16, 300)
    xs = {M: _x(dev, M, K, M) for M in Ms}
    xs[300].zero_()
    bias = torch.randn(N, generator=_gen(dev, 1), device=dev)
    ws = max((ops.linear_workspace(M, N, K, True, dev) for M in Ms), key=lambda t: t.numel())
    for _ in range(2):
        for M in Ms:
            for fmt in ("w4a16", "w4a4"):
                for kw in ({}, dict(bias=bias)):
                    got = ops.linear(xs[M], w, fmt, ws=ws, **kw)
                    assert (ws[64:72] == 0).all(), (M, fmt, kw)
                    assert torch.equal(got, ops.linear(xs[M], w, fmt, **kw)), (M, fmt)


@pytest.mark.parametrize("fmt", ["w4a4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", KERNELS)
def test_quantised_nan_is_the_plain_layers(dev, fmt, M, N, K):
    """NaN in quantised activations: the same operand as without an epilogue
    (a NaN takes no part in a block's scale and becomes a zero)."""
    wt = _coded_weight(fmt, N, K, False)
    x = _x(dev, M, K, 3)
    x[::2, 5], x[M - 1, K - 16:] = float("nan"), float("nan")
    got = _call(fmt, x, wt[0], bias=torch.zeros(N, device=dev), out_dtype=torch.float32)
    want = _call(fmt, x, wt[0], out_dtype=torch.float32)
    clean = torch.where(torch.isnan(x), torch.zeros_like(x), x)
    assert torch.isfinite(got).all()
    assert torch.equal(got, _call(fmt, clean, wt[0], bias=torch.zeros(N, device=dev), out_dtype=torch.float32))
    assert torch.equal(want, _call(fmt, clean, wt[0], out_dtype=torch.float32))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 16, 64, 300])
def test_default_workspace_captured(dev, fmt, M):
    """Calls without a workspace or an output, captured once: every replay on
    new inputs equals the eager calls, with eager work in between."""
    N, K = 1024, 5120                      # (W4A4 clears a small workspace whole, a larger one where it counts)
    plain, gated = _weight(fmt, N, K, False)[0], _weight(fmt, N, K, True)[0]
    x = _x(dev, M, K, 1)

    def step():
        return _call(fmt, x, plain), _call(fmt, x, gated, act="silu")

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        x.copy_(_x(dev, M, K, 20 + i))
        graph.replay()
        torch.cuda.synchronize()
        got_now = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got_now, want):
            assert torch.equal(a, b), i
