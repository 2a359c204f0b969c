"""rms_norm and int8_quantize against FP64: every type, sizes from 8 to 32768,
codes to the bit, rows at the ends of FP32, rows with NaN or infinity, results
in place, strides, streams and graphs."""
import itertools

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_03_amd import _lib, ops
from oracle import rows as orows

from parity import device, to_np

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -24          # half a step of float32, relative
HALF_BF = 2.0 ** -8


@pytest.fixture(scope="module")
def dev():
    return device()


def _gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def _inputs(dev, T, H, xt, rt, wt, seed=0):
    g = _gen(dev, 1000 * H + T + seed)
    x = torch.randn(T, H, generator=g, device=dev)
    x[:, ::37] *= 20.0
    r = (3.0 * torch.randn(T, H, generator=g, device=dev)).to(rt) if rt else None
    w = (1.0 + 0.25 * torch.randn(H, generator=g, device=dev)).to(wt)
    return x.to(xt), r, w


def _f64(t):
    return to_np(t.float()).astype(np.float64)


def _sum(x, r):
    """h as the framework defines it: FP32 sum, one rounding to the residual's type."""
    return x if r is None else (x.float().cpu() + r.float().cpu()).to(r.dtype)


def _check(n, h, w, eps, rows=slice(None)):
    """y within three FP32 roundings (the factor, two products) and its own;
    codes equal; scales within one rounding (FP64 before it)."""
    y, q, s = orows.rms_norm(_f64(h)[rows], _f64(w), eps)
    if n.y is not None:
        got = _f64(n.y)[rows]
        bound = 3.01 * HALF * np.abs(y) + 2.0 ** -147
        if n.y.dtype == BF:
            bound = bound + HALF_BF * (np.abs(y) + bound) + 2.0 ** -134
        assert (np.abs(got - y) <= bound).all()
    if n.q is not None:
        assert np.array_equal(to_np(n.q)[rows].astype(np.int64), q)
        assert (np.abs(_f64(n.s)[rows] - s) <= 1.001 * HALF * s + 2.0 ** -150).all()


SIZES = [(1, 8), (1, 64), (5, 512), (5, 520), (2, 2048), (7, 2056), (3, 4096), (2, 4104), (3, 8192), (2, 8200),
         (2, 16384), (1, 16392), (2, 24584), (2, 32768), (300, 1032),
         (1500, 64), (1501, 1032), (1100, 2056), (1030, 4104), (1025, 8200), (1027, 20488),
         (4099, 1000), (4097, 4112), (300, 16376), (257, 24584)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("xt,rt,wt,yt", [(BF, BF, BF, BF), (BF, None, BF, F32), (F32, F32, F32, F32)])
def test_sizes(dev, T, H, xt, rt, wt, yt):
    x, r, w = _inputs(dev, T, H, xt, rt, wt)
    n = ops.rms_norm(x, w, 1e-6, residual=r, outputs="both", out_dtype=yt)
    assert n.y.dtype == yt and (n.h is None) == (r is None)
    h = _sum(x, r)
    if r is not None:
        assert torch.equal(n.h.cpu(), h)
    _check(n, h, w, 1e-6)


@pytest.mark.parametrize("xt,rt,wt,yt,outputs", itertools.product((BF, F32), (None, BF, F32), (BF, F32), (BF, F32),
                                                                  ("y", "int8", "both")))
def test_types(dev, xt, rt, wt, yt, outputs):
    x, r, w = _inputs(dev, 9, 1288, xt, rt, wt)
    n = ops.rms_norm(x, w, 1e-5, residual=r, outputs=outputs, out_dtype=yt)
    assert (n.y is None) == (outputs == "int8") and (n.q is None) == (outputs == "y") == (n.s is None)
    h = _sum(x, r)
    if r is not None:
        assert n.h.dtype == rt and torch.equal(n.h.cpu(), h)
    _check(n, h, w, 1e-5)


@pytest.mark.parametrize("top", [127.0, 127.5])
@pytest.mark.parametrize("dt", [BF, F32])
def test_ties_between_codes_go_to_the_even_one(dev, dt, top):
    """Halves: with a maximum of 127 every one lies between two codes exactly."""
    H = 512
    v = torch.arange(H, dtype=torch.float64) % 255 - 127
    v[::2] = v[::2] + 0.5
    v[0] = 127.0
    v = v.clamp(max=top)
    x = torch.stack([v, v * 2.0 ** -20, -v * 2.0 ** 30]).to(dt).to(dev)
    one = torch.ones(H, device=dev, dtype=dt)
    want = orows.quantize(_f64(x))[0]
    n = ops.rms_norm(x, one, 0.0, outputs="int8")
    assert np.array_equal(to_np(n.q), want)
    q, s = ops.int8_quantize(x)
    assert np.array_equal(to_np(q), want)
    if top == 127.0:      # (bfloat16 holds the halves below 64 alone)
        half = np.abs(_f64(x)[0] % 1.0) == 0.5
        assert half.sum() > 100 and (want[:, half] % 2 == 0).all()


@pytest.mark.parametrize("xt,wt", [(BF, BF), (BF, F32), (F32, BF)])
def test_rows_at_the_ends_of_fp32(dev, xt, wt):
    """Magnitudes whose squares, products or factors leave FP32."""
    g = _gen(dev, 5)
    x = torch.randn(12, 264, generator=g, device=dev)
    for i, e in enumerate((120, 100, 64, 30, 0, -30, -58, -62, -90, -110, -120, -126)):
        x[i] *= 2.0 ** e
    x = x.to(xt)
    w = (2.0 ** -3 * torch.randn(264, generator=g, device=dev)).to(wt)
    for eps in (0.0, 1e-6):
        n = ops.rms_norm(x, w, eps, outputs="both", out_dtype=F32)
        _check(n, x, w, eps)
    q, s = ops.int8_quantize(x)
    want, ws = orows.int8_quantize(_f64(x))
    assert np.array_equal(to_np(q), want)
    assert (np.abs(_f64(s) - ws) <= 1.001 * HALF * ws + 2.0 ** -150).all()


def test_rows_without_a_value_and_rows_with_nan_or_infinity(dev):
    for dt in (BF, F32):
        x, _, w = _inputs(dev, 8, 776, dt, None, dt)
        x[1] = 0.0
        x[2, 5] = float("nan")
        x[3, 700] = float("inf")
        x[4, 0] = float("-inf")
        n = ops.rms_norm(x, w, 1e-6, outputs="both")
        good = [0, 1, 5, 6, 7]
        _check(n, x, w, 1e-6, good)
        assert float(n.s[1]) == 0.0 and not n.q[1].any() and not n.y[1].any()
        assert torch.isnan(n.s[2:5]).all() and torch.isnan(n.y[2]).all() and torch.isnan(n.y[3, 700])
        q, s = ops.int8_quantize(x)
        want, ws = orows.int8_quantize(_f64(x)[good])
        assert np.array_equal(to_np(q)[good], want) and torch.isnan(s[2:5]).all() and float(s[1]) == 0.0
        w2 = w.clone()
        w2[3] = float("nan")
        assert torch.isnan(ops.rms_norm(x, w2, outputs="int8").s).all()
        # 0 / 0: the formula's own NaN
        z = ops.rms_norm(torch.zeros(2, 64, dtype=dt, device=dev), w[:64].clone(), 0.0, outputs="both")
        assert torch.isnan(z.y).all() and torch.isnan(z.s).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,K", [(1, 8), (3, 16), (17, 528), (4, 4096), (2, 17408), (1, 32768), (513, 1040), (1030, 1000),
                                 (1027, 2048), (1026, 4088), (1025, 6136), (1029, 8192), (300, 16376), (257, 20480),
                                 (258, 24584)])
def test_int8_quantize(dev, T, K, dt):
    x, _, _ = _inputs(dev, T, K, dt, None, dt, seed=3)
    q, s = ops.int8_quantize(x)
    want, ws = orows.int8_quantize(_f64(x))
    assert np.array_equal(to_np(q), want)
    assert np.array_equal(to_np(s), ws.astype(np.float32))


def test_in_place_strides_and_guards(dev):
    T, H = 37, 1032
    x, r, w = _inputs(dev, T, H, BF, BF, BF)
    ref = ops.rms_norm(x, w, residual=r, outputs="both")
    # h over the residual, y over x
    x2, r2 = x.clone(), r.clone()
    n = ops.rms_norm(x2, w, residual=r2, outputs="both", h=r2, y=x2)
    assert n.h is r2 and n.y is x2
    for a, b in zip(n, ref):
        assert torch.equal(a, b)
    # h over x
    x3 = x.clone()
    n = ops.rms_norm(x3, w, residual=r, outputs="int8", h=x3)
    assert torch.equal(x3, ref.h) and torch.equal(n.q, ref.q) and torch.equal(n.s, ref.s)
    # rows apart, in wider buffers whose other columns stay
    big = [torch.full((T, H + 24), 7.0, dtype=BF, device=dev) for _ in range(4)]
    views = [b[:, 8:8 + H] for b in big]
    views[0].copy_(x)
    views[1].copy_(r)
    n = ops.rms_norm(views[0], w, residual=views[1], outputs="both", h=views[2], y=views[3])
    for a, b in zip(n, ref):
        assert torch.equal(a, b)
    for b in big:
        assert (b[:, :8] == 7).all() and (b[:, 8 + H:] == 7).all()
    # rows that cannot be read in pieces of eight (odd start, transposed): the same results
    odd = torch.empty(T, H + 1, dtype=BF, device=dev)[:, 1:]
    odd.copy_(x)
    n = ops.rms_norm(odd, w, residual=r.t().contiguous().t(), outputs="both")
    for a, b in zip(n, ref):
        assert torch.equal(a, b)
    # codes and scales lie between guards
    buf = torch.full((T * H + 32,), 99, dtype=torch.int8, device=dev)
    sb = torch.full((T + 2,), 5.0, device=dev)
    n = ops.rms_norm(x, w, residual=r, outputs="int8", q=buf[16:16 + T * H].view(T, H), s=sb[1:1 + T])
    assert torch.equal(n.q, ref.q) and torch.equal(n.s, ref.s)
    assert (buf[:16] == 99).all() and (buf[16 + T * H:] == 99).all() and sb[0] == 5 and sb[-1] == 5


def test_more_than_two_gigabytes_of_rows(dev):
    """Row offsets past 2^31 elements."""
    T, H = 70000, 32768
    x = torch.zeros(T, H, dtype=BF, device=dev)
    w = torch.ones(H, dtype=BF, device=dev)
    last, _, _ = _inputs(dev, 3, H, BF, None, BF)
    x[-3:] = last
    n = ops.rms_norm(x, w, outputs="both")
    _check(ops.NormOut(n.y[-3:], None, n.q[-3:], n.s[-3:]), last, w, 1e-6)
    assert not n.q[:4].any() and not n.y[65535:65540].any()


def test_more_rows_than_a_launch_has_threads_for(dev):
    T, H = (1 << 26) + 3, 8
    x = torch.zeros(T, H, dtype=BF, device=dev)
    w = torch.ones(H, dtype=BF, device=dev)
    ends = torch.tensor([0, (1 << 25) - 1, 1 << 25, (1 << 26) - 1, 1 << 26, T - 1], device=dev)
    some, _, _ = _inputs(dev, len(ends), H, BF, None, BF)
    x[ends] = some
    n = ops.rms_norm(x, w, residual=x, outputs="both")
    assert torch.equal(n.h[ends], 2 * some)
    _check(ops.NormOut(n.y[ends], None, n.q[ends], n.s[ends]), 2 * some, w, 1e-6)
    assert int((n.s != 0).sum()) == len(ends) and int(n.y.any(1).sum()) == len(ends)
    q, s = ops.int8_quantize(x)
    qe, se = ops.int8_quantize(some)
    assert torch.equal(q[ends], qe) and torch.equal(s[ends], se) and int((s != 0).sum()) == len(ends)


def test_empty_refused_and_other_streams(dev):
    w = torch.ones(64, dtype=BF, device=dev)
    n = ops.rms_norm(torch.empty(0, 64, dtype=BF, device=dev), w, outputs="both")
    assert n.y.shape == (0, 64) and n.q.shape == (0, 64) and n.s.shape == (0,)
    q, s = ops.int8_quantize(torch.empty(0, 64, dtype=BF, device=dev))
    assert q.shape == (0, 64) and s.shape == (0,)
    x = torch.randn(4, 64, device=dev).to(BF)
    with pytest.raises(ValueError, match="no gradient"):
        ops.rms_norm(x, w.clone().requires_grad_())
    with pytest.raises(ValueError, match="outputs"):
        ops.rms_norm(x, w, outputs="fp8")
    with pytest.raises(ValueError, match="only with a residual"):
        ops.rms_norm(x, w, h=x)
    with pytest.raises(ValueError, match="weight"):
        ops.rms_norm(x, w[:32])
    with pytest.raises(ValueError, match="residual"):
        ops.rms_norm(x, w, residual=x[:2])
    with pytest.raises(ValueError, match="h must be"):
        ops.rms_norm(x, w, residual=x.float(), h=x)
    with pytest.raises(ValueError, match="not made"):
        ops.rms_norm(x, w, outputs="int8", y=x)
    with pytest.raises(ValueError, match="lives on"):
        ops.rms_norm(x, w.cpu())
    with pytest.raises(TypeError):
        ops.rms_norm(x.half(), w)
    with pytest.raises(_lib.Nvfp4Error, match="H=60"):
        ops.rms_norm(x[:, :60].contiguous(), w[:60].contiguous())
    with torch.no_grad():
        ops.rms_norm(x, w.clone().requires_grad_())
    # work ordered on a stream of its own
    x, r, w = _inputs(dev, 257, 2056, BF, BF, BF)
    ref = ops.rms_norm(x, w, residual=r, outputs="both")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x2 = x * 1.0
        n = ops.rms_norm(x2, w, residual=r, outputs="both")
    side.synchronize()
    for a, b in zip(n, ref):
        assert torch.equal(a, b)


def test_graph_replays(dev):
    x, r, w = _inputs(dev, 64, 2048, BF, BF, BF)
    bufs = ops.rms_norm(x, w, residual=r, outputs="both")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.rms_norm(x, w, residual=r, outputs="both", **bufs._asdict())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.rms_norm(x, w, residual=r, outputs="both", **bufs._asdict())
    for seed in range(3):
        x2, r2, _ = _inputs(dev, 64, 2048, BF, BF, BF, seed=seed + 50)
        x.copy_(x2)
        r.copy_(r2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(bufs, ops.rms_norm(x2, w, residual=r2, outputs="both")):
            assert torch.equal(a, b)
