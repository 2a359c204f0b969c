"""int8_linear against FP64: sizes from one row to hundreds, odd M, N and K,
plain and gated layers with every epilogue, codes at their ends, strides,
guards, streams and graphs."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_03_amd import _lib, ops
from oracle import linear as olin
from oracle import rows as orows

from parity import device, to_np

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    return device()


def _gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def _f64(t):
    return to_np(t.float()).astype(np.float64)


def _codes(dev, rows, K, seed):
    g = _gen(dev, seed)
    q = (40.0 * torch.randn(rows, K, generator=g, device=dev)).round().clamp(-128, 127).to(torch.int8)
    return q, 0.001 + 0.002 * torch.rand(rows, generator=g, device=dev)


def _act_error(z, dz, act):
    """Bound of the activation's error for an argument off by dz: the hardware
    exponential and reciprocal, or the polynomial of the normal distribution."""
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


def _reference(xq, sx, wq, sw, bias, act, gated, res, out_dtype):
    """(FP64 result, bound): the sum is exact; its conversion, the scales'
    product and the product with it round once each."""
    v = orows.int8_product(xq, sx, wq, sw)
    dv = 3.01 * HALF * np.abs(v)
    b = None if bias is None else _f64(bias)
    r = None if res is None else _f64(res)
    ref = olin.epilogue(v, b, act, gated, r)
    if b is not None:
        v = v + b
        dv = dv + HALF * (np.abs(v) + dv)
    if gated:
        h = v.shape[1] // 2
        a, u = np.abs(olin.activation(v[:, :h], act)), np.abs(v[:, h:])
        da, du = _act_error(v[:, :h], dv[:, :h], act), dv[:, h:]
        err = da * u + a * du + da * du + HALF * a * u
    else:
        err = _act_error(v, dv, act)
    if r is not None:
        err = err + HALF * (np.abs(ref) + err)
    if out_dtype == BF:
        err = err + 2.0 ** -8 * (np.abs(ref) + err)
    return ref, err + 2.0 ** -125


def _check(got, xq, sx, wq, sw, bias=None, act="none", gated=False, res=None):
    ref, bound = _reference(to_np(xq), to_np(sx), to_np(wq), to_np(sw), bias, act, gated, res, got.dtype)
    assert got.shape == ref.shape
    err = np.abs(_f64(got) - ref)
    assert (err <= bound).all(), f"{float((err / bound).max())} times the bound"


# (act, gated, bias, residual, out)
CONFIGS = [
    ("none", False, False, None, F32),
    ("none", False, True, BF, BF),
    ("relu", False, True, F32, F32),
    ("gelu", False, True, BF, F32),
    ("silu", True, False, None, BF),
    ("silu", True, True, BF, F32),
    ("gelu_tanh", True, True, F32, F32),
    ("gelu_tanh", False, False, None, BF),
]


def _case(dev, M, N, K, cfg, seed=0, codes=True):
    act, gated, with_bias, rt, ot = cfg
    wq, sw = _codes(dev, N, K, 17 + seed)
    w = ops.prepare_int8_weight(wq, sw, gated)
    g = _gen(dev, 31 + M + seed)
    bias = 0.5 * torch.randn(N, generator=g, device=dev) if with_bias else None
    n_out = N // 2 if gated else N
    res = torch.randn(M, n_out, generator=g, device=dev).to(rt) if rt else None
    kw = dict(bias=bias, act=act, residual=res, out_dtype=ot)
    if codes:
        xq, sx = _codes(dev, M, K, 50 + M + seed)
        got = ops.int8_linear(xq, w, sx, **kw)
    else:
        x = (3.0 * torch.randn(M, K, generator=g, device=dev)).to(BF)
        xq, sx = ops.int8_quantize(x)
        got = ops.int8_linear(x, w, **kw)
    assert got.dtype == ot
    _check(got, xq, sx, wq, sw, bias, act, gated, res)
    return got


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 127, 129, 203, 256, 300, 515])
def test_rows(dev, M):
    _case(dev, M, 264, 272, CONFIGS[0])
    _case(dev, M, 264, 400, CONFIGS[5])


@pytest.mark.parametrize("N", [4, 20, 60, 64, 68, 132, 256, 260, 516])
@pytest.mark.parametrize("M", [3, 70, 300])
def test_columns(dev, M, N):
    _case(dev, M, N, 208, CONFIGS[1])
    _case(dev, M, 2 * N, 208, CONFIGS[6])


@pytest.mark.parametrize("K", [16, 48, 64, 80, 112, 128, 144, 192, 256, 272, 384, 512, 528, 1040, 4112])
@pytest.mark.parametrize("M", [1, 40, 290])
def test_contraction(dev, M, K):
    _case(dev, M, 132, K, CONFIGS[2])
    _case(dev, M, 136, K, CONFIGS[4])


@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: "-".join(str(v) for v in c))
@pytest.mark.parametrize("M", [1, 19, 100, 301])
def test_epilogues(dev, M, cfg):
    _case(dev, M, 392, 640, cfg)
    _case(dev, M, 392, 640, cfg, seed=7, codes=False)


# every kernel of the larger sizes, with left-over rows and columns
@pytest.mark.parametrize("M,N,K", [(64, 8200, 1040), (130, 4104, 2064), (700, 2056, 1040), (1030, 4104, 528),
                                   (2049, 1032, 272), (4100, 8200, 144), (600, 40000, 80), (16, 65544, 208),
                                   (17, 1032, 8208), (129, 1032, 8208), (40, 520, 8208), (300, 1032, 8208),
                                   (4096, 4360, 1040), (4100, 4360, 2064), (2100, 16400, 528), (700, 136, 16400)])
@pytest.mark.parametrize("cfg", [CONFIGS[1], CONFIGS[5]], ids=["plain", "gated"])
def test_larger_layers(dev, M, N, K, cfg):
    act, gated, with_bias, rt, ot = cfg
    got = _rows_of_large(dev, M, N, K, cfg)
    assert got.shape == (M, N // 2 if gated else N)


# a handful of rows, on their own kernel and on the tiles'
@pytest.mark.parametrize("M", [1, 4, 9, 16, 17])
@pytest.mark.parametrize("N,K", [(264, 4112), (5128, 1040), (16392, 272), (16392, 2064), (34824, 528), (520, 16400),
                                 (8200, 8208)])
@pytest.mark.parametrize("cfg", [CONFIGS[1], CONFIGS[5]], ids=["plain", "gated"])
def test_a_handful_of_rows(dev, M, N, K, cfg):
    got = _rows_of_large(dev, M, N, K, cfg)
    assert got.shape == (M, N // 2 if cfg[1] else N)


# every tile size, in one part and with K in parts
@pytest.mark.parametrize("M,N,K", [(42, 104, 400), (16, 72, 2576), (61, 136, 128), (17, 2120, 4352), (51, 8648, 128),
                                   (65, 1960, 4624), (65, 16168, 144), (72, 2952, 7440), (36, 34304, 144),
                                   (40, 34824, 272), (17, 16616, 8064), (100, 34824, 272), (66, 18280, 4368),
                                   (1240, 6472, 1536), (5780, 360, 6416), (964, 8552, 1680), (140, 17832, 14336)])
@pytest.mark.parametrize("cfg", [CONFIGS[1], CONFIGS[5]], ids=["plain", "gated"])
def test_tile_sizes(dev, M, N, K, cfg):
    got = _rows_of_large(dev, M, N, K, cfg)
    assert got.shape == (M, N // 2 if cfg[1] else N)


def _rows_of_large(dev, M, N, K, cfg):
    """As _case, with the reference's product on the GPU in FP64 (exact)."""
    act, gated, with_bias, rt, ot = cfg
    wq, sw = _codes(dev, N, K, 5)
    xq, sx = _codes(dev, M, K, 6)
    g = _gen(dev, 7)
    bias = 0.5 * torch.randn(N, generator=g, device=dev)
    n_out = N // 2 if gated else N
    res = torch.randn(M, n_out, generator=g, device=dev).to(rt)
    got = ops.int8_linear(xq, ops.prepare_int8_weight(wq, sw, gated), sx, bias=bias, act=act, residual=res, out_dtype=ot)
    acc = torch.empty(M, N, dtype=torch.float64, device=dev)
    for r in range(0, M, 512):
        acc[r:r + 512] = xq[r:r + 512].double() @ wq.double().t()
    v = acc * sx.double()[:, None] * sw.double()[None]
    dv = 3.01 * HALF * v.abs()
    v = v + bias.double()
    dv = dv + HALF * (v.abs() + dv)
    if gated:
        a, u = v[:, :n_out], v[:, n_out:]
        y = a * torch.sigmoid(a)
        da = 1.13 * dv[:, :n_out] + (8 + 4 * a.abs()) * HALF * y.abs() + 2.0 ** -120
        err = da * u.abs() + y.abs() * dv[:, n_out:] + da * dv[:, n_out:] + HALF * (y * u).abs()
        y = y * u
    else:
        y, err = v, dv
    y = y + res.double()
    err = err + HALF * (y.abs() + err)
    if ot == BF:
        err = err + 2.0 ** -8 * (y.abs() + err)
    assert ((got.double() - y).abs() <= err + 2.0 ** -125).all()
    return got


@pytest.mark.parametrize("M", [2, 20, 100, 300])
def test_codes_at_their_ends(dev, M):
    """|sum| up to 2^14 K just below 2^31, either sign."""
    K = 131056
    xq = torch.full((M, K), -128, dtype=torch.int8, device=dev)
    wq = torch.full((8, K), -128, dtype=torch.int8, device=dev)
    wq[1::2] = 127
    one = lambda n: torch.ones(n, device=dev)
    got = ops.int8_linear(xq, ops.prepare_int8_weight(wq, one(8)), one(M), out_dtype=F32)
    want = torch.tensor([16384.0 * K, -16256.0 * K]).repeat(M, 4)
    assert torch.equal(got.cpu(), want.float())


def test_bf16_input_equals_its_codes(dev):
    wq, sw = _codes(dev, 264, 528, 3)
    w = ops.prepare_int8_weight(wq, sw)
    ws = ops.int8_linear_workspace(400, 264, 528, dev)
    for M in (1, 30, 65, 400):
        x = torch.randn(M, 528, generator=_gen(dev, M), device=dev).to(BF)
        q, s = ops.int8_quantize(x)
        ref = ops.int8_linear(q, w, s)
        assert torch.equal(ops.int8_linear(x, w), ref)
        assert torch.equal(ops.int8_linear(x, w, ws=ws), ref)
        assert torch.equal(ops.int8_linear(q, w, s, ws=ws), ref)


@pytest.mark.parametrize("M,K", [(1, 16), (1, 64), (1, 528), (1, 4112), (1, 32752), (2, 272), (2, 16368), (3, 1040), (4, 8176),
                                 (5, 144), (6, 5440), (7, 4656), (8, 80), (8, 4080), (8, 4096), (3, 16384), (1, 32768)])
def test_few_bf16_rows_equal_their_codes(dev, M, K):
    """Zeros, the ends of the range, infinities and NaN among them, strided or not."""
    wq, sw = _codes(dev, 72, K, 9)
    g = _gen(dev, M + K)
    wide = torch.randn(M, K + 24, generator=g, device=dev).to(BF)
    for x in (wide[:, 8:K + 8], wide[:, :K].contiguous()):
        x[0, K // 2] = 90.0                                    # codes of small parts of the maximum
        for i, what in enumerate((0.0, 2.0 ** -120, 2.0 ** 110, float("inf"), float("nan"))):
            if M > i + 1:
                x[i + 1] = x[i + 1] * what if 0 < what < 2.0 ** 120 else x[i + 1]
                if what == 0.0:
                    x[i + 1] = 0.0
                elif not what < 2.0 ** 120:
                    x[i + 1, K - 1] = what
        for gated in (False, True):
            w = ops.prepare_int8_weight(wq, sw, gated)
            q, s = ops.int8_quantize(x)
            ref = ops.int8_linear(q, w, s, out_dtype=F32)
            got = ops.int8_linear(x, w, out_dtype=F32)
            assert torch.equal(torch.isnan(got), torch.isnan(ref))
            assert torch.equal(got.nan_to_num(), ref.nan_to_num())


def test_quantised_weight(dev):
    w = 0.02 * torch.randn(136, 272, generator=_gen(dev, 1), device=dev)
    x = torch.randn(9, 272, generator=_gen(dev, 2), device=dev).to(BF)
    for gated in (False, True):
        q, s = ops.int8_quantize(w)
        ref = ops.int8_linear(x, ops.prepare_int8_weight(q, s, gated), act="silu")
        assert torch.equal(ops.int8_linear(x, ops.quantize_int8_weight(w, gated), act="silu"), ref)


def test_nan_scales_reach_their_row_and_column(dev):
    for M in (5, 300):
        wq, sw = _codes(dev, 72, 144, 3)
        xq, sx = _codes(dev, M, 144, 4)
        sx[2] = float("nan")
        sw[7] = float("nan")
        bad = torch.isnan(ops.int8_linear(xq, ops.prepare_int8_weight(wq, sw), sx))
        want = torch.zeros_like(bad)
        want[2] = True
        want[:, 7] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("M", [3, 100, 300])
def test_strides_guards_and_results_in_place(dev, M):
    N, K = 136, 272
    wq, sw = _codes(dev, N, K, 3)
    w = ops.prepare_int8_weight(wq, sw)
    xq, sx = _codes(dev, M, K, 4)
    res = torch.randn(M, N, generator=_gen(dev, 5), device=dev).to(BF)
    ref = ops.int8_linear(xq, w, sx, residual=res)
    wide = torch.full((M, K + 32), 127, dtype=torch.int8, device=dev)
    wide[:, 16:16 + K] = xq
    out = torch.full((M + 2, N + 8), 7.0, dtype=BF, device=dev)
    rw = torch.full((M, N + 16), 3.0, dtype=BF, device=dev)
    rw[:, 4:4 + N] = res
    got = ops.int8_linear(wide[:, 16:16 + K], w, sx, residual=rw[:, 4:4 + N], out=out[1:1 + M, 4:4 + N])
    assert torch.equal(got, ref)
    assert (out[0] == 7).all() and (out[-1] == 7).all() and (out[:, :4] == 7).all() and (out[:, 4 + N:] == 7).all()
    odd = torch.empty(M, K + 1, dtype=torch.int8, device=dev)[:, 1:]     # rows that are no whole units apart
    odd.copy_(xq)
    acc = res.clone()
    assert torch.equal(ops.int8_linear(odd, w, sx, residual=acc, out=acc), ref) and torch.equal(acc, ref)


def test_empty_and_refused(dev):
    wq, sw = _codes(dev, 64, 128, 3)
    w = ops.prepare_int8_weight(wq, sw)
    xq, sx = _codes(dev, 4, 128, 4)
    assert ops.int8_linear(xq[:0], w, sx[:0]).shape == (0, 64)
    assert ops.int8_linear(torch.empty(0, 128, dtype=BF, device=dev), w).shape == (0, 64)
    for bad, frag in ((lambda: ops.int8_linear(xq, w), "scales"), (lambda: ops.int8_linear(xq, w, sx[:2]), "scales"),
                      (lambda: ops.int8_linear(xq.to(BF), w, sx), "belong"),
                      (lambda: ops.int8_linear(xq.float(), w), "int8 or bfloat16"),
                      (lambda: ops.int8_linear(xq[:, :64], w, sx), "int8 or bfloat16"),
                      (lambda: ops.int8_linear(xq, w, sx, act="tanh"), "act"),
                      (lambda: ops.int8_linear(xq, w, sx, bias=sx), "bias"),
                      (lambda: ops.int8_linear(xq, w, sx, residual=torch.zeros(4, 32, device=dev)), "residual"),
                      (lambda: ops.int8_linear(xq, w, sx, out=torch.zeros(4, 32, device=dev)), "out must"),
                      (lambda: ops.int8_linear(xq, w, sx.cpu()), "lives on"),
                      (lambda: ops.int8_linear(xq.to(BF).requires_grad_(), w), "no gradient"),
                      (lambda: ops.prepare_int8_weight(wq.float(), sw), "int8"),
                      (lambda: ops.prepare_int8_weight(wq, sw[:3]), "float32")):
        with pytest.raises(ValueError, match=frag):
            bad()
    with pytest.raises(_lib.Nvfp4Error, match="EWORKSPACE"):
        ops.int8_linear(xq.to(BF), w, ws=torch.empty(256, dtype=torch.uint8, device=dev))
    with pytest.raises(_lib.Nvfp4Error, match="N=6"):
        ops.prepare_int8_weight(wq[:6].contiguous(), sw[:6].contiguous())


def test_two_streams_at_once(dev):
    wq, sw = _codes(dev, 2056, 1040, 3)
    w = ops.prepare_int8_weight(wq, sw)
    xs = [torch.randn(M, 1040, generator=_gen(dev, M), device=dev).to(BF) for M in (200, 210)]
    refs = [ops.int8_linear(x, w) for x in xs]
    outs = [torch.empty_like(r) for r in refs]
    wss = [ops.int8_linear_workspace(210, 2056, 1040, dev) for _ in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        for x, o, ws, st in zip(xs, outs, wss, streams):
            with torch.cuda.stream(st):
                ops.int8_linear(x, w, out=o, ws=ws)
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)


@pytest.mark.parametrize("M", [1, 64, 200])
def test_two_graphs_share_a_workspace(dev, M):
    wq, sw = _codes(dev, 1032, 2064, 3)
    ws = ops.int8_linear_workspace(M, 1032, 2064, dev)
    w = [ops.prepare_int8_weight(wq, sw), ops.prepare_int8_weight(wq, sw, gated=True)]
    x = torch.randn(M, 2064, generator=_gen(dev, M), device=dev).to(BF)
    outs = [torch.empty(M, n, dtype=BF, device=dev) for n in (1032, 516)]
    run = lambda i, o: ops.int8_linear(x, w[i], act="silu", out=o, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(2):
            run(i, outs[i])
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(i, outs[i])
        graphs.append(g)
    for seed in range(3):
        x.copy_(torch.randn(M, 2064, generator=_gen(dev, 90 + seed), device=dev))
        for g in (graphs if seed % 2 else graphs[::-1]):
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], ops.int8_linear(x, w[i], act="silu"))


def test_outputs_past_two_gigaelements(dev):
    M, N, K = 33000, 65536, 16
    wq, sw = _codes(dev, N, K, 3)
    xq, sx = _codes(dev, M, K, 4)
    out = ops.int8_linear(xq, ops.prepare_int8_weight(wq, sw), sx)
    assert out.numel() > 1 << 31
    for r in (0, M - 200):
        part = ops.int8_linear(xq[r:r + 200], ops.prepare_int8_weight(wq[-264:].contiguous(), sw[-264:].contiguous()),
                               sx[r:r + 200])
        assert torch.equal(out[r:r + 200, -264:], part)
    _check(out[-3:], xq[-3:], sx[-3:], wq, sw)
