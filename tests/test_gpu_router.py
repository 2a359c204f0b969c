"""GPU parity of the router: moe_gate and moe_route against oracle/routing.py.

moe_gate: the products are exact, so the FP32 logits may be off by the
rounding of H - 1 sums, each at most half a step of a partial sum that
|x| |w|^T bounds, and of the bias: (H + 1) 2^-24 (|x| |w|^T + |b|).

moe_route: ids equal; weights within the one rounding from FP64 to FP32, half
a step (2^-24), and a few FP64 steps of the exponentials (2^-48).  The inputs
keep choice values further apart than two exponential implementations are
(checked), or exactly equal.
"""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_03_amd import _lib, ops
from oracle import routing as orr

from parity import device, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return device()


def _gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


# ---------------------------------------------------------------- the product
def _check_gate(x, w, b, got):
    xf, wf = to_np(x.float()).astype(np.float64), to_np(w.float()).astype(np.float64)
    bf = None if b is None else to_np(b).astype(np.float64)
    ref = orr.gate_logits(xf, wf, bf)
    bound = (x.shape[1] + 1) * 2.0 ** -24 * (np.abs(xf) @ np.abs(wf).T + (0 if bf is None else np.abs(bf))) + 1e-37
    err = np.abs(to_np(got).astype(np.float64) - ref)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,H", [(1, 1, 8), (1, 128, 2048), (3, 7, 40), (16, 16, 32), (17, 33, 264), (64, 128, 2048),
                                   (65, 60, 1000), (130, 129, 512), (256, 512, 4096), (300, 1024, 72),
                                   (1024, 200, 776), (4100, 128, 256)])
def test_gate(dev, T, E, H, wdt):
    g = _gen(dev, 1000 * T + E)
    x = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    w = (0.05 * torch.randn(E, H, generator=g, device=dev)).to(wdt)
    b = torch.randn(E, generator=g, device=dev)
    _check_gate(x, w, None, ops.gate_logits(x, w))
    _check_gate(x, w, b, ops.gate_logits(x, w, b))


@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32])
def test_gate_strided_rows_and_neighbours(dev, wdt):
    """Rows further apart than H, an output inside a larger buffer whose
    other rows stay as they were."""
    T, E, H = 37, 50, 136
    g = _gen(dev, 5)
    big = torch.randn(T, 3 * H + 8, generator=g, device=dev).to(torch.bfloat16)
    x = big[:, H + 8:2 * H + 8]
    w = torch.randn(E, H, generator=g, device=dev).to(wdt)
    buf = torch.full((T + 2, E), 7.0, device=dev)
    got = ops.gate_logits(x, w, out=buf[1:T + 1])
    _check_gate(x, w, None, got)
    assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    # an odd stride or start is taken by copying
    _check_gate(big[:, 3:H + 3], w, None, ops.gate_logits(big[:, 3:H + 3], w))
    _check_gate(x.t().contiguous().t(), w, None, ops.gate_logits(x.t().contiguous().t(), w))


def test_gate_f32_weights_keep_24_bits(dev):
    """One-hot activations return the float32 weights themselves."""
    H = 64
    w = torch.randn(48, H, generator=_gen(dev, 9), device=dev) * torch.logspace(-20, 20, 48, device=dev)[:, None]
    x = torch.eye(H, device=dev).to(torch.bfloat16)
    assert torch.equal(ops.gate_logits(x, w), w.t())


def test_gate_row_stays_its_own(dev):
    """A row of NaN or infinity changes no other row, and every row is the
    same whatever the batch around it (one kernel choice for equal T)."""
    g = _gen(dev, 11)
    x = torch.randn(40, 256, generator=g, device=dev).to(torch.bfloat16)
    w = torch.randn(24, 256, generator=g, device=dev).to(torch.bfloat16)
    clean = ops.gate_logits(x, w)
    x2 = x.clone()
    x2[5], x2[17] = float("nan"), float("inf")
    got = ops.gate_logits(x2, w)
    keep = [t for t in range(40) if t not in (5, 17)]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,H", [(1, 24, 256), (3, 24, 256), (4, 130, 2056), (40, 24, 256), (300, 130, 520),
                                   (1100, 128, 128), (4100, 128, 72)])
def test_gate_row_whatever_its_place(dev, T, E, H, wdt):
    """At one T a row's logits are the same bits in any place and beside any
    other rows, NaN and infinity among them."""
    g = _gen(dev, T)
    x = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    w = torch.randn(E, H, generator=g, device=dev).to(wdt)
    b = torch.randn(E, generator=g, device=dev)
    want = ops.gate_logits(x, w, b)
    at = torch.randperm(T, generator=g, device=dev)
    assert torch.equal(ops.gate_logits(x[at], w, b), want[at])
    keep = torch.arange(T, device=dev) % 3 == 0
    other = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    other[1::6], other[4::6] = float("nan"), float("inf")
    assert torch.equal(ops.gate_logits(torch.where(keep[:, None], x, other), w, b)[keep], want[keep])


@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,H", [(5, 128, 8192), (64, 60, 8256), (120, 16, 16384), (1000, 120, 4096), (2000, 40, 4104)])
def test_gate_long_ring(dev, T, E, H, wdt):
    """Many trips around the ring of a one-wavefront group, beside another
    stream's traffic: the same bits every time."""
    g = _gen(dev, T)
    x = torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)
    w = (0.05 * torch.randn(E, H, generator=g, device=dev)).to(wdt)
    first = ops.gate_logits(x, w)
    _check_gate(x, w, None, first)
    side, a = torch.cuda.Stream(), torch.empty(1 << 26, device=dev)
    b = torch.zeros_like(a)
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(side):
            a.copy_(b)
        assert torch.equal(ops.gate_logits(x, w), first)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [4, 7])
def test_gate_rows_far_apart(dev, T):
    """Rows whose offsets pass 2^31 elements."""
    H, E, apart = 72, 20, 1 << 30
    buf = torch.empty(T * apart, dtype=torch.bfloat16, device=dev)
    x = buf.view(T, apart)[:, :H]
    x.copy_(torch.randn(T, H, generator=_gen(dev, T), device=dev))
    wg = torch.randn(E, H, generator=_gen(dev, 1), device=dev)
    assert torch.equal(ops.gate_logits(x, wg), ops.gate_logits(x.clone(), wg))
    del buf, x
    torch.cuda.empty_cache()


def test_gate_many_logits(dev):
    """More than 2^31 logits, few of them checked."""
    T, H, E = (1 << 21) + 40, 16, 1024
    x = torch.randn(T, H, generator=_gen(dev, 5), device=dev).to(torch.bfloat16)
    wg = torch.randn(E, H, generator=_gen(dev, 6), device=dev).to(torch.bfloat16)
    z = ops.gate_logits(x, wg)
    for t in (0, T // 2, T - 64):
        rows = slice(t, t + 64)
        ref = orr.gate_logits(to_np(x[rows].float()), to_np(wg.float()))
        bound = H * 2.0 ** -23 * (np.abs(to_np(x[rows].float())) @ np.abs(to_np(wg.float())).T) + 2.0 ** -140
        assert (np.abs(to_np(z[rows]) - ref) <= bound).all()
    # and the choice among them
    ids, w = ops.route_scored(z, 2)
    _check_route(z[T - 64:], (ids[T - 64:], w[T - 64:]), 2)
    del z
    torch.cuda.empty_cache()


# ----------------------------------------------------------------- the choice
def _check_route(logits, got, k, **kw):
    bias = kw.get("bias")
    kw = dict(kw, bias=None if bias is None else to_np(bias))
    ids, w = orr.route_scored(to_np(logits.float()), k, **kw)
    gi, gw = to_np(got[0]), to_np(got[1]).astype(np.float64)
    assert np.array_equal(gi, ids), np.argwhere(gi != ids)[:5]
    err = np.abs(gw - w)
    assert (err <= (2.0 ** -24 + 2.0 ** -48) * np.abs(w) + 2.0 ** -150).all(), float(err.max())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 60, 4), (64, 128, 8), (33, 200, 32), (9, 257, 10),
                                   (40, 512, 10), (7, 1024, 32), (3, 32, 32)])
def test_route(dev, T, E, k, renorm, score, dt):
    g = _gen(dev, 7 * T + E)
    z = (2 * torch.randn(T, E, generator=g, device=dev)).to(dt)
    b = 0.01 * (4 * torch.randn(E, generator=g, device=dev)).round()
    for bias in (None, b):
        kw = dict(score=score, bias=bias, renormalize=renorm, scale=1.0 if renorm else 2.5)
        _check_route(z, ops.route_scored(z, k, **kw), k, **kw)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("T,E,k,groups,keep", [(4, 256, 8, 8, 4), (3, 64, 6, 64, 9), (17, 160, 6, 8, 3),
                                               (2, 1024, 16, 2, 1), (65, 6, 2, 2, 1), (5, 120, 1, 40, 1),
                                               (8, 96, 12, 3, 3), (6, 960, 32, 30, 2)])
def test_route_groups(dev, T, E, k, groups, keep, group_score, score, dt):
    g = _gen(dev, 13 * T + E)
    z = (1.5 * torch.randn(T, E, generator=g, device=dev)).to(dt)
    b = 0.02 * (3 * torch.randn(E, generator=g, device=dev)).round()
    for bias in (None, b):
        kw = dict(score=score, bias=bias, groups=groups, topk_groups=keep, group_score=group_score)
        _check_route(z, ops.route_scored(z, k, **kw), k, **kw)


def test_route_equals_the_plain_router(dev):
    """Softmax without bias or groups: moe_route_topk's results, bit for bit."""
    for T, E, k in ((64, 128, 8), (256, 512, 10), (1, 8, 2)):
        z = torch.randn(T, E, generator=_gen(dev, E), device=dev)
        a, b = ops.route_scored(z, k), ops.route_topk(z, k)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("E", [8, 100, 300, 1024])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties(dev, E, score):
    """Equal logits throughout, and logits from a grid of four values: the
    lower index first, among experts and among groups."""
    flat = torch.zeros(3, E, device=dev)
    grid = torch.randint(0, 4, (50, E), generator=_gen(dev, E), device=dev).float()
    b = torch.full((E,), 0.125, device=dev)
    for z in (flat, grid):
        for bias in (None, b):
            for groups in (1, 2, 4):
                kw = dict(score=score, bias=bias, groups=groups, topk_groups=(groups + 1) // 2, group_score="top2")
                _check_route(z, ops.route_scored(z, 2, **kw), 2, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_route_unavailable(dev, groups, score, dt):
    """Rows masked in part, but for one expert, and whole; infinities, NaN and
    the type's lowest value; biases that close experts."""
    E, k = 32, 6
    g = _gen(dev, 3)
    z = torch.randn(40, E, generator=g, device=dev)
    z[torch.rand(40, E, generator=g, device=dev) < 0.5] = -float("inf")
    z[0] = -float("inf")
    z[1] = float("nan")
    z[2, :-1] = -float("inf")
    z[3, 5], z[3, 9] = float("inf"), float("inf")
    z = z.to(dt)
    z[4] = torch.finfo(dt).min
    z[5] = torch.finfo(dt).max
    z[6, ::2] = torch.finfo(dt).min
    b = 0.1 * torch.randn(E, generator=g, device=dev)
    shut = b.clone()
    shut[::3], shut[1] = -float("inf"), float("nan")
    for bias in (None, b, shut):
        for renorm in (True, False):
            for gs in ("max", "top2"):
                kw = dict(score=score, bias=bias, groups=groups, topk_groups=max(1, groups // 2), group_score=gs,
                          renormalize=renorm)
                got = ops.route_scored(z, k, **kw)
                assert torch.isfinite(got[1]).all()
                _check_route(z, got, k, **kw)


def test_route_strided_logits_and_buffers(dev):
    big = torch.randn(20, 100, generator=_gen(dev, 2), device=dev)
    z = big[:, 10:74]
    ids = torch.full((22, 4), 77, dtype=torch.int32, device=dev)
    w = torch.full((22, 4), 7.0, device=dev)
    got = ops.route_scored(z, 4, ids=ids[1:21], weights=w[1:21])
    _check_route(z, got, 4)
    assert (ids[[0, 21]] == 77).all() and (w[[0, 21]] == 7).all()
    _check_route(z.t().contiguous().t(), ops.route_scored(z.t().contiguous().t(), 4), 4)


def test_route_no_tokens(dev):
    ids, w = ops.route_scored(torch.empty(0, 16, device=dev), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    assert ops.gate_logits(torch.empty(0, 64, dtype=torch.bfloat16, device=dev),
                           torch.zeros(8, 64, device=dev)).shape == (0, 8)


def test_refusals(dev):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(8, 64, device=dev)
    with pytest.raises(ValueError):
        ops.gate_logits(x.float(), w)
    with pytest.raises(ValueError):
        ops.gate_logits(x, w[:, :56])
    with pytest.raises(ValueError):
        ops.gate_logits(x, w, bias=torch.zeros(7, device=dev))
    with pytest.raises(ValueError):
        ops.gate_logits(x, w, out=torch.zeros(4, 9, device=dev))
    with pytest.raises(ValueError):
        ops.gate_logits(x, w.cpu())
    with pytest.raises(TypeError):
        ops.gate_logits(x, w.half())
    with pytest.raises(_lib.Nvfp4Error):
        ops.gate_logits(x[:, :60], w[:, :60])
    z = torch.zeros(4, 8, device=dev)
    for bad in (dict(score="tanh"), dict(group_score="mean"), dict(bias=torch.zeros(9, device=dev)),
                dict(ids=torch.zeros(4, 3, dtype=torch.int32, device=dev)),
                dict(weights=torch.zeros(4, 2, dtype=torch.bfloat16, device=dev))):
        with pytest.raises(ValueError):
            ops.route_scored(z, 2, **bad)
    for bad in (dict(groups=3), dict(groups=2, topk_groups=3), dict(groups=0), dict(scale=0.0),
                dict(scale=float("nan")), dict(groups=8, topk_groups=1)):
        with pytest.raises(_lib.Nvfp4Error):
            ops.route_scored(z, 2, **bad)
    with pytest.raises(TypeError):
        ops.route_scored(z.half(), 2)
    with pytest.raises(_lib.Nvfp4Error):
        ops.route_scored(z, 9)


def test_captured_and_replayed(dev):
    """A captured router (product, choice, alignment): every replay, on new
    activations, equals the eager call."""
    T, E, H, k = 48, 64, 256, 6
    g = _gen(dev, 21)
    w = torch.randn(E, H, generator=g, device=dev)
    b = 0.05 * torch.randn(E, generator=g, device=dev)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    logits = torch.empty(T, E, device=dev)
    ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    wts = torch.empty(T, k, device=dev)

    def step():
        ops.gate_logits(x, w, out=logits)
        ops.route_scored(logits, k, score="sigmoid", bias=b, groups=8, topk_groups=4, group_score="top2", scale=2.5,
                         ids=ids, weights=wts)

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
        replayed = [t.clone() for t in (logits, ids, wts)]
        step()
        torch.cuda.synchronize()
        for a, c in zip(replayed, (logits, ids, wts)):
            assert torch.equal(a, c)


def test_on_another_stream(dev):
    x = torch.randn(512, 512, generator=_gen(dev, 4), device=dev).to(torch.bfloat16)
    w = torch.randn(64, 512, generator=_gen(dev, 5), device=dev)
    want = ops.route_scored(ops.gate_logits(x, w), 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ops.route_scored(ops.gate_logits(x, w), 4)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
