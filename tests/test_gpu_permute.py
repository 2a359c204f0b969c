"""moe_permute and moe_unpermute against FP64: both types, shared experts,
dropped pairs, the same expert twice, odd widths, gradients by the formula and
by differences, strides, streams and graphs."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_03_amd import _lib, ops
from oracle import rows as orows

from parity import device, to_np

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF, HALF_BF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def dev():
    return device()


def _f64(t):
    return to_np(t.detach().float()).astype(np.float64)


def _setup(dev, T, k, E, shared, seed=0, dropped=0.0):
    g = torch.Generator(device=dev).manual_seed(100 * T + 10 * k + E + seed)
    ids = torch.randint(0, E, (T, k), generator=g, device=dev, dtype=torch.int32)      # (repeats among them)
    if dropped:
        ids = torch.where(torch.rand(T, k, generator=g, device=dev) < dropped, torch.full_like(ids, -1), ids)
    d = ops.dims(T, k, E, 128, 128, shared)
    w = torch.rand(T, k, generator=g, device=dev) - 0.3
    _, inv = orows.align(to_np(ids), E, shared)
    return g, d, ops.moe_align(d, ids), w, inv


def _rand(g, dev, dt, *shape):
    return torch.randn(*shape, generator=g, device=dev).to(dt)


CASES = [(1, 1, 1, 0, 0.0), (1, 8, 16, 1, 0.0), (3, 2, 4, 0, 0.5), (5, 10, 12, 1, 0.3), (17, 3, 5, 1, 0.0),
         (40, 8, 64, 0, 0.9), (6, 4, 4, 0, 1.0), (6, 4, 4, 1, 1.0), (130, 5, 9, 1, 0.2),
         (4, 26, 30, 1, 0.1), (9, 80, 90, 0, 0.5)]


@pytest.mark.parametrize("dt,ot", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,k,E,shared,dropped", CASES)
@pytest.mark.parametrize("W", [8, 72, 512, 1032])
def test_there_and_back(dev, T, k, E, shared, dropped, W, dt, ot):
    g, d, al, w, inv = _setup(dev, T, k, E, shared, W, dropped)
    P = T * (k + shared)
    x = _rand(g, dev, dt, T, W)
    rows = ops.moe_permute(d, x, al)
    assert np.array_equal(_f64(rows), orows.permute(_f64(x), inv, k, shared, np.zeros((P, W))))
    into = torch.full((P, W), 3.0, dtype=dt, device=dev)
    assert ops.moe_permute(d, x, al, out=into) is into
    assert np.array_equal(_f64(into), orows.permute(_f64(x), inv, k, shared, np.full((P, W), 3.0)))
    rows = _rand(g, dev, dt, P, W)
    rows[int((inv >= 0).sum()):] = float("nan")       # rows of no pair are not read
    for weights in (w, None):
        got = ops.moe_unpermute(d, rows, al, weights, out_dtype=ot)
        assert got.dtype == ot
        want, mag = orows.unpermute(_f64(rows), inv, T, k, shared, None if weights is None else _f64(weights))
        bound = (k + shared) * HALF * mag
        if ot == BF:
            bound = bound + HALF_BF * (np.abs(want) + bound) + 2.0 ** -134
        assert (np.abs(_f64(got) - want) <= bound).all()
        out = torch.empty(T, W, dtype=ot, device=dev)
        assert ops.moe_unpermute(d, rows, al, weights, out=out) is out and torch.equal(out, got)


@pytest.mark.parametrize("dt,ot", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,k,E,shared,dropped", CASES)
@pytest.mark.parametrize("W", [8, 520, 2056])
def test_gradients(dev, T, k, E, shared, dropped, W, dt, ot):
    g, d, al, w, inv = _setup(dev, T, k, E, shared, W, dropped)
    P = T * (k + shared)
    # of the sorted rows: every token's sum, in x's type
    x = _rand(g, dev, dt, T, W).requires_grad_()
    d_rows = _rand(g, dev, dt, P, W)
    dx, = torch.autograd.grad(ops.moe_permute(d, x, al), x, d_rows)
    want, mag = orows.unpermute(_f64(d_rows), inv, T, k, shared)
    bound = (k + shared) * HALF * mag
    if dt == BF:
        bound = bound + HALF_BF * (np.abs(want) + bound)
    assert dx.dtype == dt and (np.abs(_f64(dx) - want) <= bound).all()
    # of the weighted sum
    rows, w = _rand(g, dev, dt, P, W).requires_grad_(), w.requires_grad_()
    d_out = _rand(g, dev, ot, T, W)
    gr, gw = torch.autograd.grad(ops.moe_unpermute(d, rows, al, w, out_dtype=ot), (rows, w), d_out)
    wr, ww, mag = orows.unpermute_backward(_f64(d_out), _f64(rows), inv, k, shared, _f64(w))
    bound = HALF * np.abs(wr) + (HALF_BF * np.abs(wr) * (1 + HALF) if dt == BF else 0.0) + 2.0 ** -134
    assert gr.dtype == dt and (np.abs(_f64(gr) - wr) <= bound).all()
    assert gw.dtype == F32 and (np.abs(_f64(gw) - ww) <= (W / 64 + 8) * HALF * mag + 2.0 ** -140).all()
    # one of the two alone, and without weights
    assert torch.equal(torch.autograd.grad(ops.moe_unpermute(d, rows.detach(), al, w, out_dtype=ot), w, d_out)[0], gw)
    assert torch.equal(torch.autograd.grad(ops.moe_unpermute(d, rows, al, w.detach(), out_dtype=ot), rows, d_out)[0], gr)
    one, = torch.autograd.grad(ops.moe_unpermute(d, rows, al, out_dtype=ot), rows, d_out)
    wr, _, _ = orows.unpermute_backward(_f64(d_out), _f64(rows), inv, k, shared)
    assert np.array_equal(_f64(one), wr) if dt == F32 or ot == BF else (np.abs(_f64(one) - wr) <= HALF_BF * np.abs(wr)).all()


@pytest.mark.parametrize("W", [1032, 3584, 4112])
@pytest.mark.parametrize("dt", [BF, F32])
def test_gradients_of_more_pairs(dev, dt, W):
    """On both sides of the pairs from which one wavefront takes a row."""
    test_gradients(dev, 60, 8, 20, 1, 0.1, W, dt, BF)
    test_gradients(dev, 500, 8, 20, 1, 0.1, W, dt, BF)


def test_gradients_against_differences(dev):
    """The whole way, x -> rows -> (row by row) -> sum, in float32: linear in x
    and in the weights, so that a difference is exact but for its roundings."""
    T, k, E, W = 6, 3, 4, 16
    g, d, al, w, inv = _setup(dev, T, k, E, 1, 5, 0.2)
    x = _rand(g, dev, F32, T, W).requires_grad_()
    w.requires_grad_()
    gain = 0.5 + torch.rand(T * (k + 1), 1, generator=g, device=dev)
    d_out = _rand(g, dev, F32, T, W)
    f = lambda a, b: (ops.moe_unpermute(d, ops.moe_permute(d, a, al) * gain, al, b).double() * d_out.double()).sum()
    f(x, w).backward()
    with torch.no_grad():
        scale = float(sum(ops.moe_permute(d, x, al).double().abs().sum() for _ in range(1))) * float(d_out.abs().max()) * 2
        for leaf, other in ((x, lambda v: f(v, w)), (w, lambda v: f(x, v))):
            for i in range(leaf.numel()):
                e = torch.zeros_like(leaf).view(-1)
                e[i] = 0.5
                diff = float(other(leaf + e.view_as(leaf)) - other(leaf - e.view_as(leaf)))
                assert abs(diff - float(leaf.grad.view(-1)[i])) <= 64 * HALF * scale


def test_expanded_gradients_and_repeated_backward(dev):
    g, d, al, w, inv = _setup(dev, 9, 2, 4, 1)
    x = _rand(g, dev, BF, 9, 64).requires_grad_()
    y = ops.moe_permute(d, x, al)
    y.sum().backward(retain_graph=True)                 # (a gradient of stride 0)
    first = x.grad.clone()
    y.sum().backward()
    assert torch.equal(x.grad, 2 * first) and torch.equal(first, torch.full_like(x, 3.0))
    # a permutation made anew in the same buffers before the backward pass is noticed
    y = ops.moe_permute(d, x, al)
    ops.moe_align(d, torch.zeros(9, 2, dtype=torch.int32, device=dev), al)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_strides_widths_and_refusals(dev):
    g, d, al, w, inv = _setup(dev, 12, 2, 4, 0)
    wide = _rand(g, dev, BF, 12, 96)
    ref = ops.moe_permute(d, wide[:, 16:80].contiguous(), al)
    assert torch.equal(ops.moe_permute(d, wide[:, 16:80], al), ref)          # strided rows
    assert torch.equal(ops.moe_permute(d, wide[:, 16:80].t().contiguous().t(), al), ref)
    odd = torch.empty(24 * 64 + 1, dtype=BF, device=dev)[1:].view(24, 64)    # rows 2 bytes off
    odd.copy_(ref)
    assert torch.equal(ops.moe_unpermute(d, odd, al, w), ops.moe_unpermute(d, ref, al, w))
    assert torch.equal(ops.moe_unpermute(d, ref, al, w.t().contiguous().t()), ops.moe_unpermute(d, ref, al, w))
    x = wide[:, :64].contiguous()
    for bad, frag in ((lambda: ops.moe_permute(d, x[:5], al), "x must be"),
                      (lambda: ops.moe_permute(ops.dims(12, 2, 5, 128, 128), x, al), "alignment"),
                      (lambda: ops.moe_permute(d, x, al, out=x), "out must be"),
                      (lambda: ops.moe_permute(d, x.clone().requires_grad_(), al, out=ref), "no gradient"),
                      (lambda: ops.moe_unpermute(d, ref[:5], al), "rows must be"),
                      (lambda: ops.moe_unpermute(d, ref, al, w[:, :1]), "topk_w"),
                      (lambda: ops.moe_unpermute(d, ref, al, w.to(BF)), "topk_w"),
                      (lambda: ops.moe_unpermute(d, ref, al, w.cpu()), "lives on"),
                      (lambda: ops.moe_unpermute(d, ref, al, w, out=ref), "out must be")):
        with pytest.raises(ValueError, match=frag):
            bad()
    with pytest.raises(_lib.Nvfp4Error, match="width=60"):
        ops.moe_permute(d, wide[:, :60].contiguous(), al)
    with pytest.raises(TypeError):
        ops.moe_permute(d, x.half(), al)
    # no tokens
    d0 = ops.dims(0, 2, 4, 128, 128)
    al0 = ops.moe_align(d0, torch.empty(0, 2, dtype=torch.int32, device=dev))
    rows = ops.moe_permute(d0, x[:0], al0)
    assert rows.shape == (0, 64) and ops.moe_unpermute(d0, rows, al0).shape == (0, 64)


def test_rows_past_two_gigaelements(dev):
    T, k, E, W = 35000, 8, 16, 8192
    ids = torch.arange(T * k, device=dev, dtype=torch.int32).view(T, k) % E
    d = ops.dims(T, k, E, 128, 128)
    al = ops.moe_align(d, ids)
    x = torch.randn(T, W, generator=torch.Generator(device=dev).manual_seed(1), device=dev).to(BF)
    rows = ops.moe_permute(d, x, al)
    assert rows.numel() > 1 << 31
    tok = (al.sorted_pair // k).long()
    for p in (0, T * k // 2, T * k - 500):
        assert torch.equal(rows[p:p + 500], x[tok[p:p + 500]])
    assert torch.equal(ops.moe_unpermute(d, rows, al), (8 * x.float()).to(BF))     # eight equal rows: exact
    w = torch.full((T, k), 0.5, device=dev, requires_grad=True)
    rows.requires_grad_()
    gr, gw = torch.autograd.grad(ops.moe_unpermute(d, rows, al, w), (rows, w), x)
    assert torch.equal(gr[-500:], (0.5 * x.float()).to(BF)[tok[-500:]])
    dots = (x[-100:].double() ** 2).sum(1, keepdim=True).expand(-1, k)
    assert (gw[-100:].double() - dots).abs().max() <= (W / 64 + 8) * HALF * float(dots.max())


def test_as_many_tokens_as_there_can_be(dev):
    T, W = 1 << 24, 8
    d = ops.dims(T, 1, 2, 128, 128)
    al = ops.moe_align(d, torch.arange(T, device=dev, dtype=torch.int32).view(T, 1) % 2)
    x = torch.randn(T, W, generator=torch.Generator(device=dev).manual_seed(1), device=dev).to(BF)
    rows = ops.moe_permute(d, x, al)
    assert torch.equal(rows, x.view(T // 2, 2, W).transpose(0, 1).reshape(T, W))
    w = torch.full((T, 1), 0.5, device=dev, requires_grad=True)
    rows.requires_grad_()
    out = ops.moe_unpermute(d, rows, al, w)
    gr, gw = torch.autograd.grad(out, (rows, w), x)
    assert torch.equal(out, (0.5 * x.float()).to(BF)) and torch.equal(gr, (0.5 * rows.detach().float()).to(BF))
    dots = (x.double() ** 2).sum(1, keepdim=True)
    assert ((gw.double() - dots).abs() <= 8 * HALF * dots).all()


def test_second_derivatives_are_refused(dev):
    g, d, al, w, inv = _setup(dev, 5, 2, 4, 0)
    x = _rand(g, dev, F32, 5, 16).requires_grad_()
    w = w.requires_grad_()
    out = ops.moe_unpermute(d, ops.moe_permute(d, x, al), al, w)
    gx, gw = torch.autograd.grad((out * out).sum(), (x, w), create_graph=True)
    ref = torch.autograd.grad(ops.moe_unpermute(d, ops.moe_permute(d, x, al), al, w), (x, w), 2 * out.detach())
    assert torch.equal(gx, ref[0]) and torch.equal(gw, ref[1])
    with pytest.raises(RuntimeError):                    # (torch finds no way from the gradients to x)
        torch.autograd.grad(gx.sum() + gw.sum(), x, retain_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (gx.sum() + gw.sum()).backward()


def test_other_stream_and_graph_with_gradients(dev):
    T, k, E, W = 50, 4, 8, 264
    g, d, al, w, inv = _setup(dev, T, k, E, 1, 3, 0.2)
    x0 = _rand(g, dev, BF, T, W)
    d_out = _rand(g, dev, BF, T, W)

    def step(x, w):
        rows = ops.moe_permute(d, x, al)
        out = ops.moe_unpermute(d, rows, al, w)
        return (out, *torch.autograd.grad(out, (x, w), d_out))

    ref = step(x0.clone().requires_grad_(), w.clone().requires_grad_())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step(x0.clone().requires_grad_(), w.clone().requires_grad_())
    side.synchronize()
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    # leaves of the graph's own, made before its capture
    xs, ws = x0.clone().requires_grad_(), w.clone().requires_grad_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(xs, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(xs, ws)
    for seed in range(3):
        x1 = _rand(torch.Generator(device=dev).manual_seed(seed), dev, BF, T, W)
        ids = torch.randint(-1, E, (T, k), generator=torch.Generator(device=dev).manual_seed(seed), device=dev,
                            dtype=torch.int32)
        ops.moe_align(d, ids, al)                        # a new permutation in the captured buffers
        with torch.no_grad():
            xs.copy_(x1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step(x1.clone().requires_grad_(), w.clone().requires_grad_())):
            assert torch.equal(a, b)
