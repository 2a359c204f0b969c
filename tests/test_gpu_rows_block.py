"""Norm, router, rows by expert, experts, weighted sum and an 8-bit shared
expert together, as one layer uses them: against the same layer in FP64 from the
framework's own codes and choices, eager and captured, with the routed experts
of the framework's own layer beside it."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_03_amd import ops
from oracle import linear as olin
from oracle import rows as orows

from parity import device, to_np

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    return device()


def _f64(t):
    return to_np(t.detach().float()).astype(np.float64)


class _Layer:
    def __init__(self, dev, T, H, I, E, k, seed=1):
        g = torch.Generator(device=dev).manual_seed(seed)
        r = lambda *s, c=1.0: c * torch.randn(*s, generator=g, device=dev)
        self.d = ops.dims(T, k, E, H, I)
        self.k, self.E = k, E
        self.norm_w = (1 + 0.2 * r(H)).to(BF)
        self.gate = r(E, H, c=0.05)
        self.experts = [ops.quantize_int8_weight(r(H, H, c=0.05)) for _ in range(E)]
        self.up_w, self.down_w = r(2 * I, H, c=0.05), r(H, I, c=0.05)
        self.up, self.down = ops.quantize_int8_weight(self.up_w, gated=True), ops.quantize_int8_weight(self.down_w)
        self.x, self.res = r(T, H).to(BF), r(T, H, c=3.0).to(BF)

    def route(self, y):
        return ops.route_scored(ops.gate_logits(y, self.gate), self.k, score="sigmoid")

    def shared(self, n, out):
        h = ops.int8_linear(n.q, self.up, n.s, act="silu")
        return ops.int8_linear(h, self.down, residual=out)

    def forward(self):
        n = ops.rms_norm(self.x, self.norm_w, residual=self.res, outputs="both")
        ids, w = self.route(n.y)
        al = ops.moe_align(self.d, ids)
        rows = ops.moe_permute(self.d, n.y, al)
        return n, ids, w, al, rows, self.shared(n, ops.moe_unpermute(self.d, rows, al, w))


def test_block_against_fp64(dev):
    T, H, I, E, k = 45, 256, 128, 8, 2
    L = _Layer(dev, T, H, I, E, k)
    n, ids, w, al, rows, out = L.forward()
    # the routed part is the token's own norm times the sum of its weights
    y = _f64(n.y)
    routed = y * _f64(w).sum(1, keepdims=True)
    uq, us = ops.int8_quantize(L.up_w)
    dq, ds = ops.int8_quantize(L.down_w)
    h = olin.epilogue(orows.int8_product(to_np(n.q), to_np(n.s), to_np(uq), to_np(us)), None, "silu", True, None)
    got_h = ops.int8_linear(n.q, L.up, n.s, act="silu")
    # bf16 h: half a step and the FP32 error in front of it
    assert (np.abs(_f64(got_h) - h) <= 2.0 ** -7 * np.abs(h) + 2.0 ** -16).all()
    hq, hs = ops.int8_quantize(got_h)
    want = orows.int8_product(to_np(hq), to_np(hs), to_np(dq), to_np(ds)) + routed
    # two bf16 roundings: the routed sum's and the output's
    bound = 2.0 ** -8 * (np.abs(routed) + np.abs(want)) * 1.01 + 2.0 ** -18 * (np.abs(want) + np.abs(routed) + 1)
    assert (np.abs(_f64(out) - want) <= bound).all()
    # codes stand for the norm to half a step
    top = np.abs(_f64(n.q)).max(1)
    assert (top == 127).all()


def test_experts_by_rows_against_the_grouped_layer_of_eight_bits(dev):
    """Every expert's slice of the sorted rows through int8_linear, and back: the
    same as token by token."""
    T, H, I, E, k = 33, 256, 128, 4, 2
    L = _Layer(dev, T, H, I, E, k)
    n, ids, w, al, rows, _ = L.forward()
    off = to_np(al.offsets)
    done = torch.empty_like(rows)
    for e in range(E):
        ops.int8_linear(rows[off[e]:off[e + 1]], L.experts[e], out=done[off[e]:off[e + 1]])
    out = ops.moe_unpermute(L.d, done, al, w, out_dtype=torch.float32)
    want = torch.zeros(T, H, dtype=torch.float64)
    mag = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            r = ops.int8_linear(n.y[t:t + 1], L.experts[int(ids[t, j])])[0]
            want[t] += (r.double() * w[t, j].double()).cpu()
            mag[t] += (r.double() * w[t, j].double()).abs().cpu()
    assert ((out.double().cpu() - want).abs() <= k * 2.0 ** -24 * mag).all()


def test_captured_block(dev):
    L = _Layer(dev, 64, 256, 128, 8, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.forward()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = L.forward()[-1]
    for seed in range(3):
        g = torch.Generator(device=dev).manual_seed(70 + seed)
        L.x.copy_(torch.randn(64, 256, generator=g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, L.forward()[-1])


def test_training_through_the_rows(dev):
    """Gradients of x, the experts and the router's weights through permute,
    a product per expert and the weighted sum, against the same step by token."""
    T, H, E, k = 21, 64, 4, 2
    g = torch.Generator(device=dev).manual_seed(3)
    ids = torch.randint(0, E, (T, k), generator=g, device=dev, dtype=torch.int32)
    d = ops.dims(T, k, E, 128, 128)
    al = ops.moe_align(d, ids)
    off = to_np(al.offsets)
    leaves = [torch.randn(*s, generator=g, device=dev) for s in ((T, H), (E, H, H), (T, k))]
    d_out = torch.randn(T, H, generator=g, device=dev)
    x, we, w = [v.clone().requires_grad_() for v in leaves]
    rows = ops.moe_permute(d, x, al)
    done = torch.cat([rows[off[e]:off[e + 1]] @ we[e].t() for e in range(E)])
    got = torch.autograd.grad(ops.moe_unpermute(d, done, al, w), (x, we, w), d_out)
    x, we, w = [v.double().cpu().requires_grad_() for v in leaves]
    i = ids.long().cpu()
    y = torch.stack([sum(w[t, j] * (we[i[t, j]] @ x[t]) for j in range(k)) for t in range(T)])
    want = torch.autograd.grad(y, (x, we, w), d_out.double().cpu())
    # sums of at most H + T k + H terms in FP32, magnitudes by the same sums of magnitudes
    xa, wea, wa = [v.double().abs().cpu().requires_grad_() for v in leaves]
    ya = torch.stack([sum(wa[t, j] * (wea[i[t, j]] @ xa[t]) for j in range(k)) for t in range(T)])
    mags = torch.autograd.grad(ya, (xa, wea, wa), d_out.double().abs().cpu())
    for a, b, m in zip(got, want, mags):
        assert ((a.double().cpu() - b).abs() <= (2 * H + T * k) * 2.0 ** -24 * m).all()
