"""A whole expert block as a model runs it: the router's product, the choice of
experts, the routed experts, and a shared expert as a gated dense layer and a
down projection that adds the routed experts' result in its epilogue.

Each stage is compared with its FP64 definition on the operands that it was
given (so that a later bound needs no allowance for an earlier rounding), and
the captured block with the eager one, bit for bit, on every replay.
"""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_03_amd import ops
from oracle import moe as omoe
from oracle import routing as orr

from parity import check_layer_out, device, to_np
from test_gpu_linear_fused import _check, _weight

pytestmark = pytest.mark.gpu

H, I, E, K = 512, 256, 32, 4
ROUTE = dict(score="sigmoid", groups=4, topk_groups=2, group_score="top2", scale=2.5)


@pytest.fixture(scope="module")
def dev():
    return device()


class Block:
    def __init__(self, dev, T, fmt):
        g = torch.Generator(device=dev).manual_seed(31)
        self.T, self.fmt = T, fmt
        self.wg = 0.05 * torch.randn(E, H, generator=g, device=dev)
        self.bias = 0.02 * (3 * torch.randn(E, generator=g, device=dev)).round()
        self.w13 = 0.05 * torch.randn(E, 2 * I, H, generator=g, device=dev)
        self.w2 = 0.05 * torch.randn(E, H, I, generator=g, device=dev)
        self.up, self.down = _weight(fmt, 2 * I, H, True, 5), _weight(fmt, H, I, False, 6)
        d = ops.dims(T, K, E, H, I, 0)
        if fmt == "mxfp4":
            layer = ops.MxMoELayer(d, ops.quantize_mx_expert_weights(d, self.w13, self.w2), device=dev)
            self.routed = layer.forward
        else:
            layer = ops.MoELayer(d, ops.quantize_expert_weights(d, self.w13, self.w2, keep_canonical=False),
                                 torch.tensor([0.003], device=dev), device=dev)
            self.routed = lambda x, ids, tw, out: layer.forward(x, ids, tw, fmt, out=out)
        self.layer = layer
        f32, bf16 = dict(dtype=torch.float32, device=dev), dict(dtype=torch.bfloat16, device=dev)
        self.z, self.tw = torch.empty(T, E, **f32), torch.empty(T, K, **f32)
        self.ids = torch.empty(T, K, dtype=torch.int32, device=dev)
        self.sum = torch.empty(T, H, **f32)
        self.h, self.out = torch.empty(T, I, **bf16), torch.empty(T, H, **bf16)

    def _dense(self, x, w, **kw):
        return ops.mx_linear(x, w, **kw) if self.fmt == "mxfp4" else ops.linear(x, w, self.fmt, **kw)

    def __call__(self, x):
        ops.gate_logits(x, self.wg, out=self.z)
        ops.route_scored(self.z, K, bias=self.bias, ids=self.ids, weights=self.tw, **ROUTE)
        self.routed(x, self.ids, self.tw, out=self.sum)
        self._dense(x, self.up[0], act="silu", out=self.h)
        return self._dense(self.h, self.down[0], residual=self.sum, out=self.out)


def _x(dev, T, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(T, H, generator=g, device=dev).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["w4a4", "w4a16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 37, 300])
def test_block(dev, T, fmt):
    b, x = Block(dev, T, fmt), _x(dev, T, T)
    out = b(x)
    xf = to_np(x.float()).astype(np.float64)
    wg = to_np(b.wg).astype(np.float64)
    # FP32 accumulation of exact products
    bound = H * 2.0 ** -23 * (np.abs(xf) @ np.abs(wg).T) + 2.0 ** -140
    assert (np.abs(to_np(b.z).astype(np.float64) - xf @ wg.T) <= bound).all()
    ids, w = orr.route_scored(to_np(b.z), K, bias=to_np(b.bias), **ROUTE)
    assert np.array_equal(to_np(b.ids), ids)
    assert (np.abs(to_np(b.tw).astype(np.float64) - w) <= (2.0 ** -24 + 2.0 ** -48) * np.abs(w)).all()
    if fmt == "w4a16":
        ew = omoe.ExpertWeights(lambda e: to_np(b.w13[e]), lambda e: to_np(b.w2[e]))
        ref = omoe.layer(xf, ids, to_np(b.tw), ew, E, I, variant="w4a16")
        check_layer_out(to_np(b.sum).astype(np.float64), ref.out, "routed experts")
    else:
        again = b.routed(x, torch.from_numpy(ids).to(dev), b.tw, out=torch.empty_like(b.sum))
        assert torch.equal(again, b.sum) and float(b.sum.abs().max()) > 0
    _check(fmt, x, b.up, None, "silu", True, None, b.h)
    _check(fmt, b.h, b.down, None, "none", False, b.sum, out)


@pytest.mark.parametrize("fmt", ["w4a4", "w4a16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 70])
def test_block_captured(dev, T, fmt):
    b, x, x2 = Block(dev, T, fmt), _x(dev, T, 3), _x(dev, T, 4)
    first, second = b(x).clone(), b(x2).clone()
    assert not torch.equal(first, second)
    held = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b(held)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b(held)
    for i in range(4):
        held.copy_(x2 if i & 1 else x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out, second if i & 1 else first), f"replay {i}"
        assert torch.equal(b(x2), second)   # eager work between replays
        torch.cuda.synchronize()
