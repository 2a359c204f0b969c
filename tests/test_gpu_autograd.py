"""What autograd may take for differentiable in the norm, the int8 layers and
the movement of rows by expert: refused, or noticed."""
import pytest
import torch
from torch.autograd import forward_ad

from nvfp4_block_scaled_03_amd import ops

from parity import device

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dev():
    return device()


class _Calls:
    """Arguments of every operator, and calls with one of them put in."""

    def __init__(self, dev):
        g = torch.Generator(device=dev).manual_seed(1)
        r = lambda *s: torch.randn(*s, generator=g, device=dev)
        T, H, k, E = 6, 64, 2, 4
        ids = torch.randint(0, E, (T, k), generator=g, device=dev, dtype=torch.int32)
        d = ops.dims(T, k, E, 128, 128)
        al = ops.moe_align(d, ids)
        x, weight, res, w8 = r(T, H).to(BF), r(H), r(T, H), r(32, H)
        wq, ws = ops.int8_quantize(w8)
        xq, xs = ops.int8_quantize(x)
        self.tensors = dict(x=x, weight=weight, residual=res, s=xs, w_s=ws, bias=r(32), added=r(T, 32), rows=r(T * k, H),
                            topk_w=r(T, k))
        t = self.tensors
        get = lambda new, name: new.get(name, t[name])
        layer = lambda **n: ops.int8_linear(xq, ops.prepare_int8_weight(wq, get(n, "w_s")), get(n, "s"),
                                            bias=get(n, "bias"), residual=get(n, "added"), out_dtype=F32)
        self.calls = {
            "rms_norm": (lambda **n: ops.rms_norm(get(n, "x"), get(n, "weight"), residual=get(n, "residual")).y,
                         ("x", "weight", "residual")),
            "int8_quantize": (lambda **n: ops.int8_quantize(get(n, "x"))[1], ("x",)),
            "int8_linear": (layer, ("s", "w_s", "bias", "added")),
            "int8_linear of bf16": (lambda **n: ops.int8_linear(get(n, "x"), ops.prepare_int8_weight(wq, ws)), ("x",)),
            "moe_permute": (lambda **n: ops.moe_permute(d, get(n, "x"), al), ("x",)),
            "moe_unpermute": (lambda **n: ops.moe_unpermute(d, get(n, "rows"), al, get(n, "topk_w")), ("rows", "topk_w")),
        }


OPERATORS = ["rms_norm", "int8_quantize", "int8_linear", "int8_linear of bf16", "moe_permute", "moe_unpermute"]


@pytest.mark.parametrize("name", OPERATORS)
def test_forward_mode_derivatives_are_refused(dev, name):
    """A tensor with a tangent: the result would come without one, a derivative of zero."""
    c = _Calls(dev)
    call, names = c.calls[name]
    ref = call()
    with forward_ad.dual_level():
        for arg in names:
            dual = forward_ad.make_dual(c.tensors[arg], torch.ones_like(c.tensors[arg]))
            with pytest.raises(ValueError, match="forward-mode"):
                call(**{arg: dual})
            with torch.no_grad(), pytest.raises(ValueError, match="forward-mode"):    # (tangents live on there)
                call(**{arg: dual})
            assert torch.equal(call(**{arg: forward_ad.unpack_dual(dual).primal}), ref)
        assert torch.equal(call(), ref)


def test_a_jacobian_in_forward_mode_is_refused(dev):
    c = _Calls(dev)
    call, _ = c.calls["moe_permute"]
    with pytest.raises(ValueError, match="forward-mode"):
        torch.autograd.functional.jacobian(lambda x: call(x=x), c.tensors["x"].float(), strategy="forward-mode",
                                           vectorize=True)


@pytest.mark.parametrize("name", OPERATORS[:4])
def test_gradients_that_do_not_exist_are_refused(dev, name):
    c = _Calls(dev)
    call, names = c.calls[name]
    for arg in names:
        leaf = c.tensors[arg].clone().requires_grad_()
        with pytest.raises(ValueError, match="no gradient"):
            call(**{arg: leaf})
        with torch.no_grad():
            call(**{arg: leaf})


def test_results_into_tensors_that_take_gradients_are_refused(dev):
    x, w = torch.randn(4, 64, device=dev), torch.ones(64, device=dev)
    leaf = lambda *s: torch.zeros(*s, device=dev, requires_grad=True)
    q = torch.empty(4, 64, dtype=torch.int8, device=dev)
    w8 = ops.quantize_int8_weight(torch.randn(32, 64, device=dev))
    for bad in (lambda: ops.rms_norm(x, w, y=leaf(4, 64)),
                lambda: ops.rms_norm(x, w, residual=x, h=leaf(4, 64)),
                lambda: ops.rms_norm(x, w, outputs="int8", q=q, s=leaf(4)),
                lambda: ops.int8_quantize(x, s=leaf(4)),
                lambda: ops.int8_linear(x.to(BF), w8, out=leaf(4, 32))):
        with pytest.raises(ValueError, match="no gradient"):
            bad()


def _written_by(dev):
    """(tensors, call that writes into them) for every operator with results of the caller's."""
    g = torch.Generator(device=dev).manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)
    e = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device=dev)
    x, w = r(4, 128), r(128)
    xb = x.to(BF)
    al_d = ops.dims(4, 2, 4, 128, 128)
    al = ops.moe_align(al_d, torch.randint(0, 4, (4, 2), generator=g, device=dev, dtype=torch.int32))
    w8, w8g = ops.quantize_int8_weight(r(64, 128)), ops.quantize_int8_weight(r(64, 128), gated=True)
    w4, w4g = ops.quantize_linear_weight(r(128, 128)), ops.quantize_linear_weight(r(256, 128), gated=True)
    mx, mxg = ops.quantize_mx_weight(r(128, 128)), ops.quantize_mx_weight(r(256, 128), gated=True)
    cases = {}
    y, h, q, s = e(4, 128), e(4, 128), e(4, 128, dt=torch.int8), e(4)
    cases["rms_norm"] = ((y, h, q, s), lambda: ops.rms_norm(x, w, residual=x, outputs="both", y=y, h=h, q=q, s=s))
    x2, r2 = x.clone(), x.clone()
    cases["rms_norm in place"] = ((x2, r2), lambda: ops.rms_norm(x2, w, residual=r2, y=x2, h=r2))
    q2, s2 = e(4, 128, dt=torch.int8), e(4)
    cases["int8_quantize"] = ((q2, s2), lambda: ops.int8_quantize(x, q2, s2))
    o1, o2, o3 = e(4, 64), e(4, 32, dt=BF), e(8, 64)
    cases["int8_linear"] = ((o1,), lambda: ops.int8_linear(xb, w8, out=o1))
    cases["int8_linear gated"] = ((o2,), lambda: ops.int8_linear(xb, w8g, act="silu", out=o2))
    cases["int8_linear, some rows"] = ((o3,), lambda: ops.int8_linear(xb, w8, out=o3[2:6]))
    p1, p2 = e(8, 128), e(4, 128)
    cases["moe_permute"] = ((p1,), lambda: ops.moe_permute(al_d, x, al, out=p1))
    rows = r(8, 128)
    cases["moe_unpermute"] = ((p2,), lambda: ops.moe_unpermute(al_d, rows, al, out=p2))
    l1, l2, l3, l4, l5 = (e(4, 128, dt=BF) for _ in range(5))
    cases["linear"] = ((l1,), lambda: ops.linear(xb, w4, out=l1))
    cases["linear w4a16"] = ((l5,), lambda: ops.linear(xb, w4, "w4a16", out=l5))
    cases["linear gated"] = ((l2,), lambda: ops.linear(xb, w4g, act="silu", out=l2))
    cases["mx_linear"] = ((l3,), lambda: ops.mx_linear(xb, mx, out=l3))
    cases["mx_linear gated"] = ((l4,), lambda: ops.mx_linear(xb, mxg, act="silu", out=l4))
    lo = e(4, 8)
    cases["gate_logits"] = ((lo,), lambda: ops.gate_logits(xb, w.expand(8, 128).contiguous(), out=lo))
    ids, tw = e(4, 2, dt=torch.int32), e(4, 2)
    logits = r(4, 8)
    cases["route_scored"] = ((ids, tw), lambda: ops.route_scored(logits, 2, ids=ids, weights=tw))
    gs = e(1)
    cases["global_scale"] = ((gs,), lambda: ops.global_scale(x, out=gs))
    one = torch.ones(1, device=dev)
    c4, s4, d4 = e(4, 64, dt=torch.uint8), e(4, 8, dt=torch.uint8), e(4, 128, dt=torch.float16)
    cases["quantize"] = ((c4, s4, d4), lambda: ops.quantize(xb, one, q=c4, sf=s4, deq=d4))
    cm, em = e(4, 64, dt=torch.uint8), e(4, 4, dt=torch.uint8)
    cases["mx_quantize"] = ((cm, em), lambda: ops.mx_quantize(xb, cm, em))
    d4b = e(4, 128, dt=torch.float16)
    chosen = torch.randint(0, 4, (4, 2), generator=g, device=dev, dtype=torch.int32)
    share = torch.full((4, 2), 0.5, device=dev)
    cases["quantize_and_align"] = ((d4b,), lambda: ops.quantize_and_align(al_d, xb, chosen, deq=d4b))
    al2 = ops.moe_align(al_d, chosen)
    cases["moe_align"] = ((al2.offsets, al2.inv_pos, al2.sorted_pair), lambda: ops.moe_align(al_d, chosen, al2))
    w13, w2 = r(4, 256, 128), r(4, 128, 128)
    we, wm = ops.quantize_expert_weights(al_d, w13, w2), ops.quantize_mx_expert_weights(al_d, w13, w2)
    layer, mxl = ops.MoELayer(al_d, we, one), ops.MxMoELayer(al_d, wm)
    f1, f2, f3, f4, f5, f6, f7 = (e(4, 128, dt=BF) for _ in range(7))
    cases["MoELayer"] = ((f1,), lambda: layer.forward(xb, chosen, share, out=f1))
    cases["MoELayer w4a16"] = ((f2,), lambda: layer.forward(xb, chosen, share, "w4a16", out=f2))
    cases["MxMoELayer"] = ((f3,), lambda: mxl.forward(xb, chosen, share, out=f3))
    a2 = e(8, 128, dt=BF)
    cases["gemm1_w4a16"] = ((a2,), lambda: ops.gemm1_w4a16(al_d, xb, al2, we, a2=a2))
    filled = ops.gemm1_w4a16(al_d, xb, al2, we)
    cases["gemm2_w4a16"] = ((f4,), lambda: ops.gemm2_w4a16(al_d, filled, al2, share, we, out=f4))
    g1, q1, sf1, al3 = ops.quantize_and_align(al_d, xb, chosen)
    g2 = one
    q2b, sf2b, deq2 = e(8, 64, dt=torch.uint8), e(8, 8, dt=torch.uint8), e(8, 128, dt=torch.float16)
    cases["gemm1_w4a4"] = ((q2b, sf2b, deq2), lambda: ops.gemm1_w4a4(al_d, q1, sf1, g1, al3, we, g2, q2b, sf2b,
                                                                     a2_deq=deq2))
    q2f, sf2f = ops.gemm1_w4a4(al_d, q1, sf1, g1, al3, we, g2)
    cases["gemm2_w4a4"] = ((f5,), lambda: ops.gemm2_w4a4(al_d, q2f, sf2f, g2, al3, share, we, out=f5))
    cases["gemm2_w4a4_noalloc"] = ((f6,), lambda: ops.gemm2_w4a4_noalloc(al_d, q2f, sf2f, g2, al3, share, we, f6))

    def second(o):
        layer.forward(xb, chosen, share, "w4a16")
        layer.gemm2("w4a16", o)

    cases["MoELayer.gemm2"] = ((f7,), lambda: second(f7))
    return cases


WRITERS = ["rms_norm", "rms_norm in place", "int8_quantize", "int8_linear", "int8_linear gated", "int8_linear, some rows",
           "moe_permute", "moe_unpermute", "linear", "linear w4a16", "linear gated", "mx_linear", "mx_linear gated",
           "gate_logits", "route_scored", "global_scale", "quantize", "mx_quantize", "quantize_and_align", "moe_align",
           "MoELayer", "MoELayer w4a16", "MxMoELayer", "gemm1_w4a16", "gemm2_w4a16", "gemm1_w4a4", "gemm2_w4a4",
           "gemm2_w4a4_noalloc", "MoELayer.gemm2"]


@pytest.mark.parametrize("name", WRITERS)
def test_a_saved_tensor_written_over_is_noticed(dev, name):
    """A product saves a tensor, a call writes into it: no gradient from the new values."""
    tensors, call = _written_by(dev)[name]
    for t in tensors:
        if not t.is_floating_point():
            before = t._version
            call()
            assert t._version > before
            continue
        leaf = torch.ones_like(t, requires_grad=True)
        y = leaf * t
        call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
        y = leaf * t                 # (written before it is saved: as ever)
        y.sum().backward()
        assert torch.equal(leaf.grad, t)


def test_rows_saved_by_the_weighted_sum_and_written_over(dev):
    d = ops.dims(5, 2, 4, 128, 128)
    g = torch.Generator(device=dev).manual_seed(3)
    al = ops.moe_align(d, torch.randint(0, 4, (5, 2), generator=g, device=dev, dtype=torch.int32))
    rows, x = torch.randn(10, 64, generator=g, device=dev), torch.randn(5, 64, generator=g, device=dev)
    w = torch.rand(5, 2, generator=g, device=dev, requires_grad=True)
    out = ops.moe_unpermute(d, rows, al, w)
    ops.moe_permute(d, x, al, out=rows)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_inference_tensors_are_written(dev):
    """Tensors made under inference_mode have no versions; a call outside writes them as before."""
    with torch.inference_mode():
        x, w, y = torch.randn(4, 64, device=dev), torch.ones(64, device=dev), torch.empty(4, 64, device=dev)
    with torch.no_grad():
        assert torch.equal(ops.rms_norm(x, w, y=y, out_dtype=F32).y, ops.rms_norm(x.clone(), w.clone(), out_dtype=F32).y)
