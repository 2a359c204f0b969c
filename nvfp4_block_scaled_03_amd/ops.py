"""Thin torch binding over the C ABI: argument marshalling only.

Every step runs in the HIP library; torch provides device memory and the
current stream.  Names follow include/nvfp4_moe.h.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from . import _lib
from ._lib import NVFP4_BF16, NVFP4_F32, NVFP4_I8, Dims, Epilogue, RmsNormArgs, RouteParams, call


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


_DTYPE_CODES = {torch.bfloat16: NVFP4_BF16, torch.float32: NVFP4_F32}


def _dtype_code(t: torch.Tensor) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must live on the GPU")


# Handle of a device's current stream (torch.cuda.current_stream, whose Python
# object alone takes 2.8 us, most of a short call).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _same_device(device: int, *tensors) -> bool:
    """Checks that the tensors (None among them) live on the GPU ``device``;
    whether that is the current device."""
    if device < 0:
        raise ValueError("tensors must live on the GPU")
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"a tensor lives on {t.device}, another on GPU {device}")
    return torch._C._cuda_getDevice() == device


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(cond: bool, what: str):
    if not cond:
        raise ValueError(what)


def dims(T: int, topk: int, E: int, H: int, I: int, shared: int = 0) -> Dims:
    return Dims(T, topk, E, H, I, shared)


# ---------------------------------------------------------------- codec
def global_scale(x: torch.Tensor, batches: int = 1, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """g[b] = fl32(max |x[b]| / 2688) over ``batches`` equal contiguous slices."""
    _need_cuda(x)
    x = x.contiguous()
    n = x.numel() // batches if batches else 0
    g = out if out is not None else torch.empty(batches, dtype=torch.float32, device=x.device)
    lib = _lib.load()
    wsb = lib.nvfp4_global_scale_workspace_size(batches, n)
    ws = torch.zeros(max(wsb, 16), dtype=torch.uint8, device=x.device)
    call("nvfp4_global_scale", _p(x), _dtype_code(x), batches, n, _p(g), _p(ws), wsb, _stream())
    if out is not None:
        _written((out,))
    return g


def quantize(x: torch.Tensor, g: torch.Tensor, rows_per_g: Optional[int] = None,
             q: Optional[torch.Tensor] = None, sf: Optional[torch.Tensor] = None,
             deq: Optional[torch.Tensor] = None):
    """NVFP4-encode the rows of ``x`` [rows, K]: (codes [rows, K/2], scales [rows, K/16]).
    ``deq`` (float16 [rows, K]) optionally receives the exact decoded values."""
    _need_cuda(x, g)
    K = x.shape[-1]
    x2 = x.reshape(-1, K)
    if x2.stride(-1) != 1:
        x2 = x2.contiguous()
    rows = x2.shape[0]
    given = [t for t in (q, sf, deq) if t is not None]
    if q is None:
        q = torch.empty(rows, K // 2, dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty(rows, K // 16, dtype=torch.uint8, device=x.device)
    call("nvfp4_quantize", _p(x2), _dtype_code(x2), rows, K, x2.stride(0), _p(g),
         rows if rows_per_g is None else rows_per_g, _p(q), _p(sf), _p(deq), _stream())
    if given:
        _written(given)
    return q, sf


# ---------------------------------------------------------------- routing
def route_topk(logits: torch.Tensor, k: int):
    _need_cuda(logits)
    logits = logits.contiguous().float()
    T, E = logits.shape
    ids = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    call("moe_route_topk", _p(logits), T, E, k, _p(ids), _p(w), _stream())
    return ids, w


def gate_logits(x: torch.Tensor, wg: torch.Tensor, bias: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The router's product: float32 logits [T, E] = x wg^T (+ bias), x bf16
    [T, H], wg [E, H] bf16 or float32, bias float32 [E]."""
    dev = x.get_device()
    if not _same_device(dev, wg, bias, out):
        with torch.cuda.device(dev):
            return gate_logits(x, wg, bias, out)
    if x.dim() != 2 or wg.dim() != 2 or wg.shape[1] != x.shape[1] or x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16 [T, H] and wg [E, H]")
    T, H = x.shape
    E = wg.shape[0]
    ld, one = x.stride()
    at = x.data_ptr()
    if one != 1 or ld % 8 or ld < H or at % 16:
        x = x.clone(memory_format=torch.contiguous_format)
        at, ld = x.data_ptr(), H
    if bias is not None:
        if bias.shape != (E,) or bias.dtype != torch.float32:
            raise ValueError("bias must be float32 [E]")
        bias = bias.contiguous()
    fresh = out is None
    if fresh:
        out = torch.empty(T, E, dtype=torch.float32, device=x.device)
    elif out.shape != (T, E) or out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be contiguous float32 [T, E]")
    wg = wg.contiguous()
    call("moe_gate", at, ld, wg.data_ptr(), _dtype_code(wg), _ptr(bias), T, E, H, out.data_ptr(),
         _raw_stream(dev))
    if not fresh:
        _written((out,))
    return out


@functools.lru_cache(maxsize=64)
def _route_params(score, groups, topk_groups, group_score, renormalize, scale):
    """The host struct moe_route reads (a function of these values alone)."""
    _need(score in ROUTE_SCORES, f"score must be one of {sorted(ROUTE_SCORES)}")
    _need(group_score in GROUP_SCORES, f"group_score must be one of {sorted(GROUP_SCORES)}")
    return ctypes.pointer(
        RouteParams(ROUTE_SCORES[score], groups, topk_groups, GROUP_SCORES[group_score], int(renormalize), scale))


ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}


def route_scored(logits: torch.Tensor, k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
                 groups: int = 1, topk_groups: int = 1, group_score: str = "max", renormalize: bool = True,
                 scale: float = 1.0, ids: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None):
    """Choice of k experts per token from logits [T, E] (float32 or bf16):
    (ids int32 [T, k], weights float32 [T, k]).  ``score``: "softmax" or
    "sigmoid"; ``bias`` (float32 [E]) moves the choice and not the weights;
    the experts are chosen from the ``topk_groups`` best of ``groups`` groups,
    valued by their largest score ("max") or the sum of their two largest
    ("top2"); the weights are the scores of the chosen, divided by their sum
    with ``renormalize``, times ``scale``.  Experts with a logit or bias of
    -inf or NaN are not available; ids that no expert fills are -1."""
    params = _route_params(score, groups, topk_groups, group_score, renormalize, scale)
    dev = logits.get_device()
    if not _same_device(dev, bias, ids, weights):
        with torch.cuda.device(dev):
            return route_scored(logits, k, score, bias, groups, topk_groups, group_score, renormalize, scale, ids,
                                weights)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    ld, one = logits.stride()
    if one != 1 or ld < E:
        logits = logits.contiguous()
        ld = E
    if bias is not None:
        if bias.shape != (E,) or bias.dtype != torch.float32:
            raise ValueError("bias must be float32 [E]")
        bias = bias.contiguous()
    if ids is None:
        ids = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    elif ids.shape != (T, k) or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be contiguous int32 [T, k]")
    else:
        _written((ids,))
    if weights is None:
        weights = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    elif weights.shape != (T, k) or weights.dtype != torch.float32 or not weights.is_contiguous():
        raise ValueError("weights must be contiguous float32 [T, k]")
    else:
        _written((weights,))
    call("moe_route", params, logits.data_ptr(), _dtype_code(logits), ld, _ptr(bias), T, E, k, ids.data_ptr(),
         weights.data_ptr(), _raw_stream(dev))
    return ids, weights


@dataclasses.dataclass
class Alignment:
    offsets: torch.Tensor
    sorted_pair: torch.Tensor
    inv_pos: torch.Tensor
    plan: torch.Tensor
    workspace: torch.Tensor


# Tells autograd that the library wrote into tensors of the caller (a sequence
# of them), which a graph may have saved.
_written = torch._C._increment_version


def _alignment(d: Dims, al: Optional[Alignment], device) -> Alignment:
    """``al`` to be written anew, or a fresh one."""
    if al is None:
        return alloc_alignment(d, device)
    _written((al.offsets, al.inv_pos, al.sorted_pair))
    return al


def alloc_alignment(d: Dims, device) -> Alignment:
    lib = _lib.load()
    P = d.T * d.topk + d.shared * d.T
    return Alignment(
        offsets=torch.empty(d.E + d.shared + 1, dtype=torch.int32, device=device),
        sorted_pair=torch.empty(max(P, 1), dtype=torch.int32, device=device),
        inv_pos=torch.empty(max(P, 1), dtype=torch.int32, device=device),
        plan=torch.empty(lib.moe_align_plan_size(ctypes.byref(d)) // 4, dtype=torch.int32,
                         device=device),
        workspace=torch.empty(max(lib.moe_align_workspace_size(ctypes.byref(d)), 16),
                              dtype=torch.uint8, device=device))


def moe_align(d: Dims, topk_ids: torch.Tensor, al: Optional[Alignment] = None) -> Alignment:
    _need_cuda(topk_ids)
    al = _alignment(d, al, topk_ids.device)
    call("moe_align", ctypes.byref(d), _p(topk_ids.contiguous()), _p(al.offsets),
         _p(al.sorted_pair), _p(al.inv_pos), _p(al.plan), _p(al.workspace),
         al.workspace.numel(), _stream())
    return al


def route_and_align(d: Dims, logits: torch.Tensor, al: Optional[Alignment] = None):
    """Router (top-k + softmax over the selection) and moe_align in one call:
    (topk_ids int32 [T, topk], topk_w float32 [T, topk], Alignment)."""
    _need_cuda(logits)
    al = _alignment(d, al, logits.device)
    ids = torch.empty(max(d.T, 1), d.topk, dtype=torch.int32, device=logits.device)
    wts = torch.empty(max(d.T, 1), d.topk, dtype=torch.float32, device=logits.device)
    call("moe_route_and_align", ctypes.byref(d), _p(logits.contiguous().float()), _p(ids), _p(wts),
         _p(al.offsets), _p(al.sorted_pair), _p(al.inv_pos), _p(al.plan), _p(al.workspace),
         al.workspace.numel(), _stream())
    return ids[:d.T], wts[:d.T], al


def quantize_and_align(d: Dims, x: torch.Tensor, topk_ids: torch.Tensor, al: Optional[Alignment] = None,
                       deq: Optional[torch.Tensor] = None):
    """Global scale, NVFP4 quantisation and moe_align of bf16 ``x`` [T, H] in
    one call: (g, codes, scales, Alignment); ``deq`` optionally receives the
    exact f16 values."""
    _need_cuda(x, topk_ids)
    al = _alignment(d, al, x.device)
    g = torch.empty(1, dtype=torch.float32, device=x.device)
    q = torch.empty(max(d.T, 1), d.H // 2, dtype=torch.uint8, device=x.device)
    sf = torch.empty(max(d.T, 1), d.H // 16, dtype=torch.uint8, device=x.device)
    wsb = _lib.load().nvfp4_global_scale_workspace_size(1, d.T * d.H)
    gs_ws = torch.zeros(max(wsb, 16), dtype=torch.uint8, device=x.device)
    call("moe_quantize_and_align", ctypes.byref(d), _p(x.contiguous()), _p(g), _p(gs_ws), wsb,
         _p(q), _p(sf), _p(deq), _p(topk_ids.contiguous()), _p(al.offsets), _p(al.sorted_pair),
         _p(al.inv_pos), _p(al.plan), _p(al.workspace), al.workspace.numel(), _stream())
    if deq is not None:
        _written((deq,))
    return g, q, sf, al


def mx_quantize_and_align(d: Dims, x: torch.Tensor, topk_ids: torch.Tensor, al: Optional[Alignment] = None):
    """OCP MXFP4 quantisation and moe_align of bf16 ``x`` [T, H] in one call:
    (codes [T, H/2], E8M0 bytes [T, H/32], Alignment)."""
    _need_cuda(x, topk_ids)
    al = _alignment(d, al, x.device)
    q = torch.empty(max(d.T, 1), d.H // 2, dtype=torch.uint8, device=x.device)
    ex = torch.empty(max(d.T, 1), d.H // 32, dtype=torch.uint8, device=x.device)
    call("moe_mxfp4_quantize_and_align", ctypes.byref(d), _p(x.contiguous()), _p(q), _p(ex),
         _p(topk_ids.contiguous()), _p(al.offsets), _p(al.sorted_pair), _p(al.inv_pos), _p(al.plan),
         _p(al.workspace), al.workspace.numel(), _stream())
    return q, ex, al


def scale_and_align(d: Dims, x: torch.Tensor, topk_ids: torch.Tensor, al: Optional[Alignment] = None):
    """Activation global scale of bf16 ``x`` [T, H] and moe_align in one call: (g, Alignment)."""
    _need_cuda(x, topk_ids)
    al = _alignment(d, al, x.device)
    g = torch.empty(1, dtype=torch.float32, device=x.device)
    wsb = _lib.load().nvfp4_global_scale_workspace_size(1, d.T * d.H)
    gs_ws = torch.zeros(max(wsb, 16), dtype=torch.uint8, device=x.device)
    call("moe_scale_and_align", ctypes.byref(d), _p(x.contiguous()), _p(g), _p(gs_ws), wsb,
         _p(topk_ids.contiguous()), _p(al.offsets), _p(al.sorted_pair), _p(al.inv_pos), _p(al.plan),
         _p(al.workspace), al.workspace.numel(), _stream())
    return g, al, gs_ws


# ---------------------------------------------------------------- weights
def prep_weights(d: Dims, which: int, q: torch.Tensor, sf: torch.Tensor) -> torch.Tensor:
    _need_cuda(q, sf)
    n = _lib.load().nvfp4_prep_weights_size(ctypes.byref(d), which)
    prep = torch.empty(n, dtype=torch.uint8, device=q.device)
    call("nvfp4_prep_weights", ctypes.byref(d), which, _p(q.contiguous()), _p(sf.contiguous()),
         _p(prep), _stream())
    return prep


@dataclasses.dataclass
class ExpertWeights:
    """NVFP4 expert weights of one layer: canonical codes/scales, per-matrix
    global scales, and the library's streaming layout."""
    q13: torch.Tensor    # uint8 [S, 2I, H/2]
    sf13: torch.Tensor   # uint8 [S, 2I, H/16]
    g13: torch.Tensor    # f32 [S]
    q2: torch.Tensor     # uint8 [S, H, I/2]
    sf2: torch.Tensor    # uint8 [S, H, I/16]
    g2: torch.Tensor     # f32 [S]
    prep13: torch.Tensor
    prep2: torch.Tensor


def quantize_expert_weights(d: Dims, w13: torch.Tensor, w2: torch.Tensor,
                            keep_canonical: bool = True) -> ExpertWeights:
    """Quantise FP32 expert weights (w13 [S, 2I, H], w2 [S, H, I]) on the GPU:
    one global scale per expert matrix, then block quantisation and prep."""
    S = d.E + d.shared
    assert w13.shape == (S, 2 * d.I, d.H) and w2.shape == (S, d.H, d.I)
    g13 = global_scale(w13, batches=S)
    q13, sf13 = quantize(w13.reshape(S * 2 * d.I, d.H), g13, rows_per_g=2 * d.I)
    g2 = global_scale(w2, batches=S)
    q2, sf2 = quantize(w2.reshape(S * d.H, d.I), g2, rows_per_g=d.H)
    q13 = q13.view(S, 2 * d.I, d.H // 2)
    sf13 = sf13.view(S, 2 * d.I, d.H // 16)
    q2 = q2.view(S, d.H, d.I // 2)
    sf2 = sf2.view(S, d.H, d.I // 16)
    prep13 = prep_weights(d, 13, q13, sf13)
    prep2 = prep_weights(d, 2, q2, sf2)
    if not keep_canonical:
        empty = torch.empty(0, dtype=torch.uint8, device=w13.device)
        q13 = sf13 = q2 = sf2 = empty
    return ExpertWeights(q13, sf13, g13, q2, sf2, g2, prep13, prep2)


# ---------------------------------------------------------------- GEMMs
def gemm1_w4a4(d: Dims, a1_q, a1_sf, g1, al: Alignment, w: ExpertWeights, g2, a2_q=None, a2_sf=None,
               a1_deq=None, a2_deq=None):
    """GEMM1 + SwiGLU + requantisation.  ``a1_deq`` (the decoded copy from
    ``quantize``) is read instead of the codes when given; ``a2_deq``
    optionally receives the decoded copy of a2."""
    P = d.T * d.topk + d.shared * d.T
    dev = g1.device
    given = [t for t in (a2_q, a2_sf, a2_deq) if t is not None]
    a2_q = a2_q if a2_q is not None else torch.empty(max(P, 1), d.I // 2, dtype=torch.uint8, device=dev)
    a2_sf = a2_sf if a2_sf is not None else torch.empty(max(P, 1), d.I // 16, dtype=torch.uint8, device=dev)
    call("grouped_gemm1_swiglu", ctypes.byref(d), _p(a1_q), _p(a1_sf), _p(a1_deq), _p(g1),
         _p(al.sorted_pair), _p(al.offsets), _p(al.plan), _p(w.prep13), _p(w.g13), _p(g2),
         _p(a2_q), _p(a2_sf), _p(a2_deq), _stream())
    if given:
        _written(given)
    return a2_q, a2_sf


def gemm1_w4a16(d: Dims, x, al: Alignment, w: ExpertWeights, a2=None):
    P = d.T * d.topk + d.shared * d.T
    fresh = a2 is None
    a2 = a2 if a2 is not None else torch.empty(max(P, 1), d.I, dtype=torch.bfloat16, device=x.device)
    call("grouped_gemm1_swiglu_w4a16", ctypes.byref(d), _p(x), _p(al.sorted_pair), _p(al.offsets),
         _p(al.plan), _p(w.prep13), _p(w.g13), _p(a2), _stream())
    if not fresh:
        _written((a2,))
    return a2


def gemm_workspace(d: Dims, device) -> torch.Tensor:
    n = _lib.load().grouped_gemm_workspace_size(ctypes.byref(d))
    return torch.empty(max(n // 4, 4), dtype=torch.float32, device=device)


def gemm2_w4a4(d: Dims, a2_q, a2_sf, g2, al: Alignment, topk_w, w: ExpertWeights,
               out_dtype=torch.bfloat16, out=None, ws=None, a2_deq=None):
    dev = g2.device
    fresh = out is None
    out = out if out is not None else torch.empty(d.T, d.H, dtype=out_dtype, device=dev)
    ws = ws if ws is not None else gemm_workspace(d, dev)
    call("grouped_gemm2_combine", ctypes.byref(d), _p(a2_q), _p(a2_sf), _p(a2_deq), _p(g2),
         _p(al.offsets), _p(al.inv_pos), _p(al.plan), _p(topk_w), _p(w.prep2), _p(w.g2), _p(out),
         _dtype_code(out), _p(ws), ws.numel() * 4, _stream())
    if not fresh:
        _written((out,))
    return out


def gemm2_w4a4_noalloc(d: Dims, a2_q, a2_sf, g2, al: Alignment, topk_w, w: ExpertWeights,
                       out: torch.Tensor, a2_deq=None):
    """grouped_gemm2_combine_noalloc: GEMM2 + combine with the library's
    static scratch instead of a workspace (``out`` is caller-allocated)."""
    call("grouped_gemm2_combine_noalloc", ctypes.byref(d), _p(a2_q), _p(a2_sf), _p(a2_deq), _p(g2),
         _p(al.offsets), _p(al.inv_pos), _p(al.plan), _p(topk_w), _p(w.prep2), _p(w.g2), _p(out),
         _dtype_code(out), _stream())
    _written((out,))
    return out


def gemm2_w4a16(d: Dims, a2, al: Alignment, topk_w, w: ExpertWeights, out_dtype=torch.bfloat16,
                out=None, ws=None):
    dev = a2.device
    fresh = out is None
    out = out if out is not None else torch.empty(d.T, d.H, dtype=out_dtype, device=dev)
    ws = ws if ws is not None else gemm_workspace(d, dev)
    call("grouped_gemm2_combine_w4a16", ctypes.byref(d), _p(a2), _p(al.offsets), _p(al.inv_pos),
         _p(al.plan), _p(topk_w), _p(w.prep2), _p(w.g2), _p(out), _dtype_code(out), _p(ws),
         ws.numel() * 4, _stream())
    if not fresh:
        _written((out,))
    return out


# ---------------------------------------------------------------- dense linear
class LinearWeight:
    """An NVFP4 weight W [N, K] prepared for nvfp4_linear*; ``gated``: rows
    [0, N/2) are a gate projection and [N/2, N) the matching up projection."""

    def __init__(self, prep: torch.Tensor, g: torch.Tensor, N: int, K: int, gated: bool = False):
        self.prep, self.g, self.N, self.K, self.gated = prep, g, N, K, gated


def _gated_dims(N: int, K: int) -> Dims:
    """One expert whose gate/up weights are the gated layer's W [N, K]."""
    _need(N % 256 == 0, f"a gated layer's N={N} must be a multiple of 256")
    return dims(1, 1, 1, K, N // 2, 0)


def prepare_linear_weight(w_q: torch.Tensor, w_sf: torch.Tensor, g: torch.Tensor, gated: bool = False) -> LinearWeight:
    """From canonical NVFP4 (codes [N, K/2], scales [N, K/16], global scale)."""
    N, K = w_q.shape[0], w_q.shape[1] * 2
    d = _gated_dims(N, K) if gated else dims(1, 1, 1, N, K, 0)
    prep = prep_weights(d, 13 if gated else 2, w_q.reshape(1, N, K // 2), w_sf.reshape(1, N, K // 16))
    return LinearWeight(prep, g.reshape(1).float(), N, K, gated)


def quantize_linear_weight(w: torch.Tensor, gated: bool = False) -> LinearWeight:
    """FP32 W [N, K] -> global scale, NVFP4 quantisation on the GPU, prep."""
    g = global_scale(w)
    q, sf = quantize(w.contiguous().float(), g)
    return prepare_linear_weight(q, sf, g, gated)


def linear_workspace(M: int, N: int, K: int, w4a4: bool, device) -> torch.Tensor:
    """Workspace of every ``linear`` of up to M rows with a weight [N, K]."""
    n = _lib.load().nvfp4_linear_workspace_size(M, N, K, int(w4a4))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def _linear_call_workspace(M: int, N: int, K: int, w4a4: bool, fused: bool, device) -> torch.Tensor:
    """Workspace of one ``linear`` alone: what that call demands, with zeros
    where W4A4 counts (its first 512 bytes).  A small one is cleared whole: the
    time is the host's, and taking a slice of it costs 1 us."""
    n = _lib.load().nvfp4_linear_call_workspace_size(M, N, K, int(w4a4), int(fused))
    if w4a4 and n <= 1 << 20:
        return torch.zeros(n, dtype=torch.uint8, device=device)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    if w4a4:
        ws.narrow(0, 0, 512).zero_()
    return ws


ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _rows4(t: torch.Tensor) -> bool:
    """Whether the rows of t [M, n] lie apart and can be read and written
    four elements at a time."""
    return (t.stride(1) == 1 and t.data_ptr() % (4 * t.element_size()) == 0
            and (t.shape[0] <= 1 or (t.stride(0) >= t.shape[1] and t.stride(0) % 4 == 0)))


def _row_stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _linear_fused(name: str, x, w, scale, bias, act, residual, out_dtype, out, ws):
    """The fused call ``name`` after its checks; ``scale``: the weight's
    global scale (NVFP4), or None (MXFP4)."""
    dev = x.get_device()
    if not _same_device(dev, w.prep, scale, bias, residual, out, ws):
        with torch.cuda.device(dev):
            return _linear_fused(name, x, w, scale, bias, act, residual, out_dtype, out, ws)
    N, K = w.N, w.K
    if x.dim() != 2 or x.shape[1] != K or x.dtype != torch.bfloat16:
        raise ValueError(f"x must be bfloat16 [M, {K}]")
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    M, n_out = x.shape[0], N // 2 if w.gated else N
    fresh = out is None
    if fresh:
        out = torch.empty(M, n_out, dtype=out_dtype, device=x.device)
    elif out.shape != (M, n_out) or not _rows4(out):
        raise ValueError(f"out must be [{M}, {n_out}] with rows of consecutive elements, starts and strides "
                         "multiples of 4")
    epi = Epilogue(ACTIVATIONS[act], int(w.gated), ld_out=_row_stride(out))
    if bias is not None:
        if bias.shape != (N,) or bias.dtype != torch.float32:
            raise ValueError(f"bias must be float32 [{N}]")
        bias = bias.contiguous()
        epi.bias = bias.data_ptr()
    if residual is not None:
        if residual.shape != (M, n_out):
            raise ValueError(f"residual must be [{M}, {n_out}]")
        if not _rows4(residual):
            residual = residual.clone(memory_format=torch.contiguous_format)
        epi.residual, epi.residual_dtype = residual.data_ptr(), _dtype_code(residual)
        epi.ld_residual = _row_stride(residual)
    x = x.contiguous()
    weight = (w.prep.data_ptr(),) if scale is None else (w.prep.data_ptr(), scale.data_ptr())
    call(name, x.data_ptr(), M, N, K, *weight, epi, out.data_ptr(), _dtype_code(out), ws.data_ptr(),
         ws.numel() * ws.element_size(), _raw_stream(dev))
    if not fresh:
        _written((out,))
    return out


def linear(x: torch.Tensor, w: LinearWeight, variant: str = "w4a4", out_dtype=torch.bfloat16,
           out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
           bias: Optional[torch.Tensor] = None, act: str = "none",
           residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] = x [M, K] W^T (bf16 x; W4A4 quantises x, W4A16 uses it as is).

    With ``bias`` (float32 [N]), ``act`` (a key of ACTIVATIONS), ``residual``
    (bf16 or float32 [M, N]; it may be ``out``) or a gated weight, the rest of
    the layer runs in the product's epilogue: act(y + bias) + residual, or
    act(gate) * up + residual [M, N/2] with gate, up the halves of y + bias."""
    _need_cuda(x)
    M = x.shape[0]
    w4a4 = variant == "w4a4"
    if bias is not None or act != "none" or residual is not None or w.gated:
        if variant not in ("w4a4", "w4a16"):
            raise ValueError(f"variant {variant!r}: w4a4 or w4a16")
        ws = ws if ws is not None else _linear_call_workspace(M, w.N, w.K, w4a4, True, x.device)
        return _linear_fused("nvfp4_linear_fused" if w4a4 else "nvfp4_linear_w4a16_fused", x, w, w.g, bias, act,
                             residual, out_dtype, out, ws)
    fresh = out is None
    if fresh:
        out = torch.empty(M, w.N, dtype=out_dtype, device=x.device)
    ws = ws if ws is not None else _linear_call_workspace(M, w.N, w.K, w4a4, False, x.device)
    call("nvfp4_linear" if w4a4 else "nvfp4_linear_w4a16", _p(x.contiguous()), M, w.N, w.K, _p(w.prep),
         _p(w.g), _p(out), _dtype_code(out), _p(ws), ws.numel(), _stream())
    if not fresh:
        _written((out,))
    return out


# ---------------------------------------------------------------- OCP MXFP4
def mx_quantize(x: torch.Tensor, q: Optional[torch.Tensor] = None, ex: Optional[torch.Tensor] = None):
    """MXFP4-encode the rows of ``x`` [rows, K]: (codes [rows, K/2], E8M0 bytes [rows, K/32])."""
    _need_cuda(x)
    K = x.shape[-1]
    x2 = x.reshape(-1, K)
    if x2.stride(-1) != 1:
        x2 = x2.contiguous()
    rows = x2.shape[0]
    given = [t for t in (q, ex) if t is not None]
    q = q if q is not None else torch.empty(rows, K // 2, dtype=torch.uint8, device=x.device)
    ex = ex if ex is not None else torch.empty(rows, K // 32, dtype=torch.uint8, device=x.device)
    call("mxfp4_quantize", _p(x2), _dtype_code(x2), rows, K, x2.stride(0), _p(q), _p(ex), _stream())
    if given:
        _written(given)
    return q, ex


class MxLinearWeight:
    """An MXFP4 weight W [N, K] prepared for mxfp4_linear; ``gated`` as for LinearWeight."""

    def __init__(self, prep: torch.Tensor, N: int, K: int, gated: bool = False):
        self.prep, self.N, self.K, self.gated = prep, N, K, gated


def prepare_mx_weight(w_q: torch.Tensor, w_ex: torch.Tensor, gated: bool = False) -> MxLinearWeight:
    """From canonical MXFP4 (codes [N, K/2], exponent bytes [N, K/32])."""
    _need_cuda(w_q, w_ex)
    N, K = w_q.shape[0], w_q.shape[1] * 2
    if gated:
        return MxLinearWeight(prep_mx_expert_weights(_gated_dims(N, K), 13, w_q, w_ex), N, K, True)
    n = _lib.load().mxfp4_prep_weights_size(N, K)
    prep = torch.empty(max(n, 16), dtype=torch.uint8, device=w_q.device)
    call("mxfp4_prep_weights", N, K, _p(w_q.contiguous()), _p(w_ex.contiguous()), _p(prep), _stream())
    return MxLinearWeight(prep, N, K)


def quantize_mx_weight(w: torch.Tensor, gated: bool = False) -> MxLinearWeight:
    """FP32 or bf16 W [N, K] -> MXFP4 quantisation on the GPU, prep."""
    q, ex = mx_quantize(w.contiguous())
    return prepare_mx_weight(q, ex, gated)


def mx_linear_workspace(M: int, N: int, K: int, device) -> torch.Tensor:
    n = _lib.load().mxfp4_linear_workspace_size(M, N, K)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def mx_linear(x: torch.Tensor, w: MxLinearWeight, out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, act: str = "none",
              residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] = Q(x) W^T, x bf16 [M, K] quantised to MXFP4 in the call;
    ``bias``, ``act``, ``residual`` and gated weights as for ``linear``."""
    _need_cuda(x)
    M = x.shape[0]
    if bias is not None or act != "none" or residual is not None or w.gated:
        ws = ws if ws is not None else mx_linear_workspace(M, w.N, w.K, x.device)
        return _linear_fused("mxfp4_linear_fused", x, w, None, bias, act, residual, out_dtype, out, ws)
    fresh = out is None
    if fresh:
        out = torch.empty(M, w.N, dtype=out_dtype, device=x.device)
    ws = ws if ws is not None else mx_linear_workspace(M, w.N, w.K, x.device)
    call("mxfp4_linear", _p(x.contiguous()), M, w.N, w.K, _p(w.prep), _p(out), _dtype_code(out), _p(ws),
         ws.numel(), _stream())
    if not fresh:
        _written((out,))
    return out


# ---------------------------------------------------------------- norm and int8 layers
def _no_tangent(name: str, *tensors):
    """Refuses tensors that carry a tangent of the forward-mode level there is
    (callers look whether there is one): the result would have none."""
    if torch._C._is_fwd_grad_enabled():
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError(f"{name} has no forward-mode derivative: call it with the primal tensors")


def _no_gradient(name: str, *tensors):
    """Refuses a call that autograd would take for a differentiable one."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError(f"{name} has no gradient: call it under torch.no_grad()")
    if forward_ad._current_level >= 0:
        _no_tangent(name, *tensors)


def _rows_at(t: torch.Tensor, unit: int = 8):
    """(address, row stride) of t [rows, n] if its rows lie apart and can be read
    and written ``unit`` elements at a time, else None."""
    rows, n = t.shape
    ld, step = t.stride()
    at = t.data_ptr()
    if rows <= 1:
        ld = n
    return None if step != 1 or at % 16 or ld < n or ld % unit else (at, ld)


class NormOut(NamedTuple):
    """What rms_norm makes; None for what was not asked for."""
    y: Optional[torch.Tensor]   # the norm [T, H]
    h: Optional[torch.Tensor]   # x + residual [T, H], the residual's type
    q: Optional[torch.Tensor]   # int8 codes of the norm [T, H]
    s: Optional[torch.Tensor]   # float32 scales [T]: y = q s to half a step


NORM_OUTPUTS = {"y": (True, False), "int8": (False, True), "both": (True, True)}


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
             outputs: str = "y", out_dtype=torch.bfloat16, y: Optional[torch.Tensor] = None,
             h: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
             s: Optional[torch.Tensor] = None) -> NormOut:
    """Root-mean-square norm of the rows of x [T, H] (+ residual): h = x +
    residual, y = h / sqrt(mean h^2 + eps) * weight.  ``outputs``: "y" (in
    ``out_dtype``), "int8" (codes with a scale per row, as int8_linear takes
    them) or "both".  x, residual and weight bf16 or float32; ``h``, ``y``, ``q``
    and ``s`` take the results (``h`` may be ``residual`` or ``x``, ``y`` may be
    ``x``).  No gradient."""
    if outputs not in NORM_OUTPUTS:
        raise ValueError(f"outputs must be one of {sorted(NORM_OUTPUTS)}")
    dev = x.get_device()
    if not _same_device(dev, weight, residual, y, h, q, s):
        with torch.cuda.device(dev):
            return rms_norm(x, weight, eps, residual, outputs, out_dtype, y, h, q, s)
    _no_gradient("rms_norm", x, weight, residual, y, h, s)
    if x.dim() != 2 or weight.shape != x.shape[1:]:
        raise ValueError("x must be [T, H] and weight [H]")
    T, H = x.shape
    want_y, want_q = NORM_OUTPUTS[outputs]
    at_r = at_h = at_y = (None, 0)
    r_type = y_type = 0
    given = []                 # the caller's tensors that are written
    if residual is not None:
        if residual.shape != (T, H):
            raise ValueError(f"residual must be [{T}, {H}]")
        r_type = _dtype_code(residual)
        if h is None:
            h = torch.empty(T, H, dtype=residual.dtype, device=x.device)
            at_h = h.data_ptr(), H
        elif h.shape != (T, H) or h.dtype != residual.dtype or (at_h := _rows_at(h)) is None:
            raise ValueError(f"h must be [{T}, {H}] in the residual's type, with rows of consecutive elements, 16-byte "
                             "aligned, strides multiples of 8")
        else:
            given.append(h)
        at_r = _rows_at(residual)
        if at_r is None:
            residual = residual.clone(memory_format=torch.contiguous_format)
            at_r = residual.data_ptr(), H
    elif h is not None:
        raise ValueError("h is made only with a residual")
    at_x = _rows_at(x)
    if at_x is None:
        x = x.clone(memory_format=torch.contiguous_format)
        at_x = x.data_ptr(), H
    at_w = weight.data_ptr()
    if at_w % 16 or not weight.is_contiguous():
        weight = weight.clone(memory_format=torch.contiguous_format)
        at_w = weight.data_ptr()
    if want_y:
        if y is None:
            y = torch.empty(T, H, dtype=out_dtype, device=x.device)
            at_y = y.data_ptr(), H
        elif y.shape != (T, H) or (at_y := _rows_at(y)) is None:
            raise ValueError(f"y must be [{T}, {H}] with rows of consecutive elements, 16-byte aligned, strides multiples "
                             "of 8")
        else:
            given.append(y)
        y_type = _dtype_code(y)
    elif y is not None:
        raise ValueError(f"y is not made with outputs={outputs!r}")
    at_q = at_s = None
    if want_q:
        q, s = _int8_rows(T, H, x.device, q, s, given)
        at_q, at_s = q.data_ptr(), s.data_ptr()
    elif q is not None or s is not None:
        raise ValueError(f"q and s are not made with outputs={outputs!r}")
    a = RmsNormArgs(*at_x, *at_r, at_w, *at_h, *at_y, at_q, at_s, _dtype_code(x), r_type, _dtype_code(weight), y_type,
                    eps)
    call("rms_norm", a, T, H, _raw_stream(dev))
    if given:
        _written(given)
    return NormOut(y, h, q, s)


def _int8_rows(T: int, H: int, device, q, s, given: list):
    """q and s, checked or fresh; those of the caller join ``given``."""
    if q is None:
        q = torch.empty(T, H, dtype=torch.int8, device=device)
    elif q.shape != (T, H) or q.dtype != torch.int8 or not q.is_contiguous():
        raise ValueError(f"q must be contiguous int8 [{T}, {H}]")
    else:
        given.append(q)
    if s is None:
        s = torch.empty(T, dtype=torch.float32, device=device)
    elif s.shape != (T,) or s.dtype != torch.float32 or not s.is_contiguous():
        raise ValueError(f"s must be contiguous float32 [{T}]")
    else:
        given.append(s)
    return q, s


def int8_quantize(x: torch.Tensor, q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None):
    """Codes and scales of the rows of x [rows, K] (bf16 or float32): (q int8
    [rows, K], s float32 [rows]), q = 127 x / max|x| to the nearest, ties to even."""
    dev = x.get_device()
    if not _same_device(dev, q, s):
        with torch.cuda.device(dev):
            return int8_quantize(x, q, s)
    _no_gradient("int8_quantize", x, s)
    if x.dim() != 2:
        raise ValueError("x must be [rows, K]")
    rows, K = x.shape
    at = _rows_at(x)
    if at is None:
        x = x.clone(memory_format=torch.contiguous_format)
        at = x.data_ptr(), K
    given = []
    q, s = _int8_rows(rows, K, x.device, q, s, given)
    call("int8_quantize", at[0], _dtype_code(x), rows, K, at[1], q.data_ptr(), s.data_ptr(), _raw_stream(dev))
    if given:
        _written(given)
    return q, s


class Int8LinearWeight:
    """An int8 weight W [N, K] with a scale per row, prepared for int8_linear;
    ``gated`` as for LinearWeight."""

    def __init__(self, prep: torch.Tensor, s: torch.Tensor, N: int, K: int, gated: bool = False):
        self.prep, self.s, self.N, self.K, self.gated = prep, s, N, K, gated


def prepare_int8_weight(q: torch.Tensor, s: torch.Tensor, gated: bool = False) -> Int8LinearWeight:
    """From codes int8 [N, K] and scales float32 [N]."""
    dev = q.get_device()
    if not _same_device(dev, s):
        with torch.cuda.device(dev):
            return prepare_int8_weight(q, s, gated)
    if q.dim() != 2 or q.dtype != torch.int8 or s.shape != q.shape[:1] or s.dtype != torch.float32:
        raise ValueError("q must be int8 [N, K] and s float32 [N]")
    N, K = q.shape
    q = q.contiguous()
    if q.data_ptr() % 16:
        q = q.clone()
    n = _lib.load().int8_prep_weights_size(N, K, int(gated))
    prep = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    call("int8_prep_weights", N, K, int(gated), q.data_ptr(), prep.data_ptr(), _raw_stream(dev))
    return Int8LinearWeight(prep, s.contiguous(), N, K, gated)


def quantize_int8_weight(w: torch.Tensor, gated: bool = False) -> Int8LinearWeight:
    """FP32 or bf16 W [N, K] -> codes with a scale per row on the GPU, prep."""
    q, s = int8_quantize(w.detach())
    return prepare_int8_weight(q, s, gated)


def int8_linear_workspace(M: int, N: int, K: int, device) -> torch.Tensor:
    """Workspace of every ``int8_linear`` of up to M rows with a weight [N, K]
    (beyond K = 32768 of int8 codes, which alone are taken there)."""
    lib = _lib.load()
    n = max(lib.int8_linear_workspace_size(M, N, K, t) for t in (NVFP4_BF16, NVFP4_I8))
    if n == 0 and (M != 0 or lib.int8_prep_weights_size(N, K, 0) == 0):
        raise ValueError(f"int8_linear takes no M={M} N={N} K={K}")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def int8_linear(x: torch.Tensor, w: Int8LinearWeight, s: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                bias: Optional[torch.Tensor] = None, act: str = "none",
                residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] = x W^T in 8 bits: x int8 codes [M, K] with scales ``s`` float32
    [M] (rms_norm's or int8_quantize's), or bf16, quantised in the call;
    ``bias``, ``act``, ``residual`` and gated weights as for ``linear``."""
    dev = x.get_device()
    if not _same_device(dev, w.prep, w.s, s, bias, residual, out, ws):
        with torch.cuda.device(dev):
            return int8_linear(x, w, s, out_dtype, out, ws, bias, act, residual)
    _no_gradient("int8_linear", x, s, w.s, bias, residual, out)
    N, K = w.N, w.K
    if x.dim() != 2 or x.shape[1] != K or x.dtype not in (torch.bfloat16, torch.int8):
        raise ValueError(f"x must be int8 or bfloat16 [M, {K}]")
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}")
    M, n_out = x.shape[0], N // 2 if w.gated else N
    codes = x.dtype == torch.int8
    if codes:
        if s is None or s.shape != (M,) or s.dtype != torch.float32:
            raise ValueError(f"int8 x comes with its scales s, float32 [{M}]")
        s = s.contiguous()
    elif s is not None:
        raise ValueError("scales belong to int8 x")
    at_x = _rows_at(x, 16 if codes else 8)
    if at_x is None or at_x[1] > 1 << 22:
        x = x.clone(memory_format=torch.contiguous_format)
        at_x = x.data_ptr(), K
    fresh = out is None
    if fresh:
        out = torch.empty(M, n_out, dtype=out_dtype, device=x.device)
    elif out.shape != (M, n_out) or not _rows4(out):
        raise ValueError(f"out must be [{M}, {n_out}] with rows of consecutive elements, starts and strides "
                         "multiples of 4")
    epi = Epilogue(ACTIVATIONS[act], int(w.gated), ld_out=_row_stride(out))
    if bias is not None:
        if bias.shape != (N,) or bias.dtype != torch.float32:
            raise ValueError(f"bias must be float32 [{N}]")
        bias = bias.contiguous()
        epi.bias = bias.data_ptr()
    if residual is not None:
        if residual.shape != (M, n_out):
            raise ValueError(f"residual must be [{M}, {n_out}]")
        if not _rows4(residual):
            residual = residual.clone(memory_format=torch.contiguous_format)
        epi.residual, epi.residual_dtype = residual.data_ptr(), _dtype_code(residual)
        epi.ld_residual = _row_stride(residual)
    x_dtype = NVFP4_I8 if codes else NVFP4_BF16
    if ws is None:
        n = _lib.load().int8_linear_workspace_size(M, N, K, x_dtype)
        ws = torch.empty(n, dtype=torch.uint8, device=x.device) if n else None
    call("int8_linear", at_x[0], x_dtype, at_x[1], _ptr(s), M, N, K, w.prep.data_ptr(), w.s.data_ptr(), epi,
         out.data_ptr(), _dtype_code(out), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
         _raw_stream(dev))
    if not fresh:
        _written((out,))
    return out


# ---------------------------------------------------------------- rows by expert
def _pairs(d: Dims) -> int:
    return d.T * (d.topk + d.shared)


def _permute(d: Dims, x, offsets, inv_pos, out):
    T, W = x.shape
    fresh = out is None
    if fresh:
        out = torch.empty(_pairs(d), W, dtype=x.dtype, device=x.device)
    at = _rows_at(x)
    if at is None:
        x = x.clone(memory_format=torch.contiguous_format)
        at = x.data_ptr(), W
    call("moe_permute", d, at[0], _dtype_code(x), W, at[1], offsets.data_ptr(), inv_pos.data_ptr(),
         out.data_ptr(), int(fresh), _raw_stream(x.get_device()))
    if not fresh:
        _written((out,))
    return out


def _unpermute(d: Dims, rows, offsets, inv_pos, topk_w, out, out_dtype):
    W = rows.shape[1]
    fresh = out is None
    if fresh:
        out = torch.empty(d.T, W, dtype=out_dtype or rows.dtype, device=rows.device)
    call("moe_unpermute", d, rows.data_ptr(), _dtype_code(rows), W, offsets.data_ptr(), inv_pos.data_ptr(),
         _ptr(topk_w), out.data_ptr(), _dtype_code(out), _raw_stream(rows.get_device()))
    if not fresh:
        _written((out,))
    return out


def _whole(t: torch.Tensor) -> torch.Tensor:
    """t contiguous and 16-byte aligned."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, d, offsets, inv_pos):
        ctx.d = Dims.from_buffer_copy(d)
        ctx.save_for_backward(offsets, inv_pos)
        return _permute(d, x, offsets, inv_pos, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_rows):
        return _unpermute(ctx.d, _whole(d_rows), *ctx.saved_tensors, None, None, None), None, None, None


class _Unpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, topk_w, d, offsets, inv_pos, out_dtype):
        ctx.d = Dims.from_buffer_copy(d)
        # (the rows enter only the weights' gradient)
        keep = rows if topk_w is not None and ctx.needs_input_grad[1] else None
        ctx.dtype = rows.dtype
        ctx.save_for_backward(keep, topk_w, offsets, inv_pos)
        return _unpermute(d, rows, offsets, inv_pos, topk_w, None, out_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_out):
        rows, topk_w, offsets, inv_pos = ctx.saved_tensors
        d, d_out = ctx.d, _whole(d_out)
        W, dev = d_out.shape[1], d_out.device
        d_rows = torch.empty(_pairs(d), W, dtype=ctx.dtype, device=dev) if ctx.needs_input_grad[0] else None
        d_w = torch.empty(d.T, d.topk, dtype=torch.float32, device=dev) if rows is not None else None
        call("moe_unpermute_backward", d, d_out.data_ptr(), _dtype_code(d_out), _ptr(rows),
             NVFP4_BF16 if ctx.dtype == torch.bfloat16 else NVFP4_F32, W, offsets.data_ptr(), inv_pos.data_ptr(),
             _ptr(topk_w), _ptr(d_rows), _ptr(d_w), 1, _raw_stream(d_out.get_device()))
        return d_rows, d_w, None, None, None, None


def _check_alignment(d: Dims, al: Alignment):
    # (an empty batch keeps one word of inv_pos)
    if al.inv_pos.numel() != max(_pairs(d), 1) or al.offsets.numel() != d.E + d.shared + 1:
        raise ValueError(f"the alignment is not one of {d}")


def moe_permute(d: Dims, x: torch.Tensor, al: Alignment, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows of x [T, width] (bf16 or float32) in the order of their experts: row
    p is that of the token of ``al.sorted_pair[p]``.  ``al``: moe_align's for the
    T, topk, E and shared of ``d`` (whose H plays no part).  Rows behind the last
    kept pair are zeros, in ``out`` [P, width] left as they were.  Differentiable
    in x (without ``out``), once and in reverse mode; a backward pass that is
    captured into a graph needs leaves that no other autograd graph alive has used."""
    dev = x.get_device()
    if not _same_device(dev, al.offsets, al.inv_pos, out):
        with torch.cuda.device(dev):
            return moe_permute(d, x, al, out)
    if x.dim() != 2 or x.shape[0] != d.T:
        raise ValueError(f"x must be [{d.T}, width]")
    _check_alignment(d, al)
    if forward_ad._current_level >= 0:
        _no_tangent("moe_permute", x)
    if out is not None:
        _no_gradient("moe_permute with out", x, out)
        if out.shape != (_pairs(d), x.shape[1]) or out.dtype != x.dtype or not out.is_contiguous() \
                or out.data_ptr() % 16:
            raise ValueError(f"out must be contiguous, 16-byte aligned [{_pairs(d)}, {x.shape[1]}] in the type of x")
    elif x.requires_grad and torch.is_grad_enabled():
        return _Permute.apply(x, d, al.offsets, al.inv_pos)
    return _permute(d, x, al.offsets, al.inv_pos, out)


def moe_unpermute(d: Dims, rows: torch.Tensor, al: Alignment, topk_w: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, out_dtype=None) -> torch.Tensor:
    """Every token's rows summed, [T, width]: out[t] = sum_j topk_w[t, j] row of
    pair (t, j), plus the shared expert's row (FP32, rounded once to
    ``out_dtype``, the rows' type by default).  ``rows`` [P, width] in moe_permute's
    order; without ``topk_w`` (float32 [T, topk]) every weight is 1.  Differentiable
    in rows and topk_w (without ``out``), as moe_permute."""
    dev = rows.get_device()
    if not _same_device(dev, al.offsets, al.inv_pos, topk_w, out):
        with torch.cuda.device(dev):
            return moe_unpermute(d, rows, al, topk_w, out, out_dtype)
    if rows.dim() != 2 or rows.shape[0] != _pairs(d):
        raise ValueError(f"rows must be [{_pairs(d)}, width]")
    _check_alignment(d, al)
    if forward_ad._current_level >= 0:
        _no_tangent("moe_unpermute", rows, topk_w)
    if topk_w is not None:
        if topk_w.shape != (d.T, d.topk) or topk_w.dtype != torch.float32:
            raise ValueError(f"topk_w must be float32 [{d.T}, {d.topk}]")
        topk_w = topk_w.contiguous()
    rows = _whole(rows)
    if out is not None:
        _no_gradient("moe_unpermute with out", rows, topk_w, out)
        if out.shape != (d.T, rows.shape[1]) or not out.is_contiguous() or out.data_ptr() % 16:
            raise ValueError(f"out must be contiguous, 16-byte aligned [{d.T}, {rows.shape[1]}]")
    elif torch.is_grad_enabled() and (rows.requires_grad or (topk_w is not None and topk_w.requires_grad)):
        return _Unpermute.apply(rows, topk_w, d, al.offsets, al.inv_pos, out_dtype)
    return _unpermute(d, rows, al.offsets, al.inv_pos, topk_w, out, out_dtype)


# ---------------------------------------------------------------- MXFP4 layer
@dataclasses.dataclass
class MxExpertWeights:
    """OCP MXFP4 expert weights prepared for the grouped MXFP4 GEMMs."""
    prep13: torch.Tensor
    prep2: torch.Tensor


def prep_mx_expert_weights(d: Dims, which: int, q: torch.Tensor, ex: torch.Tensor) -> torch.Tensor:
    _need_cuda(q, ex)
    n = _lib.load().mxfp4_prep_expert_weights_size(ctypes.byref(d), which)
    prep = torch.empty(n, dtype=torch.uint8, device=q.device)
    call("mxfp4_prep_expert_weights", ctypes.byref(d), which, _p(q.contiguous()), _p(ex.contiguous()),
         _p(prep), _stream())
    return prep


def quantize_mx_expert_weights(d: Dims, w13: torch.Tensor, w2: torch.Tensor) -> MxExpertWeights:
    """FP32 expert weights (w13 [S, 2I, H], w2 [S, H, I]) -> MXFP4 on the GPU -> prep."""
    S = d.E + d.shared
    # mxfp4_quantize takes fewer than 2^31 elements per call: expert groups
    per = max(1, ((1 << 31) - 1) // (2 * d.I * d.H))
    q13 = torch.empty(S * 2 * d.I, d.H // 2, dtype=torch.uint8, device=w13.device)
    e13 = torch.empty(S * 2 * d.I, d.H // 32, dtype=torch.uint8, device=w13.device)
    q2 = torch.empty(S * d.H, d.I // 2, dtype=torch.uint8, device=w13.device)
    e2 = torch.empty(S * d.H, d.I // 32, dtype=torch.uint8, device=w13.device)
    for s0 in range(0, S, per):
        s1 = min(S, s0 + per)
        mx_quantize(w13[s0:s1].reshape(-1, d.H), q=q13[s0 * 2 * d.I:s1 * 2 * d.I], ex=e13[s0 * 2 * d.I:s1 * 2 * d.I])
        mx_quantize(w2[s0:s1].reshape(-1, d.I), q=q2[s0 * d.H:s1 * d.H], ex=e2[s0 * d.H:s1 * d.H])
    return MxExpertWeights(prep_mx_expert_weights(d, 13, q13, e13), prep_mx_expert_weights(d, 2, q2, e2))


PART_ALL, PART_SHORT, PART_TALL, PART_COMBINE = 0, 1, 2, 3


def _side_stream_if_parts(d: Dims, side_stream):
    """The side stream to use, or None when these dims run the GEMMs whole."""
    if side_stream is None or not _lib.load().grouped_gemm_runs_in_parts(ctypes.byref(d)):
        return None
    return side_stream


def _run_gemms(side, gemm1, gemm2, marks=None):
    """GEMM1 then GEMM2 + combine of one layer; ``gemm1(part, stream)`` and
    ``gemm2(part, stream)`` launch one part.  With a side stream, the tall
    experts' part of both GEMMs runs there (each part's GEMM2 reads only the
    rows its GEMM1 wrote) while the short experts' part runs on the current
    stream, which then waits for the side stream and runs the combine.  The
    events make the fork and the join part of a captured graph too."""
    main = torch.cuda.current_stream()
    s = ctypes.c_void_p(main.cuda_stream)
    if side is None:
        gemm1(PART_ALL, s)
        if marks:
            marks[1].record()
        gemm2(PART_ALL, s)
    else:
        side.wait_stream(main)
        ss = ctypes.c_void_p(side.cuda_stream)
        gemm1(PART_TALL, ss)
        gemm2(PART_TALL, ss)
        gemm1(PART_SHORT, s)
        if marks:
            marks[1].record()
        gemm2(PART_SHORT, s)
        main.wait_stream(side)
        gemm2(PART_COMBINE, s)
    if marks:
        marks[2].record()


class MxMoELayer:
    """One OCP MXFP4 expert layer with its intermediates preallocated (a call
    launches kernels only): mxfp4_quantize, moe_align,
    grouped_gemm1_swiglu_mxfp4, grouped_gemm2_combine_mxfp4."""

    def __init__(self, d: Dims, weights: MxExpertWeights, device="cuda", side_stream=None):
        """``side_stream``: a second stream for layers that run their GEMMs
        in two parts (``grouped_gemm_runs_in_parts``): the tall experts' part
        then runs on it beside the short experts' part."""
        self.d, self.w = d, weights
        dev = torch.device(device)
        self.side = _side_stream_if_parts(d, side_stream)
        P = d.T * d.topk + d.shared * d.T
        self.a1_q = torch.empty(max(d.T, 1), d.H // 2, dtype=torch.uint8, device=dev)
        self.a1_e = torch.empty(max(d.T, 1), d.H // 32, dtype=torch.uint8, device=dev)
        self.al = alloc_alignment(d, dev)
        self.a2_q = torch.empty(max(P, 1), d.I // 2, dtype=torch.uint8, device=dev)
        self.a2_e = torch.empty(max(P, 1), d.I // 32, dtype=torch.uint8, device=dev)
        self.ws = gemm_workspace(d, dev)

    def forward(self, x, topk_ids, topk_w, out=None, out_dtype=torch.bfloat16, weights=None, marks=None):
        d, w, s = self.d, weights or self.w, _stream()
        _written((self.al.offsets, self.al.inv_pos, self.al.sorted_pair))
        fresh = out is None
        if fresh:
            out = torch.empty(d.T, d.H, dtype=out_dtype, device=x.device)
        call("moe_mxfp4_quantize_and_align", ctypes.byref(d), _p(x), _p(self.a1_q), _p(self.a1_e), _p(topk_ids),
             _p(self.al.offsets), _p(self.al.sorted_pair), _p(self.al.inv_pos), _p(self.al.plan),
             _p(self.al.workspace), self.al.workspace.numel(), s)
        if marks:
            marks[0].record()
        g1 = lambda part, st: call(
            "grouped_gemm1_swiglu_mxfp4_part", ctypes.byref(d), _p(self.a1_q), _p(self.a1_e),
            _p(self.al.sorted_pair), _p(self.al.offsets), _p(self.al.plan), _p(w.prep13),
            _p(self.a2_q), _p(self.a2_e), part, st)
        g2 = lambda part, st: call(
            "grouped_gemm2_combine_mxfp4_part", ctypes.byref(d), _p(self.a2_q), _p(self.a2_e),
            _p(self.al.offsets), _p(self.al.inv_pos), _p(self.al.plan), _p(topk_w), _p(w.prep2),
            _p(out), _dtype_code(out), _p(self.ws), self.ws.numel() * 4, part, st)
        _run_gemms(self.side, g1, g2, marks)
        if not fresh:
            _written((out,))
        return out

    def gemm1(self, weights=None):
        d, w = self.d, weights or self.w
        call("grouped_gemm1_swiglu_mxfp4", ctypes.byref(d), _p(self.a1_q), _p(self.a1_e),
             _p(self.al.sorted_pair), _p(self.al.offsets), _p(self.al.plan), _p(w.prep13),
             _p(self.a2_q), _p(self.a2_e), _stream())

    def gemm2(self, out, topk_w, weights=None):
        d, w = self.d, weights or self.w
        call("grouped_gemm2_combine_mxfp4", ctypes.byref(d), _p(self.a2_q), _p(self.a2_e),
             _p(self.al.offsets), _p(self.al.inv_pos), _p(self.al.plan), _p(topk_w), _p(w.prep2),
             _p(out), _dtype_code(out), _p(self.ws), self.ws.numel() * 4, _stream())
        _written((out,))


# ---------------------------------------------------------------- the layer
class MoELayer:
    """One NVFP4 expert layer with all intermediates preallocated, so that a
    call launches kernels only (and can be captured in a HIP graph)."""

    def __init__(self, d: Dims, weights: ExpertWeights, g2: torch.Tensor, device="cuda",
                 decoded_copies: Optional[bool] = None, side_stream=None):
        """``decoded_copies``: W4A4 keeps exact f16 copies of a1 and a2 next to
        their codes and the GEMMs read those instead of decoding the codes.
        None (default) asks the library which is faster for these dims (the
        copies pay off for tall tiles, not for decode-sized batches).
        ``side_stream``: as for MxMoELayer (W4A4 splits only with the copies)."""
        self.d = d
        self.w = weights
        self.g2 = g2
        P = d.T * d.topk + d.shared * d.T
        self.P = P
        dev = torch.device(device)
        lib = _lib.load()
        self.g1 = torch.empty(1, dtype=torch.float32, device=dev)
        wsb = lib.nvfp4_global_scale_workspace_size(1, d.T * d.H)
        self.gs_ws = torch.zeros(max(wsb, 16), dtype=torch.uint8, device=dev)  # zero once
        self.gs_ws_bytes = wsb
        self.a1_q = torch.empty(max(d.T, 1), d.H // 2, dtype=torch.uint8, device=dev)
        self.a1_sf = torch.empty(max(d.T, 1), d.H // 16, dtype=torch.uint8, device=dev)
        self.al = alloc_alignment(d, dev)
        self.a2_q = torch.empty(max(P, 1), d.I // 2, dtype=torch.uint8, device=dev)
        self.a2_sf = torch.empty(max(P, 1), d.I // 16, dtype=torch.uint8, device=dev)
        self.a2_bf16 = torch.empty(max(P, 1), d.I, dtype=torch.bfloat16, device=dev)
        self.a1_deq = self.a2_deq = None
        if decoded_copies is None:
            decoded_copies = bool(lib.grouped_gemm_prefers_decoded(ctypes.byref(d)))
        self.decoded_copies = decoded_copies
        if decoded_copies:
            self.a1_deq = torch.empty(max(d.T, 1), d.H, dtype=torch.float16, device=dev)
            self.a2_deq = torch.empty(max(P, 1), d.I, dtype=torch.float16, device=dev)
        self.ws = gemm_workspace(d, dev)
        self.side = _side_stream_if_parts(d, side_stream)

    def _gemm1_w4a4(self, w, s):
        d = self.d
        call("grouped_gemm1_swiglu", ctypes.byref(d), _p(self.a1_q), _p(self.a1_sf), _p(self.a1_deq),
             _p(self.g1), _p(self.al.sorted_pair), _p(self.al.offsets), _p(self.al.plan),
             _p(w.prep13), _p(w.g13), _p(self.g2), _p(self.a2_q), _p(self.a2_sf), _p(self.a2_deq), s)

    def _gemm2_w4a4(self, w, tw, out, s):
        d = self.d
        call("grouped_gemm2_combine", ctypes.byref(d), _p(self.a2_q), _p(self.a2_sf), _p(self.a2_deq),
             _p(self.g2), _p(self.al.offsets), _p(self.al.inv_pos), _p(self.al.plan),
             _p(tw), _p(w.prep2), _p(w.g2), _p(out), _dtype_code(out), _p(self.ws),
             self.ws.numel() * 4, s)

    def gemm1(self, variant: str, weights: Optional[ExpertWeights] = None, x=None):
        """GEMM1 alone on the layer's current buffers (for kernel timing)."""
        d, w, s = self.d, weights or self.w, _stream()
        if variant == "w4a4":
            self._gemm1_w4a4(w, s)
        else:
            call("grouped_gemm1_swiglu_w4a16", ctypes.byref(d), _p(x if x is not None else self.x_last),
                 _p(self.al.sorted_pair), _p(self.al.offsets), _p(self.al.plan), _p(w.prep13),
                 _p(w.g13), _p(self.a2_bf16), s)

    def gemm2(self, variant: str, out, weights: Optional[ExpertWeights] = None, topk_w=None):
        """GEMM2 + combine alone on the layer's current buffers (for kernel timing)."""
        d, w, s = self.d, weights or self.w, _stream()
        tw = topk_w if topk_w is not None else self.tw_last
        if variant == "w4a4":
            self._gemm2_w4a4(w, tw, out, s)
        else:
            call("grouped_gemm2_combine_w4a16", ctypes.byref(d), _p(self.a2_bf16),
                 _p(self.al.offsets), _p(self.al.inv_pos), _p(self.al.plan), _p(tw),
                 _p(w.prep2), _p(w.g2), _p(out), _dtype_code(out), _p(self.ws),
                 self.ws.numel() * 4, s)
        _written((out,))

    def forward(self, x, topk_ids, topk_w, variant: str = "w4a4", out=None,
                out_dtype=torch.bfloat16, weights: Optional[ExpertWeights] = None, marks=None):
        """Run the layer; ``marks`` = three torch.cuda.Events recorded before
        GEMM1, between the GEMMs and after GEMM2 + combine."""
        d, w = self.d, weights or self.w
        self.x_last, self.tw_last = x, topk_w
        _written((self.al.offsets, self.al.inv_pos, self.al.sorted_pair))
        fresh = out is None
        if fresh:
            out = torch.empty(d.T, d.H, dtype=out_dtype, device=x.device)
        s = _stream()
        if variant == "w4a4":
            # Activation global scale, quantisation and the permutation (one
            # launch for decode-sized batches).
            call("moe_quantize_and_align", ctypes.byref(d), _p(x), _p(self.g1), _p(self.gs_ws),
                 self.gs_ws_bytes, _p(self.a1_q), _p(self.a1_sf), _p(self.a1_deq), _p(topk_ids),
                 _p(self.al.offsets), _p(self.al.sorted_pair), _p(self.al.inv_pos), _p(self.al.plan),
                 _p(self.al.workspace), self.al.workspace.numel(), s)
        else:
            call("moe_align", ctypes.byref(d), _p(topk_ids), _p(self.al.offsets),
                 _p(self.al.sorted_pair), _p(self.al.inv_pos), _p(self.al.plan),
                 _p(self.al.workspace), self.al.workspace.numel(), s)
        if marks:
            marks[0].record()
        if variant == "w4a4":
            g1 = lambda part, st: call(
                "grouped_gemm1_swiglu_part", ctypes.byref(d), _p(self.a1_q), _p(self.a1_sf),
                _p(self.a1_deq), _p(self.g1), _p(self.al.sorted_pair), _p(self.al.offsets),
                _p(self.al.plan), _p(w.prep13), _p(w.g13), _p(self.g2), _p(self.a2_q), _p(self.a2_sf),
                _p(self.a2_deq), part, st)
            g2 = lambda part, st: call(
                "grouped_gemm2_combine_part", ctypes.byref(d), _p(self.a2_q), _p(self.a2_sf),
                _p(self.a2_deq), _p(self.g2), _p(self.al.offsets), _p(self.al.inv_pos), _p(self.al.plan),
                _p(topk_w), _p(w.prep2), _p(w.g2), _p(out), _dtype_code(out), _p(self.ws),
                self.ws.numel() * 4, part, st)
            side = self.side if self.decoded_copies else None
        elif variant == "w4a16":
            g1 = lambda part, st: call(
                "grouped_gemm1_swiglu_w4a16_part", ctypes.byref(d), _p(x), _p(self.al.sorted_pair),
                _p(self.al.offsets), _p(self.al.plan), _p(w.prep13), _p(w.g13), _p(self.a2_bf16), part, st)
            g2 = lambda part, st: call(
                "grouped_gemm2_combine_w4a16_part", ctypes.byref(d), _p(self.a2_bf16),
                _p(self.al.offsets), _p(self.al.inv_pos), _p(self.al.plan), _p(topk_w),
                _p(w.prep2), _p(w.g2), _p(out), _dtype_code(out), _p(self.ws),
                self.ws.numel() * 4, part, st)
            side = self.side
        else:
            raise ValueError(variant)
        _run_gemms(side, g1, g2, marks)
        if not fresh:
            _written((out,))
        return out


def calibrate_g2(d: Dims, x, topk_ids, weights: ExpertWeights) -> torch.Tensor:
    """A static intermediate global scale from the GPU path itself: the
    global scale of the W4A16 intermediate (bf16 SwiGLU output) of this
    batch."""
    al = moe_align(d, topk_ids)
    a2 = gemm1_w4a16(d, x, al, weights)
    P = d.T * d.topk + d.shared * d.T
    return global_scale(a2[:P])
