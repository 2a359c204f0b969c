"""Dense NVFP4 linear layer reference: y = x W^T (FP64 NumPy).

Test infrastructure only: imported by tests/, __graft_entry__.smoke() and
bench.py's CPU baseline, never by the product path.

The pages' second workload besides the expert layer is the plain NVFP4
linear layer, timed per GEMM across batch sizes M with NVFP4 activations
(W4A4) against bf16 activations and in-kernel weight dequantisation (W4A16)
(unsloth PR #10417, "Why it matters" and its kernel-selection results).
What is computed follows the expert path's conventions (see oracle/moe.py):

* W4A4: the activations get a dynamic global scale g = fl32(max|x| / 2688)
  and block quantisation (oracle/nvfp4.py); the result is the FP64 product of
  the dequantised activations and dequantised weights, i.e. the FP32
  accumulator times alpha = g * gw taken exactly.
* W4A16: bf16 activations times the dequantised weights.
"""
from __future__ import annotations

import math

import numpy as np

from . import nvfp4


def quantize_weight(w):
    """(codes uint8 [N, K], scales uint8 [N, K/16], gw float32) of FP32 w [N, K]."""
    w = np.asarray(w, dtype=np.float32)
    gw = nvfp4.global_scale(w)
    codes, scales = nvfp4.quantize(w, gw)
    return codes, scales, gw


def linear_w4a4(x, w_codes, w_scales, gw) -> np.ndarray:
    """y [M, N] = Q(x) Q(W)^T with x [M, K] (bf16 values) quantised on the fly."""
    x = np.asarray(x, dtype=np.float64)
    g = nvfp4.global_scale(x)
    codes, scales = nvfp4.quantize(x, g)
    x_hat = nvfp4.dequantize(codes, scales, g)
    w_hat = nvfp4.dequantize(w_codes, w_scales, gw)
    return x_hat @ w_hat.T


def linear_w4a16(x, w_codes, w_scales, gw) -> np.ndarray:
    """y [M, N] = x Q(W)^T with x [M, K] used as given (bf16 values, exact in FP64)."""
    x = np.asarray(x, dtype=np.float64)
    w_hat = nvfp4.dequantize(w_codes, w_scales, gw)
    return x @ w_hat.T


def activation(v, act: str) -> np.ndarray:
    """FP64 activation: none, relu, silu z / (1 + e^-z), gelu z Phi(z),
    gelu_tanh z / (1 + e^-2u) with u = sqrt(2/pi) (z + 0.044715 z^3)."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(over="ignore"):
        if act == "none":
            return v
        if act == "relu":
            return np.maximum(v, 0.0)
        if act == "silu":
            return v / (1.0 + np.exp(-v))
        if act == "gelu":
            return 0.5 * v * np.vectorize(math.erfc, otypes=[np.float64])(-v / math.sqrt(2.0))
        if act == "gelu_tanh":
            return v / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    raise ValueError(act)


def epilogue(v, bias=None, act: str = "none", gated: bool = False, residual=None) -> np.ndarray:
    """FP64 epilogue of a dense layer on its product v [M, N]: bias, then the
    activation, or act(first half) * second half, then the residual."""
    v = np.asarray(v, dtype=np.float64)
    if bias is not None:
        v = v + np.asarray(bias, dtype=np.float64)
    if gated:
        h = v.shape[1] // 2
        y = activation(v[:, :h], act) * v[:, h:]
    else:
        y = activation(v, act)
    return y if residual is None else y + np.asarray(residual, dtype=np.float64)
