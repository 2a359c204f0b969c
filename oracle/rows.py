"""Reference (FP64 NumPy) of the norm, 8-bit rows, dense int8 layers and the
movement of rows by expert, from their definitions in include/nvfp4_moe.h.

Test infrastructure only: imported by tests/, never by the product path.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def quantize(v):
    """(codes, max|v|) of the rows of v: 127 v / max|v| to the nearest whole
    number, ties to the even one."""
    v = np.asarray(v, dtype=np.float64)
    top = np.abs(v).max(axis=1)
    safe = np.where(top > 0, top, 1.0)[:, None]
    with np.errstate(invalid="ignore"):
        t = 127.0 * v / safe
        q = np.rint(t).astype(np.int64)
        # (t is off by 2^-45 at most: next to a half the rational quotient decides)
        near = np.argwhere(np.abs(np.abs(t - np.trunc(t)) - 0.5) < 2.0 ** -40)
    for r, c in near:
        q[r, c] = round(127 * Fraction(v[r, c]) / Fraction(top[r]))
    return q, top


def int8_quantize(x):
    """(codes int64 [rows, K], scales float64 [rows])"""
    q, top = quantize(x)
    return q, top / 127.0


def rms_norm(h, w, eps):
    """(y, codes, scales) of rows h [T, H] (the sum with the residual, as stored)."""
    h, w = np.asarray(h, dtype=np.float64), np.asarray(w, dtype=np.float64)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
        q, top = quantize(h * w)
        return h * rstd[:, None] * w, q, rstd * top / 127.0


def int8_product(xq, sx, wq, sw):
    """Exact sums times the scales."""
    acc = np.asarray(xq, dtype=np.float64) @ np.asarray(wq, dtype=np.float64).T
    return acc * np.asarray(sx, dtype=np.float64)[:, None] * np.asarray(sw, dtype=np.float64)[None, :]


def align(ids, E, shared):
    """(offsets, inv_pos) of moe_align, from its definition, pair by pair."""
    T, k = ids.shape
    expert = [int(e) if 0 <= e < E else -1 for e in ids.reshape(-1)] + [E] * (T if shared else 0)
    offsets, inv = [0], np.full(len(expert), -1, dtype=np.int64)
    for e in range(E + shared):
        for f, have in enumerate(expert):
            if have == e:
                inv[f] = offsets[-1] + sum(1 for g in range(f) if expert[g] == e)
        offsets.append(offsets[-1] + sum(1 for have in expert if have == e))
    return np.array(offsets), inv


def _pairs(T, k, shared):
    """(token, weight's column or -1) of every pair"""
    return [(f // k, f % k) for f in range(T * k)] + [(t, -1) for t in range(T if shared else 0)]


def permute(x, inv, k, shared, rows):
    """``rows`` [P, W] with the rows of kept pairs put in."""
    out = np.array(rows, dtype=np.float64)
    for (t, _), p in zip(_pairs(x.shape[0], k, shared), inv):
        if p >= 0:
            out[p] = x[t]
    return out


def unpermute(rows, inv, T, k, shared, w=None):
    """(sums, sums of magnitudes)"""
    out, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for (t, j), p in zip(_pairs(T, k, shared), inv):
        if p >= 0:
            v = rows[p] * (1.0 if w is None or j < 0 else float(w[t, j]))
            out[t] += v
            mag[t] += np.abs(v)
    return out, mag


def unpermute_backward(d_out, rows, inv, k, shared, w=None):
    """(d_rows, d_w, sums of magnitudes of d_w)"""
    T = d_out.shape[0]
    d_rows, d_w, mag = np.zeros(rows.shape), np.zeros((T, k)), np.zeros((T, k))
    for (t, j), p in zip(_pairs(T, k, shared), inv):
        if p >= 0:
            d_rows[p] = d_out[t] * (1.0 if w is None or j < 0 else float(w[t, j]))
            if j >= 0:
                d_w[t, j] = d_out[t] @ rows[p]
                mag[t, j] = np.abs(d_out[t]) @ np.abs(rows[p])
    return d_rows, d_w, mag
