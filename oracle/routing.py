"""Router reference: softmax, top-k, renormalise (test infrastructure only).

The mixture-of-experts layers on the pages route each token to its top-k
experts ("512 routed + 1 shared, 10 routed per token", FlashInfer #2723,
"Model" table).  The pages do not spell out the router; the reading taken here
is the usual one: take the k largest logits (ties to the lower expert id) and
weight them by the softmax over all experts renormalised over the k chosen
ones.  Because the softmax denominator cancels in the renormalisation, the
weights equal the softmax over the k chosen logits alone; ``route_topk`` uses
that closed form and the tests check it against the two-step definition.
"""
from __future__ import annotations

import numpy as np


def route_topk(logits, k: int) -> tuple[np.ndarray, np.ndarray]:
    """Return (ids int32 [T, k], weights float32 [T, k]).

    ``logits`` is FP32 [T, E].  Experts are ordered by decreasing logit, equal
    logits by increasing id.  Weights are computed in FP64 and rounded to FP32.
    """
    z = np.asarray(logits, dtype=np.float32).astype(np.float64)
    T, E = z.shape
    if not 1 <= k <= E:
        raise ValueError("need 1 <= k <= E")
    order = np.argsort(-z, axis=1, kind="stable")      # stable: lower id first on ties
    ids = order[:, :k]
    w = selected_weights_f64(np.take_along_axis(z, ids, axis=1))
    return ids.astype(np.int32), w.astype(np.float32)


def selected_weights_f64(sel) -> np.ndarray:
    """FP64 softmax over the selected logits [T, k] (column 0 the largest):
    exp(z_j - z_0) / sum_i exp(z_i - z_0), the sum taken in the order
    i = 0, 1, ..., k-1 (the order fixes the FP64 rounding of the sum)."""
    sel = np.asarray(sel, dtype=np.float64)
    ex = np.exp(sel - sel[:, :1])
    s = ex[:, 0].copy()
    for j in range(1, ex.shape[1]):
        s = s + ex[:, j]
    return ex / s[:, None]


def fp32_rounding_near_tie(v, rel: float = 2.0 ** -40) -> np.ndarray:
    """True where the FP64 value v lies within ``rel`` (relative) of a point
    halfway between two neighbouring FP32 numbers: there, an FP64 result that
    differs from this one by a few FP64 ulps (another exp implementation) may
    round to the other FP32 neighbour.  For normal FP32 magnitudes only."""
    v = np.abs(np.asarray(v, dtype=np.float64))
    m, e = np.frexp(v)                       # v = m * 2^e, 0.5 <= m < 1
    ulp = np.ldexp(1.0, e - 24)              # FP32 spacing at v
    lo = np.floor(v / ulp) * ulp             # FP32 neighbour below (exact)
    mid = lo + 0.5 * ulp
    return (v > 0) & (np.abs(v - mid) <= rel * v)


def route_two_step(logits, k: int) -> tuple[np.ndarray, np.ndarray]:
    """Definition form: full softmax, pick top-k, divide by their sum (FP64)."""
    z = np.asarray(logits, dtype=np.float32).astype(np.float64)
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p = p / p.sum(axis=1, keepdims=True)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :k]
    sel = np.take_along_axis(p, ids, axis=1)
    return ids.astype(np.int32), (sel / sel.sum(axis=1, keepdims=True))


def gate_logits(x, wg, bias=None) -> np.ndarray:
    """FP64 logits [T, E] = x wg^T (+ bias) of x [T, H] and wg [E, H]."""
    z = np.asarray(x, dtype=np.float64) @ np.asarray(wg, dtype=np.float64).T
    return z if bias is None else z + np.asarray(bias, dtype=np.float64)


def route_scored(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, topk_groups: int = 1,
                 group_score: str = "max", renormalize: bool = True, scale: float = 1.0):
    """Choice of experts with scores, a selection bias and expert groups:
    (ids int32 [T, k], FP64 weights [T, k]), token by token in FP64.

    An expert is available unless its logit or bias is NaN or -inf (+inf is
    the largest finite float).  Scores p are over the available experts; the
    choice values are p + bias, or the logits themselves without a bias (the
    same order); of ``groups`` groups of consecutive experts the
    ``topk_groups`` with the largest value (largest score or sum of the two
    largest, of p or p + bias) remain; the k largest choice values of those
    are chosen, equal values by lower index throughout.  Missing experts:
    id -1, weight 0.
    """
    z = np.asarray(logits).astype(np.float64)
    T, E = z.shape
    top = float(np.finfo(np.float32).max)
    z = np.minimum(np.where(np.isnan(z), -np.inf, z), top)
    b = None if bias is None else np.minimum(np.where(np.isnan(bias), -np.inf, np.asarray(bias, dtype=np.float64)), top)
    ids = np.full((T, k), -1, dtype=np.int32)
    weights = np.zeros((T, k))
    per = E // groups
    for t in range(T):
        on = z[t] > -np.inf
        if b is not None:
            on &= b > -np.inf
        p = np.zeros(E)
        live = z[t] > -np.inf   # a bias keeps an expert from being chosen, not from the softmax
        if score == "softmax":
            if live.any():
                p[live] = np.exp(z[t][live] - z[t][live].max())
                p /= p.sum()
        else:
            with np.errstate(over="ignore"):
                p[live] = 1.0 / (1.0 + np.exp(-z[t][live]))
        valued = np.where(on, p if b is None else p + np.where(on, b, 0.0), -np.inf)
        order_by = valued if b is not None else np.where(on, z[t], -np.inf)
        if groups > 1:
            best = -np.sort(-valued.reshape(groups, per), axis=1)
            v = best[:, 0].copy()
            if group_score == "top2" and per > 1:
                two = best[:, 1] > -np.inf
                v[two] += best[two, 1]
            keep = np.argsort(-v, kind="stable")[:topk_groups]
            order_by = np.where(np.isin(np.arange(E) // per, keep), order_by, -np.inf)
        chosen = [e for e in np.argsort(-order_by, kind="stable")[:k] if order_by[e] > -np.inf]
        ids[t, :len(chosen)] = chosen
        if not chosen:
            continue
        if renormalize and score == "softmax":   # the full softmax's denominator cancels
            w = np.exp(z[t][chosen] - z[t][chosen].max())
        else:
            w = p[chosen]
        if renormalize:
            s = 0.0
            for v in w:
                s += v
            w = w / s if s > 0 else np.zeros_like(w)
        weights[t, :len(chosen)] = w * scale
    return ids, weights
