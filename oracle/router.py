"""The router's choice and weights, and its gradient.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

The pages take a router as given (their MoE layers route each token to the top experts); the definition
(reading, as ``workloads.route_softmax_topk`` draws it) is: a token's experts are those of its k largest
logits, largest first and equal ones by their number (a NaN counts as the largest); its weights are the
softmax over those k, or the chosen part of the softmax over all experts.  All in float64.
"""
from __future__ import annotations

import numpy as np


def _softmax(v):
    """Along the last axis; zeros where every value is -inf, NaN where one is NaN or +inf."""
    with np.errstate(invalid="ignore"):
        m = v.max(axis=-1, keepdims=True)
        e = np.exp(v - m)
        return np.where(m == -np.inf, 0.0, e / np.where(m == -np.inf, 1.0, e.sum(axis=-1, keepdims=True)))


def topk(logits, k: int, renorm: bool = True):
    """logits [T, E] -> (ids int32 [T, k], w float64 [T, k])."""
    v = np.asarray(logits, np.float64)
    T, E = v.shape
    ids = np.empty((T, k), np.int64)
    for t in range(T):
        order = sorted(range(E), key=lambda e: (not np.isnan(v[t, e]), -v[t, e] if not np.isnan(v[t, e]) else 0.0, e))
        ids[t] = order[:k]
    chosen = np.take_along_axis(v, ids, axis=1)
    w = _softmax(chosen) if renorm else np.take_along_axis(_softmax(v), ids, axis=1)
    return ids.astype(np.int32), w


def topk_backward(dw, ids, w, logits, renorm: bool = True):
    """The gradient [T, E] of the logits from that of the weights; ids outside [0, E) are left out."""
    v = np.asarray(logits, np.float64)
    T, E = v.shape
    ids = np.asarray(ids, np.int64)
    ok = (ids >= 0) & (ids < E)
    w = np.where(ok, np.asarray(w, np.float64), 0.0)
    g = np.where(ok, np.asarray(dw, np.float64), 0.0)
    mean = (w * g).sum(axis=1, keepdims=True)
    out = np.zeros((T, E))
    row = np.broadcast_to(np.arange(T)[:, None], ids.shape)
    np.add.at(out, (row[ok], ids[ok]), (w * (g - mean) if renorm else g)[ok])
    return out if renorm else _softmax(v) * (out - mean)
