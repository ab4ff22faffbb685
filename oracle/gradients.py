"""The gradients of the combine and of the router weights in the SwiGLU, the gradients' norm and clipping.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

Maps as in ``oracle.permute``; everything in float64.
  * combine: y[t] = sum_s w_i D[row(i)], i = t k + s.  dD[row(i)] = w_i dy[t]; dw_i = <dy[t], D[row(i)]>, 0
    for an entry without a row; rows that no entry names keep what they hold.
  * SwiGLU: h = w silu(g) u per row; dw of the row's entry = sum_j dh_j silu(g_j) u_j.
  * norm: sqrt of the sum of squares over all tensors; clipping multiplies by min(1, max_norm / (norm + 1e-6)),
    with max_norm = inf (the norm alone) by 1 whatever the norm.
"""
from __future__ import annotations

import numpy as np


def combine(D, tk_to_row, k: int, topk_w=None):
    rows = np.asarray(tk_to_row, np.int64).reshape(-1, k)
    D = np.asarray(D, np.float64)
    ok = (rows >= 0) & (rows < rows.size)
    w = np.ones(rows.shape) if topk_w is None else np.asarray(topk_w, np.float64).reshape(rows.shape)
    v = np.where(ok[:, :, None], D[np.where(ok, rows, 0)], 0.0)
    return (w[:, :, None] * v).sum(axis=1)


def combine_backward(dy, D, tk_to_row, k: int, topk_w=None, dD=None):
    """Returns (dD [R, H], dw [T, k]); dD: what rows without an entry hold (zeros)."""
    rows = np.asarray(tk_to_row, np.int64).reshape(-1, k)
    dy, D = np.asarray(dy, np.float64), np.asarray(D, np.float64)
    w = np.ones(rows.shape) if topk_w is None else np.asarray(topk_w, np.float64).reshape(rows.shape)
    out = np.zeros((rows.size, dy.shape[1])) if dD is None else np.array(dD, np.float64)
    dw = np.zeros(rows.shape)
    for t in range(rows.shape[0]):
        for s in range(k):
            r = rows[t, s]
            if 0 <= r < rows.size:
                out[r] = w[t, s] * dy[t]
                dw[t, s] = dy[t] @ D[r]
    return out, dw


def swiglu_weight_grad(gu, dh, row_to_tk, n_rows: int):
    """dw [R_cap] in entry order from the routed rows [0, n_rows)."""
    gu, dh = np.asarray(gu, np.float64), np.asarray(dh, np.float64)
    I = gu.shape[1] // 2
    g, u = gu[:n_rows, :I], gu[:n_rows, I:]
    with np.errstate(over="ignore"):
        per_row = (dh[:n_rows] * (g / (1.0 + np.exp(-g))) * u).sum(axis=1)
    dw = np.zeros(gu.shape[0])
    dw[np.asarray(row_to_tk, np.int64)[:n_rows]] = per_row
    return dw


def norm(tensors) -> float:
    return float(np.sqrt(sum(float((np.asarray(t, np.float64) ** 2).sum()) for t in tensors)))


def clip(tensors, max_norm: float):
    n = norm(tensors)
    if max_norm == np.inf:
        return n, [np.asarray(t, np.float64) for t in tensors]
    with np.errstate(invalid="ignore"):
        c = np.float64(max_norm) / (np.float64(n) + 1e-6)
    c = 1.0 if c >= 1.0 else c
    with np.errstate(invalid="ignore"):
        return n, [np.asarray(t, np.float64) * c for t in tensors]
