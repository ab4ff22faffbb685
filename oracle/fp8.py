"""FP8 (E4M3fn) quantisation by blocks of 128, its grouped GEMM, and the BF16 weight gradient.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

A block's scale is s = fl32(amax / 448); a code is E4M3(448 x / amax), the exact
quotient rounded once to nearest with ties to even, the sign kept, and 0 where
s == 0.  Rows have one scale per 128 elements ([blocks][rows]), weights one per
128 x 128 block ([E][N blocks][K blocks]); the last block may be shorter.

The quotient of two float32 numbers is formed in float64.  That decides as the exact
one does: for a midpoint b of the E4M3 grid, 448 x and b amax are integers of at most
29 bits in common units, so an unequal pair differs by 2^-30 or more of either.
"""
from __future__ import annotations

import numpy as np

from . import formats as of

BLOCK = 128
MAX = np.float32(448.0)
REL_TOL = 2e-5


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def encode(x, amax):
    """float32 x, its block's largest magnitude (broadcast) -> E4M3 codes uint8 (finite inputs)."""
    x = np.asarray(x, np.float64)
    live = np.broadcast_to(np.asarray(amax, np.float32) / MAX > 0, x.shape)
    q = 448.0 * np.abs(x) / np.where(live, np.asarray(amax, np.float64), 1.0)
    return np.where(live, of.e4m3_encode_nonneg(np.where(live, q, 0.0)) | (np.signbit(x).astype(np.uint8) << 7),
                    0).astype(np.uint8)


def quantize_rows(x):
    """float32 [rows, K] -> (codes uint8 [rows, K], scales float32 [blocks, rows])."""
    x = np.asarray(x, np.float32)
    rows, K = x.shape
    codes = np.zeros((rows, K), np.uint8)
    scales = np.zeros((blocks(K), rows), np.float32)
    for j in range(blocks(K)):
        b = x[:, j * BLOCK:(j + 1) * BLOCK]
        amax = np.abs(b).max(axis=1)
        scales[j] = amax / MAX
        codes[:, j * BLOCK:(j + 1) * BLOCK] = encode(b, amax[:, None])
    return codes, scales


def quantize_weights(w):
    """float32 [E, N, K] -> (codes uint8 [E, N, K], scales float32 [E, N blocks, K blocks])."""
    w = np.asarray(w, np.float32)
    E, N, K = w.shape
    codes = np.zeros((E, N, K), np.uint8)
    scales = np.zeros((E, blocks(N), blocks(K)), np.float32)
    for i in range(blocks(N)):
        for j in range(blocks(K)):
            at = (slice(None), slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            amax = np.abs(w[at]).max(axis=(1, 2))
            scales[:, i, j] = amax / MAX
            codes[at] = encode(w[at], amax[:, None, None])
    return codes, scales


def dequantize_rows(codes, scales):
    K = codes.shape[1]
    return of.e4m3_decode(codes) * np.repeat(np.asarray(scales, np.float64).T, BLOCK, axis=1)[:, :K]


def dequantize_weight(codes, scales):
    """One matrix: codes [N, K], scales [N blocks, K blocks]."""
    N, K = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), BLOCK, axis=0)[:N], BLOCK, axis=1)[:, :K]
    return of.e4m3_decode(codes) * s


def grouped_gemm_ref(a_codes, a_scales, offsets, w_codes, w_scales, row_source=None, rows=None):
    """C[r] = A[row_source[r]] W_e^T in float64, and the bound 2e-5 sum |a w|.

    `row_source` (None: r itself) is the row of A that routed row r reads; `rows`
    (None: all routed rows) restricts the output."""
    offsets = np.asarray(offsets, np.int64)
    rows = np.arange(int(offsets[-1])) if rows is None else np.asarray(rows, np.int64)
    src = rows if row_source is None else np.asarray(row_source, np.int64)[rows]
    N = w_codes.shape[1]
    C, B = np.zeros((rows.size, N)), np.zeros((rows.size, N))
    expert = np.searchsorted(offsets, rows, side="right") - 1
    for e in np.unique(expert):
        sel = np.nonzero(expert == e)[0]
        a = dequantize_rows(a_codes[src[sel]], a_scales[:, src[sel]])
        w = dequantize_weight(w_codes[e], w_scales[e])
        C[sel] = a @ w.T
        B[sel] = np.abs(a) @ np.abs(w).T
    return C, REL_TOL * B


def swiglu(gu, w=None):
    """float [R, 2I] -> h float64 [R, I] = g / (1 + exp(-g)) * u * w."""
    gu = np.asarray(gu, np.float64)
    g, u = np.split(gu, 2, axis=1)
    with np.errstate(over="ignore"):
        h = g / (1.0 + np.exp(-g)) * u
    return h if w is None else h * np.asarray(w, np.float64)[:, None]


def wgrad_ref(g, x, offsets):
    """Expert-grouped g [R, M], x [R, N] -> (dW float64 [E, M, N], sum |g x| of each element)."""
    offsets = np.asarray(offsets, np.int64)
    E = offsets.size - 1
    g, x = np.asarray(g, np.float64), np.asarray(x, np.float64)
    out = np.zeros((E, g.shape[1], x.shape[1]))
    mag = np.zeros_like(out)
    for e in range(E):
        s = slice(offsets[e], offsets[e + 1])
        out[e] = g[s].T @ x[s]
        mag[e] = np.abs(g[s]).T @ np.abs(x[s])
    return out, mag
