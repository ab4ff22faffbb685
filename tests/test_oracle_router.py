"""The oracle's gradients (router, combine, SwiGLU weights, clipping) against central differences of its
forward definitions in float64, and its router against the workloads' own."""
import numpy as np
import pytest

import workloads as W
from oracle import gradients as og, permute as op, router as orr, swiglu as os_

EPS = 1e-5   # central differences of smooth functions of order 1: error about EPS^2 + 2^-52 / EPS < 1e-9


def differences(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += EPS
        b[i] -= EPS
        g[i] = (f(a) - f(b)) / (2 * EPS)
    return g


def test_router_agrees_with_the_workloads():
    logits = W.router_logits(37, 24, 5)
    logits[3, 5] = logits[3, 9] = 4.0                       # a tie: the lower expert first
    ids, w = W.route_softmax_topk(logits, 6)
    got_ids, got_w = orr.topk(logits, 6)
    assert np.array_equal(got_ids, ids)
    assert np.allclose(got_w, w, rtol=2.0 ** -23, atol=0)


@pytest.mark.parametrize("renorm", [True, False])
def test_router_gradient_against_differences(renorm):
    rng = np.random.default_rng(1)
    v, g = rng.standard_normal((3, 9)), rng.standard_normal((3, 4))
    ids, w = orr.topk(v, 4, renorm)

    def loss(x):    # the choice is piecewise constant: the same experts
        i, y = orr.topk(x, 4, renorm)
        assert np.array_equal(i, ids)
        return float((y * g).sum())

    assert np.abs(differences(loss, v) - orr.topk_backward(g, ids, w, v, renorm)).max() < 1e-8


def test_router_masked_rows():
    inf = np.inf
    v = np.array([[-inf] * 4, [0.0, -inf, -inf, -inf], [1.0, np.nan, 2.0, 0.0], [1.0, inf, 2.0, 0.0], [0.0, -0.0, 0.0, -inf]])
    for renorm in (True, False):
        ids, w = orr.topk(v, 2, renorm)
        assert ids.tolist() == [[0, 1], [0, 1], [1, 2], [1, 2], [0, 1]]
        assert w[0].tolist() == [0, 0] and w[1].tolist() == [1, 0]
        assert np.isnan(w[2]).all() and np.isnan(w[3]).all()


@pytest.mark.parametrize("weighted", [True, False])
def test_combine_gradient_against_differences(weighted):
    rng = np.random.default_rng(2)
    T, k, E, H = 3, 3, 4, 5
    ids = np.array([[0, 3, 1], [-1, 2, 0], [3, 7, 2]])      # two entries without a row
    _, _, t2r, bad = op.permute(ids, E)
    assert bad == 2
    D, w, dy = rng.standard_normal((T * k, H)), rng.random((T, k)), rng.standard_normal((T, H))
    tw = w if weighted else None
    dD, dw = og.combine_backward(dy, D, t2r, k, tw)
    f = lambda d, x: float((og.combine(d, t2r, k, x) * dy).sum())
    assert np.abs(differences(lambda d: f(d, tw), D) - dD).max() < 1e-8
    if weighted:
        assert np.abs(differences(lambda x: f(D, x), w) - dw).max() < 1e-8
    assert dw[1, 0] == dw[2, 1] == 0


def test_swiglu_weight_gradient_against_differences():
    rng = np.random.default_rng(3)
    R, I = 6, 5
    gu, dh = rng.standard_normal((R, 2 * I)), rng.standard_normal((R, I))
    r2t = np.array([3, 0, 5, 1, -1, -1])                    # four routed rows
    w = rng.random(R)
    gu32 = gu.astype(np.float32)

    def loss(x):
        return float((os_.swiglu_h64(gu32[:4], None) * x[r2t[:4], None] * dh[:4]).sum())

    assert np.abs(differences(loss, w) - og.swiglu_weight_grad(gu32, dh, r2t, 4)).max() < 1e-8


def test_clip():
    rng = np.random.default_rng(4)
    ts = [rng.standard_normal(n) for n in (1, 0, 7, 100)]
    whole = np.concatenate(ts)
    n, out = og.clip(ts, 0.5)
    assert abs(n - np.linalg.norm(whole)) < 1e-12
    assert abs(np.linalg.norm(np.concatenate(out)) - 0.5 * n / (n + 1e-6)) < 1e-12
    assert all(np.array_equal(a, b) for a, b in zip(og.clip(ts, 1e9)[1], ts))
    assert all(not o.any() for o in og.clip(ts, 0.0)[1])
    assert og.clip([], 1.0) == (0.0, [])
