"""The router's top-k and its gradient against the float64 oracle.

Choices equal the oracle's.  Bars, counted in roundings of 2^-24 (relative): a weight is
exp(v - m) / sum.  The difference is rounded once (an exponent off by |v - m| 2^-24), exp is off by at most
two, the sum over E <= 1024 adds 16 values in a lane and six levels over the wavefront (22), each with its
own exp's errors, and the division is one more: with X the largest finite |v - m| of the row,
(2 X + 32) 2^-24 of the weight, plus 2^-140 where exp underflows.  The gradient adds a mean of k products
(a product and at most six levels of sums), a difference, a product and the sum over equal ids: 2^-24 times
12 w (|g| + sum |w g|) for each entry, or with renorm=False for p of each expert, and p's own error.
bf16 results are off by 2^-8 of their value more.
"""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
import workloads as W
from oracle import formats as of, router as orr
from helpers import assert_within, bf16_dev, bf16_host, dev, gpu_ready, host

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]

U = 2.0 ** -24


def logits_of(T, E, dtype, seed, ties=True):
    """(device logits, their float32 values); with ties, values on a grid of quarters."""
    v = 3 * W.rng(seed, 1).standard_normal((T, E)).astype(np.float32)
    if ties:
        v[::2] = np.round(v[::2] * 4) / 4
    bits = W.f32_to_bf16_bits(v)
    return (dev(v), v) if dtype == "f32" else (bf16_dev(bits), W.bf16_bits_to_f32(bits))


def spread(v):
    """X of each row; at most 110, as exp(-104) is below the least float32."""
    v = np.asarray(v, np.float64)
    with np.errstate(invalid="ignore"):
        m = np.where(np.isfinite(v), v, -np.inf).max(axis=1, keepdims=True)
        d = np.where(np.isfinite(v) & np.isfinite(m), np.abs(v - m), 0.0)
    return np.minimum(d.max(axis=1, keepdims=True), 110.0)


def check_forward(logits, v, k, renorm):
    ids, w = pmg.moe_router_topk(logits, k, renorm=renorm)
    want_ids, want = orr.topk(v, k, renorm)
    assert np.array_equal(host(ids), want_ids)
    got = host(w).astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert_within(got[ok], want[ok], ((2 * spread(v) + 32) * U * np.abs(want) + 2.0 ** -140)[ok], "weights")
    return ids, w


def check_backward(logits, v, ids, w, g, renorm):
    got = pmg.moe_router_topk_backward(dev(g), ids, w, logits, renorm=renorm)
    assert got.dtype == logits.dtype
    i, wh = host(ids), host(w)
    want = orr.topk_backward(g, i, wh, v, renorm)
    T, E = v.shape
    ok = (i >= 0) & (i < E)
    w64, g64 = np.where(ok, wh, 0).astype(np.float64), np.where(ok, g, 0).astype(np.float64)
    size = np.abs(w64 * g64).sum(1, keepdims=True)
    rows = np.broadcast_to(np.arange(T)[:, None], i.shape)
    bound = np.zeros((T, E))
    if renorm:
        np.add.at(bound, (rows[ok], i[ok]), (12 * U * w64 * (np.abs(g64) + size))[ok])
    else:
        p = orr._softmax(v.astype(np.float64))
        G = np.zeros((T, E))
        np.add.at(G, (rows[ok], i[ok]), np.abs(g64)[ok])
        bound = p * 12 * U * (G + size) + np.abs(want) * (2 * spread(v) + 34) * U
    bound += 2.0 ** -140
    if logits.dtype == torch.bfloat16:
        out = W.bf16_bits_to_f32(bf16_host(got))
        bound = bound * (1 + 2.0 ** -8) + np.abs(want) * 2.0 ** -8
    else:
        out = host(got)
    assert np.array_equal(np.isnan(out), np.isnan(want))
    fine = ~np.isnan(want)
    assert_within(out[fine], want[fine], bound[fine], "dlogits")
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 8, 8), (7, 16, 1), (5, 16, 16), (3, 17, 17), (4, 32, 32), (9, 63, 4), (4, 64, 32), (61, 65, 6),
                                   (130, 128, 8), (33, 129, 32), (17, 250, 3), (9, 256, 8), (11, 257, 7), (5, 512, 32),
                                   (6, 513, 2), (3, 1000, 9), (4, 1024, 32)])
def test_forward_and_backward(T, E, k, dtype):
    print(f"[router] T={T} E={E} k={k} {dtype}", flush=True)
    logits, v = logits_of(T, E, dtype, 21)
    g = W.rng(22, E).standard_normal((T, k)).astype(np.float32)
    for renorm in (True, False):
        ids, w = check_forward(logits, v, k, renorm)
        check_backward(logits, v, ids, w, g, renorm)


@pytest.mark.parametrize("E", [8, 128, 300])
def test_masked_infinite_and_nan_rows(E):
    inf = np.inf
    low = np.finfo(np.float32).min
    v = W.rng(23, E).standard_normal((14, E)).astype(np.float32)
    v[0] = -inf                                   # nothing left
    v[1, 1:] = -inf                               # fewer than k left
    v[2, ::2] = -inf
    v[3, 5] = np.nan
    v[4, [2, 7]] = np.nan                         # two: the lower first
    v[5, 6] = inf
    v[6, [1, 3]] = inf
    v[7] = low                                    # the type's lowest value everywhere: equal weights
    v[8, 1:] = low
    v[9] = 0.0
    v[9, 1::2] = -0.0                             # equal to 0
    v[10] = np.float32(1e-45)                     # subnormal, above both zeros
    v[10, 3] = 0.0
    v[11] = -v[11] * np.float32(1e38)
    v[12, 4] = -np.nan
    v[13, :4] = np.finfo(np.float32).max
    k = 4
    g = W.rng(24, E).standard_normal((14, k)).astype(np.float32)
    for dtype in ("f32", "bf16"):
        if dtype == "f32":
            logits, x = dev(v), v
        else:
            logits = dev(v).bfloat16()
            x = logits.float().cpu().numpy()
        for renorm in (True, False):
            ids, w = check_forward(logits, x, k, renorm)
            check_backward(logits, x, ids, w, g, renorm)


def test_backward_skips_bad_ids_and_adds_equal_ones():
    T, E, k = 6, 20, 5
    logits, v = logits_of(T, E, "f32", 25)
    ids = W.rng(26, 1).integers(0, E, (T, k)).astype(np.int32)
    ids[0] = 7                                    # the same expert in every slot
    ids[1, 2], ids[2, 0], ids[3] = -1, E, -5      # no expert
    w = W.rng(26, 2).random((T, k)).astype(np.float32)
    g = W.rng(26, 3).standard_normal((T, k)).astype(np.float32)
    for renorm in (True, False):
        got = check_backward(logits, v, dev(ids), dev(w), g, renorm)
        if renorm:
            assert not host(got)[3].any()


def test_outputs_given_and_rows_do_not_depend_on_others():
    logits, v = logits_of(257, 128, "f32", 27)
    ids, w = torch.full((257, 8), -9, dtype=torch.int32, device="cuda"), torch.full((257, 8), 9.0, device="cuda")
    a, b = pmg.moe_router_topk(logits, 8, ids=ids, weights=w)
    assert a is ids and b is w
    one_ids, one_w = pmg.moe_router_topk(logits[100:101].clone(), 8)
    assert torch.equal(one_ids[0], ids[100]) and torch.equal(one_w[0], w[100])
    dl = torch.full((257, 128), float("nan"), device="cuda")
    assert pmg.moe_router_topk_backward(w, ids, w, logits, dlogits=dl) is dl and not dl.isnan().any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,k", [(5, 2), (37, 6), (250, 8), (301, 3)])
def test_logits_that_start_anywhere(E, k, dtype):
    """Tokens of a larger batch: views that start at any element."""
    logits, v = logits_of(20, E, dtype, 28)
    g = W.rng(29, E).standard_normal((20, k)).astype(np.float32)
    flat = torch.empty(20 * E + 7, dtype=logits.dtype, device="cuda")
    whole, _ = pmg.moe_router_topk(logits, k)
    for at in (1, 3):
        part = flat[at:at + 19 * E].view(19, E)
        part.copy_(logits[1:])
        for renorm in (True, False):
            ids, w = check_forward(part, v[1:], k, renorm)
            assert torch.equal(ids, whole[1:])
            check_backward(part, v[1:], ids, w, g[1:], renorm)
        dl = torch.full((20 * E + 7,), -7.0, dtype=logits.dtype, device="cuda")
        pmg.moe_router_topk_backward(dev(g)[1:], ids, w, part, dlogits=dl[at:at + 19 * E].view(19, E))
        assert (dl[:at] == -7).all() and (dl[at + 19 * E:] == -7).all() and (dl[at:at + 19 * E] != -7).all()


def test_empty_and_refused():
    ids, w = pmg.moe_router_topk(torch.empty(0, 8, device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    x = torch.zeros(4, 8, device="cuda")
    for k in (0, 9):
        with pytest.raises(pmg.NVFP4Error):
            pmg.moe_router_topk(x, k)
    with pytest.raises(ValueError, match="contiguous"):
        pmg.moe_router_topk(x.t(), 2)
    with pytest.raises(ValueError, match="one row per token"):
        pmg.moe_router_topk_backward(x[:, :2].contiguous(), ids, w, x)
    ids, w = pmg.moe_router_topk(x, 2)
    with pytest.raises(TypeError):
        pmg.moe_router_topk_backward(w, ids, w, x.bfloat16(), dlogits=x)
    with pytest.raises(ValueError, match="holds"):
        pmg.moe_router_topk_backward(w[:3], ids, w, x)
