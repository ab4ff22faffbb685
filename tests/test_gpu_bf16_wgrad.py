"""GPU parity: the BF16 expert weight gradient dW_e = g_e^T x_e over ragged experts.

Products of bf16 values are exact in FP32; an element's sum over n rows takes at
most n roundings of half a step, so it is within (n + 1) 2^-24 sum |g x| of the
float64 value, plus half a bf16 step (2^-8 relative) where the output is bf16.
"""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
import workloads as W
from oracle import formats as of, fp8 as o8, permute as op
from helpers import assert_within, bf16_dev, dev, gpu_ready, host

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]


def _check(counts_or_off, M, N, out="f32", r2t=None, k=1, gather=None, T=0, spare=0, seed=1, experts=None):
    off = np.asarray(counts_or_off, np.int32)
    R, E = int(off[-1]), off.size - 1
    rows = {n: T if gather in (n, "both") else R + spare for n in ("g", "x")}
    gb = W.gaussian_bf16((rows["g"], M), 0.5, seed, 1)
    xb = W.activations(rows["x"], N, seed, 2)
    if spare:                                             # rows past the last routed one must never count
        for n, b in (("g", gb), ("x", xb)):
            if gather not in (n, "both"):
                b[R:] = 0x7FC0                            # NaN
    g, x = of.bf16_to_f32(gb), of.bf16_to_f32(xb)
    src = None if r2t is None else r2t.astype(np.int64) // k
    gg, xx = (v[src] if gather in (n, "both") else v[:R] for n, v in (("g", g), ("x", x)))
    dt = torch.float32 if out == "f32" else torch.bfloat16
    kw = {}
    if gather:
        kw = {"row_to_tk": dev(np.concatenate([r2t, np.full(spare, -9, np.int32)])), "k": k, "gather": gather}
    c = torch.full((E, M, N), float("nan"), dtype=dt, device="cuda")
    got = pmg.bf16_grouped_gemm_wgrad(bf16_dev(gb), bf16_dev(xb), dev(off), c=c, **kw)
    assert got is c
    got = got.float().cpu().numpy().astype(np.float64)
    for e in range(E) if experts is None else experts:
        o = np.array([0, off[e + 1] - off[e]])
        s = slice(off[e], off[e + 1])
        ref, mag = (v[0] for v in o8.wgrad_ref(gg[s], xx[s], o))
        bound = (o[1] + 1) * 2.0 ** -24 * mag
        if out == "bf16":
            bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
        assert_within(got[e], ref, bound, f"expert {e} ({o[1]} rows)")
    return c


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)])


@pytest.mark.parametrize("counts", [[0], [1], [0, 1, 0, 2, 31, 32, 33, 0], [64, 65, 96, 127], [300, 5, 0], [1500, 0, 1100]])
@pytest.mark.parametrize("M,N", [(8, 8), (128, 256), (136, 264), (72, 520)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_ragged(counts, M, N, out):
    print(f"[bf16 wgrad] {counts} {M}x{N} {out}", flush=True)
    _check(_offsets(counts), M, N, out, spare=2)


@pytest.mark.parametrize("T,E,k,kind", [(1, 8, 2, "uniform"), (100, 16, 4, "zipf"), (1021, 24, 4, "zipf"), (2100, 2, 1, "zipf")])
@pytest.mark.parametrize("gather", ["g", "x", "both"])
def test_gathered(T, E, k, kind, gather):
    print(f"[bf16 wgrad] T={T} E={E} k={k} {kind} gather={gather}", flush=True)
    ids, _ = W.make_routing(kind, T, E, k, 5)
    off, r2t, _, _ = op.permute(ids, E)
    _check(off, 144, 328, r2t=r2t, k=k, gather=gather, T=T, spare=2)


def test_layer_shape():
    """The layer's gate_up gradient at the training length, on its largest, smallest and two more experts."""
    ids, _ = W.make_routing("softmax", W.TOKENS, W.EXPERTS, W.TOPK, 3)
    off, r2t, _, _ = op.permute(ids, W.EXPERTS)
    n = np.diff(off)
    _check(off, 2 * W.INTER, W.HIDDEN, r2t=r2t, k=W.TOPK, gather="x", T=W.TOKENS,
           experts=[int(n.argmax()), int(n.argmin()), 0, W.EXPERTS - 1])


def test_many_experts():
    r = np.random.default_rng(4)
    _check(_offsets(r.integers(0, 4, 1024)), 24, 40, "bf16")


@pytest.mark.parametrize("counts", [[0, 1, 33, 1024, 1025, 0, 0, 2100, 64, 31, 5, 96, 0, 0, 3, 700],
                                    [1040] + [0] * 200 + [1] * 55, [40] * 4 + [0] + [2060]])
@pytest.mark.parametrize("M,N", [(1016, 1000), (136, 264), (776, 2056)])
@pytest.mark.parametrize("out,gather", [("f32", None), ("f32", "both"), ("bf16", "x"), ("bf16", "g")])
def test_many_tiles(counts, M, N, out, gather):
    """More tiles than CUs, of every kind in one launch: no rows, one, whole K-steps and a row more, more rows
    than are mapped at a time; output sizes that end inside a tile either way."""
    print(f"[bf16 wgrad] {len(counts)} experts {M}x{N} {out} {gather}", flush=True)
    off = _offsets(counts)
    R = int(off[-1])
    r2t = np.random.default_rng(9).permutation(R + 4).astype(np.int32)[:R]   # k = 3: some rows of T come often, some never
    pick = sorted({0, 1, 3, 4, len(counts) - 1, int(np.argmax(counts)), len(counts) // 2})
    _check(off, M, N, out, r2t=r2t, k=3, gather=gather, T=(R + 4 + 2) // 3, spare=3,
           experts=[e for e in pick if e < len(counts)])


@pytest.mark.parametrize("counts,M,N", [([0, 1, 33, 1024, 1025, 0, 2100, 64, 31, 5, 96, 3] * 4, 264, 520),
                                        ([300, 0, 32, 1, 1500, 31, 64, 1057], 1024, 1016)])
@pytest.mark.parametrize("out,gather", [("f32", None), ("f32", "both"), ("bf16", "x"), ("bf16", "g")])
def test_tiles_that_would_pad_or_leave_units_idle(counts, M, N, out, gather):
    """Outputs where 256 x 256 tiles would pad a third more, and where there are half as many of them as CUs."""
    print(f"[bf16 wgrad] {len(counts)} experts {M}x{N} {out} {gather}", flush=True)
    off = _offsets(counts)
    R = int(off[-1])
    r2t = np.random.default_rng(10).permutation(R + 4).astype(np.int32)[:R]
    _check(off, M, N, out, r2t=r2t, k=3, gather=gather, T=(R + 6) // 3, spare=3,
           experts=[e for e in (0, 1, 2, 3, 4, 6, 7, 25, 46) if e < len(counts)])


@pytest.mark.parametrize("E", [2, 5, 7, 8, 9, 13, 16, 23])
@pytest.mark.parametrize("M,N", [(72, 136), (264, 512), (520, 1032)])
def test_any_number_of_experts(E, M, N):
    """Every expert's every tile is written, however the tiles fall on the XCDs."""
    _check(_offsets([(7 * e) % 50 for e in range(E)]), M, N, "f32")


def test_same_sums_for_any_call():
    """A repeated call gives the same bits: no sum depends on the order in which workgroups end."""
    off = dev(_offsets([700, 0, 33, 1500]).astype(np.int32))
    for M, N in ((128, 256), (1024, 256), (2048, 2048)):
        g, x = bf16_dev(W.gaussian_bf16((2233, M), 0.5, 1, 1)), bf16_dev(W.activations(2233, N, 1, 2))
        a = host(pmg.bf16_grouped_gemm_wgrad(g, x, off))
        for _ in range(3):
            assert np.array_equal(a, host(pmg.bf16_grouped_gemm_wgrad(g, x, off)))


def test_infinities_and_nan_stay_in_their_columns():
    """A value next to an expert's last row reaches only what it multiplies: the padding of a K-step adds nothing."""
    off = _offsets([5, 33])
    g, x = np.ones((38, 16), np.float32), np.ones((38, 24), np.float32)
    clean = pmg.bf16_grouped_gemm_wgrad(dev(g).bfloat16(), dev(x).bfloat16(), dev(off.astype(np.int32)))
    x[4, 3], g[37, 2] = np.inf, np.nan
    got = host(pmg.bf16_grouped_gemm_wgrad(dev(g).bfloat16(), dev(x).bfloat16(), dev(off.astype(np.int32))))
    want = host(clean).copy()
    want[0, :, 3], want[1, 2, :] = np.inf, np.nan
    assert np.array_equal(got, want, equal_nan=True)


def test_against_autograd():
    """The gradient torch's autograd gives for y = x W^T per expert (float64), rows gathered through the map."""
    ids, _ = W.make_routing("uniform", 40, 6, 2, 8)
    off, r2t, _, _ = op.permute(ids, 6)
    xb, gb = W.activations(40, 64, 3), W.gaussian_bf16((80, 48), 1.0, 3, 4)
    x, g = (torch.from_numpy(of.bf16_to_f32(b).astype(np.float64)) for b in (xb, gb))
    w = torch.zeros(6, 48, 64, dtype=torch.float64, requires_grad=True)
    src = torch.from_numpy(r2t.astype(np.int64) // 2)
    sum((g[off[e]:off[e + 1]] * (x[src[off[e]:off[e + 1]]] @ w[e].T)).sum() for e in range(6)).backward()
    got = host(pmg.bf16_grouped_gemm_wgrad(bf16_dev(gb), bf16_dev(xb), dev(off), row_to_tk=dev(r2t), k=2, gather="x"))
    assert np.allclose(got, w.grad.numpy(), rtol=1e-5, atol=1e-5 * float(w.grad.abs().max()))


def test_binding_refusals():
    g, x = (torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert not pmg.bf16_grouped_gemm_wgrad(g, x, off).any()
    with pytest.raises(ValueError, match="same rows"):
        pmg.bf16_grouped_gemm_wgrad(g[:4], x, off)
    with pytest.raises(ValueError, match="row_to_tk"):
        pmg.bf16_grouped_gemm_wgrad(g, x, off, gather="x")
    with pytest.raises(ValueError, match="gather"):
        pmg.bf16_grouped_gemm_wgrad(g, x, off, gather="y")
    with pytest.raises(ValueError, match="entries"):
        pmg.bf16_grouped_gemm_wgrad(g, x, off, row_to_tk=torch.zeros(9, dtype=torch.int32, device="cuda"), gather="x")
    with pytest.raises(pmg.NVFP4Error):
        pmg.bf16_grouped_gemm_wgrad(g[:, :12].contiguous(), x, off)
