"""GPU parity: FP8 products whose two scales multiply to something outside the normal float32 numbers.

A block's term is sa sw p with p the block's sum of code products, 2^-18 <= |p| < 2^25 or 0, so it can
be an ordinary number where sa sw is subnormal, zero or infinite.  The bound is that of any product,
2e-5 sum |a w| (test_gpu_fp8), and 2^-149 for each block and one more: a term below the normal range
is rounded to a multiple of 2^-149, by half a step, and so is what is left of it in the product with the
mantissas; the sums of such terms are exact.  BF16 outputs: as in test_gpu_fp8, with half a step of the
smallest bf16 numbers (2^-134).
"""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
from oracle import fp8 as o8
from helpers import assert_within, dev, gpu_ready

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]

E, N, K = 2, 272, 400
KB, NB = o8.blocks(K), o8.blocks(N)


def _operands(R):
    """Codes and scales with sa sw between 2^-290 and 2^200; a row's block is zero where a term could overflow."""
    r = np.random.default_rng(8)
    a, _ = o8.quantize_rows(r.standard_normal((R, K)).astype(np.float32))
    w, _ = o8.quantize_weights(r.standard_normal((E, N, K)).astype(np.float32))
    mantissa = lambda shape: 1 + r.random(shape)
    sw = (mantissa((E, NB, KB)) * np.exp2(r.choice([-145, -100, -70, -63, 0, 60, 100], (E, NB, KB)))).astype(np.float32)
    sa = (mantissa((KB, R)) * np.exp2(r.choice([-145, -126, -75, -70, -60, 3, 70, 100], (KB, R)))).astype(np.float32)
    sa[:, 5], sa[1, 6], sw[1, 2, 3] = 0, 0, 0
    expert = (np.arange(R) >= R // 3).astype(int)
    for j in range(KB):
        big = sa[j].astype(np.float64) * sw[:, :, j].astype(np.float64).max(1)[expert] >= 2.0 ** 99
        a[big, 128 * j:128 * (j + 1)] = 0
    return a, sa, w, sw, np.array([0, R // 3, R], np.int32)


@pytest.mark.parametrize("R", [60, 600])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_scale_products_of_any_size(R, out):
    print(f"[fp8 scales] R={R} {out}", flush=True)
    a, sa, w, sw, off = _operands(R)
    with np.errstate(over="ignore", under="ignore"):
        prod = sa[:, :, None] * sw[0].T[:, None, :]
        assert (prod == 0).any() and np.isinf(prod).any() and ((prod > 0) & (prod < 2.0 ** -126)).any()
    ref, bound = o8.grouped_gemm_ref(a, sa, off, w, sw)
    if out == "bf16":
        bound = bound * (1 + 7 * 2.0 ** -13 / o8.REL_TOL)
    bound = bound + (KB + 1) * 2.0 ** -149
    if out == "bf16":
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound) + 2.0 ** -134
    assert (np.abs(ref) < 2.0 ** 127).all() and (np.abs(ref) > 2.0 ** -100).any()
    dt = torch.float32 if out == "f32" else torch.bfloat16
    got = pmg.fp8_grouped_gemm(dev(a), dev(sa), dev(off), dev(w), dev(sw), out_dtype=dt)
    assert torch.isfinite(got).all()
    print("  err/bound", assert_within(got.double().cpu().numpy(), ref, bound, out), flush=True)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_a_row_alone_and_in_a_batch(out):
    """The same bits from either kernel, and whatever the scales of the rows beside it are."""
    a, sa, w, sw, off = _operands(600)
    full = pmg.fp8_grouped_gemm(dev(a), dev(sa), dev(off), dev(w), dev(sw), out_dtype=out)
    for rows in (np.arange(0, 30), np.arange(150, 210), np.array([5]), np.array([599])):
        o = np.array([0, (rows < 200).sum(), rows.size], np.int32)
        got = pmg.fp8_grouped_gemm(dev(a[rows]), dev(sa[:, rows].copy()), dev(o), dev(w), dev(sw), out_dtype=out)
        assert torch.equal(got, full[torch.from_numpy(rows).cuda()])
    plain = sa.copy()                      # the other rows' scales become ordinary ones, row 300 keeps its own
    plain[:] = 0.01
    plain[:, 300] = sa[:, 300]
    got = pmg.fp8_grouped_gemm(dev(a), dev(plain), dev(off), dev(w), dev(sw), out_dtype=out)
    assert torch.equal(got[300], full[300])


@pytest.mark.parametrize("N,K", [(1032, 400), (515, 272)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_a_few_such_rows_among_many_tiles(N, K, out):
    """One row in 50, gathered; those rows and some others as they come from the few-row kernel."""
    T, E, k = 4000, 6, 3
    r = np.random.default_rng(3)
    a, sa = o8.quantize_rows(r.standard_normal((T, K)).astype(np.float32))
    w, sw = o8.quantize_weights(r.standard_normal((E, N, K)).astype(np.float32))
    sw[:, :, 1::2] = np.float32(2.0 ** -90)
    far = np.arange(0, T, 50)
    sa[:, far] = (1 + r.random((sa.shape[0], far.size))).astype(np.float32) * np.float32(2.0 ** -50)
    expert = np.argsort(r.random((T, E)), axis=1)[:, :k].reshape(-1)
    r2t = np.argsort(expert, kind="stable").astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(expert, minlength=E))]).astype(np.int32)
    full = pmg.fp8_grouped_gemm_gather(dev(a), dev(sa), dev(r2t), k, dev(off), dev(w), dev(sw), out_dtype=out)
    assert torch.isfinite(full).all()
    for tokens in (far[:20], far[-20:], far[:20] + 1, np.arange(1985, 2005)):
        rows = np.nonzero(np.isin(r2t // k, tokens))[0]
        o = np.searchsorted(rows, off).astype(np.int32)
        assert rows.size <= 128 + 8 * E
        got = pmg.fp8_grouped_gemm_gather(dev(a), dev(sa), dev(r2t[rows]), k, dev(o), dev(w), dev(sw), out_dtype=out)
        assert torch.equal(got, full[torch.from_numpy(rows).cuda()])


def test_infinite_and_nan_scales():
    """An infinite scale gives what the formula gives: an infinity, or NaN where it meets a zero."""
    one = o8.quantize_rows(np.ones((2, 128), np.float32))[0]
    w = o8.quantize_weights(np.ones((1, 16, 128), np.float32))[0]
    w[0, 3] = 0
    for R in (2, 400):
        a, sa = np.repeat(one, R // 2, 0), np.full((1, R), 2.0 ** -20, np.float32)
        sa[0, 0], sa[0, 1] = np.inf, np.nan
        got = pmg.fp8_grouped_gemm(dev(a), dev(sa), dev(np.array([0, R], np.int32)), dev(w),
                                   dev(np.full((1, 1, 1), 2.0 ** -120, np.float32))).cpu().numpy()
        assert np.isinf(np.delete(got[0], 3)).all() and np.isnan(got[0, 3]) and np.isnan(got[1]).all()
        if R > 2:
            assert np.allclose(got[2:, 0], 128 * 448.0 ** 2 * 2.0 ** -140, rtol=2e-5, atol=0) and (got[2:, 3] == 0).all()
