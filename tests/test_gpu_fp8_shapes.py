"""GPU parity of the FP8 products where their parts meet: several tiles of several K-steps to a workgroup
(a tile's stores in flight under the next one's loads, the next tile's routing map), the border between the
few-row kernel and the tiles, the longest rows; and the transposed weights alone.

Bounds as in test_gpu_fp8; FP32 outputs of K elements within (130 + K / 128) 2^-24 sum |a w|.
"""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
import workloads as W
from oracle import formats as of, fp8 as o8
from helpers import assert_within, bf16_dev, dev, gpu_ready, host
from test_gpu_fp8 import _check_gemm, _operands, _routing

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]


@pytest.mark.parametrize("T,E,k,N,K,kind", [(6000, 7, 4, 2056, 400, "zipf"), (6000, 7, 4, 1025, 400, "softmax"),
                                            (4096, 16, 8, 1536, 2048, "softmax"), (20000, 1, 1, 1288, 272, "softmax"),
                                            (5000, 300, 4, 264, 784, "zipf")])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_several_tiles_of_several_steps(T, E, k, N, K, kind, gather, out):
    print(f"[fp8 gemm] tiles T={T} E={E} k={k} N={N} K={K} {kind} gather={gather} {out}", flush=True)
    off, r2t = _routing(T, E, k, kind, 5)
    _, c = _check_gemm(off, r2t, k, E, N, K, gather, out, seed=13, spare=3, T=T, sample=250)
    assert torch.isfinite(c).all()


@pytest.mark.parametrize("E", [1, 5, 128])
@pytest.mark.parametrize("past", [0, 1])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_at_the_border_of_the_few_row_kernel(E, past, gather, out):
    """128 + 8 E rows, those past the last one included, are the most it takes."""
    T, spare = 125 + 8 * E + past, 3
    print(f"[fp8 gemm] border E={E} rows={T + spare} gather={gather} {out}", flush=True)
    off, r2t = _routing(T, E, 1, "uniform", E)
    _, c = _check_gemm(off, r2t, 1, E, 136, 400, gather, out, seed=E, spare=spare, T=T)
    assert torch.isfinite(c).all()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_rows_on_both_sides_of_the_border(out):
    """The same rows give the same bits from the few-row kernel (up to 168 rows for 5 experts) and from tiles."""
    E, N, K, T = 5, 264, 656, 400
    a, sa, w, sw = (dev(v) for v in _operands(T, E, N, K, 2))
    expert = np.random.default_rng(2).integers(0, E, T)

    def run(n):
        order = np.argsort(expert[:n], kind="stable")
        off = np.concatenate([[0], np.cumsum(np.bincount(expert[:n], minlength=E))]).astype(np.int32)
        c = pmg.fp8_grouped_gemm_gather(a, sa, dev(order.astype(np.int32)), 1, dev(off), w, sw, out_dtype=out)
        return c[torch.from_numpy(np.argsort(order, kind="stable")).cuda()]

    full = run(T)
    assert torch.isfinite(full).all()
    for n in (167, 168, 169, 170):
        assert torch.equal(run(n), full[:n]), n


@pytest.mark.parametrize("R", [40, 300])
def test_the_longest_rows_of_one_sign(R):
    """Nothing cancels over K = 65536, so every rounding of the sums counts."""
    K, N = 65536, 48
    r = np.random.default_rng(4)
    a, sa = o8.quantize_rows(r.random((R, K), np.float32) + 0.5)
    w, sw = o8.quantize_weights(r.random((1, N, K), np.float32) + 0.5)
    off = np.array([0, R], np.int32)
    at = np.arange(0, R, 7)
    ref, mag = o8.grouped_gemm_ref(a, sa, off, w, sw, rows=at)
    got = host(pmg.fp8_grouped_gemm(dev(a), dev(sa), dev(off), dev(w), dev(sw)))
    assert np.isfinite(got).all()
    print("  err/bound", assert_within(got[at], ref, (130 + K / 128) * 2.0 ** -24 * mag / o8.REL_TOL, f"R={R}"), flush=True)


@pytest.mark.parametrize("E,N,K", [(1, 16, 16), (3, 144, 272), (2, 400, 112)])
def test_transposed_weights_alone(E, N, K):
    """The C entry point without the stored order (codes and scales NULL)."""
    b = W.f32_to_bf16_bits((0.02 * np.random.default_rng(N).standard_normal((E, N, K))).astype(np.float32))
    w = bf16_dev(b)
    ct = torch.full((E, K, N), 0x55, dtype=torch.uint8, device="cuda")
    st = torch.full((E, o8.blocks(K), o8.blocks(N)), -1.0, device="cuda")
    status = pmg.load_library().fp8_quantize_weights(w.data_ptr(), E, N, K, None, None, ct.data_ptr(), st.data_ptr(),
                                                     torch.cuda.current_stream().cuda_stream)
    assert status == 0
    rc, rs = o8.quantize_weights(of.bf16_to_f32(b))
    assert np.array_equal(host(ct), rc.transpose(0, 2, 1)) and np.array_equal(host(st), rs.transpose(0, 2, 1))
