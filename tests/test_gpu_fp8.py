"""GPU parity: the FP8 block-128 quantisers and grouped GEMM.

Quantiser codes and scales are bit-exact against the oracle.  The SwiGLU's are
held to the definition's half steps around the float64 value: h itself within
2^-20 relative, a scale within that of amax / 448, a decoded value within half an
E4M3 step of h (2^-4 relative for normal codes, 2^-10 scale below), the bf16 h
within 2^-8.  FP32 GEMM outputs are within 2e-5 sum |a w| per element: the FP32
sums take at most 128 + K / 128 roundings of 2^-24 each (1.2e-5 at K = 8192).
BF16 outputs come from the FP8 matrix instruction, which cuts each product of 8
consecutive k off at 2^-13 of the largest of the 8: at most seven of them lose less
than 2^-13 of that largest product, which is at most the eight's sum |a w|, so
together less than 7 2^-13 sum |a w|; half a bf16 step (2^-8 relative) comes on
top.  Their error over all elements is also held to half a bf16 step in 2-norm.
"""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
import workloads as W
from oracle import formats as of, fp8 as o8, permute as op
from helpers import assert_within, bf16_dev, bf16_host, dev, gpu_ready, host

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]


def bits(a):
    return np.ascontiguousarray(a).view(np.uint32)


def _values(shape, seed):
    """Float32 values over many binades, with zero, tiny and repeated-maximum blocks among them."""
    r = np.random.default_rng(seed)
    x = r.standard_normal(shape) * np.exp2(r.integers(-14, 6, shape))
    x = x.astype(np.float32).reshape(-1)
    n = x.size
    x[: n // 7] *= np.float32(2.0 ** -60)
    x[n // 3: n // 3 + 200] = 0
    return x.reshape(shape)


# ------------------------------------------------------------------ quantisers
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 2048), (3, 128), (17, 144), (16, 784), (33, 8192), (1030, 2064),
                                    (4100, 640)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows(rows, K, dtype):
    print(f"[fp8 rows] {rows}x{K} {dtype}", flush=True)
    x = _values((rows, K), rows + K)
    if dtype == "bf16":
        b = W.f32_to_bf16_bits(x)
        x, t = of.bf16_to_f32(b), bf16_dev(b)
    else:
        t = dev(x)
    codes, scales = pmg.fp8_quantize_rows(t)
    rc, rs = o8.quantize_rows(x)
    assert np.array_equal(bits(host(scales)), bits(rs))
    assert np.array_equal(host(codes), rc)


def test_rows_ties_and_extremes():
    """Every E4M3 midpoint and its float32 neighbours, float32 subnormals and maxima, s underflowing to 0."""
    pos = of.e4m3_decode(np.arange(0x7F, dtype=np.uint8))
    mid = ((pos[:-1] + pos[1:]) / 2).astype(np.float32)
    rows = []
    for scale in (1.0, 2.0 ** -100, 2.0 ** 90, 3.0, 1.7e-38):
        for m in (mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)), -mid):
            v = np.zeros(128, np.float32)
            v[:126] = m
            v[127] = 448
            rows.append((v.astype(np.float64) * scale).astype(np.float32))
    tiny = np.float32(2.0 ** -149)
    for v in (tiny, 100 * tiny, 300 * tiny, 1000 * tiny, np.float32(3.4e38)):
        rows.append((np.arange(128) % 3 - 1).astype(np.float32) * v)
    rows.append(np.linspace(-1, 1, 128, dtype=np.float32) * np.float32(3.4028235e38))
    x = np.stack(rows)
    codes, scales = pmg.fp8_quantize_rows(dev(x))
    rc, rs = o8.quantize_rows(x)
    assert np.array_equal(bits(host(scales)), bits(rs))
    got = host(codes)
    zero = (rc & 0x7F) == 0                               # where s == 0 the sign of a zero code is not compared
    assert np.array_equal(got[~zero], rc[~zero]) and not (got[zero] & 0x7F).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_next_to_midpoints(dtype):
    """448 x / amax at, and a few steps of x to either side of, every midpoint, for many amax and binades."""
    r = np.random.default_rng(12)
    pos = of.e4m3_decode(np.arange(0x7F, dtype=np.uint8))
    mid = (pos[:-1] + pos[1:]) / 2
    amax = np.abs(r.standard_normal(240)) * np.exp2(r.choice([-140, -100, -79, -3, 0, 5, 70, 90], 240))
    if dtype == "bf16":
        amax = of.bf16_to_f32(W.f32_to_bf16_bits(amax.astype(np.float32)))
    amax = amax.astype(np.float32)
    x = np.zeros((240, 128), np.float32)
    x[:, :126] = amax[:, None].astype(np.float64) * mid / 448
    for i in range(240):
        for _ in range(i % 3):
            x[i] = np.nextafter(x[i], np.float32(0 if i % 2 else np.inf))
    if dtype == "bf16":
        x = of.bf16_to_f32(W.f32_to_bf16_bits(x))
    x = np.minimum(x, amax[:, None]) * np.where(np.arange(240) % 5 == 0, -1, 1).astype(np.float32)[:, None]
    x[:, 127] = amax
    codes, scales = pmg.fp8_quantize_rows(dev(x) if dtype == "f32" else bf16_dev(W.f32_to_bf16_bits(x)))
    rc, rs = o8.quantize_rows(x)
    assert np.array_equal(bits(host(scales)), bits(rs))
    live = (rs > 0).T
    assert np.array_equal(host(codes)[live[:, 0]], rc[live[:, 0]])


def test_rows_nan_and_infinity():
    x = np.ones((3, 256), np.float32)
    x[0, 5], x[1, 7], x[2, :128] = np.nan, np.inf, np.nan
    for t in (dev(x), dev(x).bfloat16()):
        codes, scales = (host(v) for v in pmg.fp8_quantize_rows(t))
        one = np.float32(1) / np.float32(448)
        assert codes[0, 5] & 0x7F == 0x7F and scales[0, 0] == one and (codes[0, 6:] == 0x7E).all()
        assert codes[1, 7] & 0x7F == 0x7F and scales[0, 1] == np.inf and (codes[1, :7] == 0).all()
        assert (codes[2, :128] & 0x7F == 0x7F).all() and scales[0, 2] == 0 and (codes[2, 128:] == 0x7E).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_long_inputs_match_short_ones(dtype):
    """Rows of a long input, several blocks to a lane, against the same rows quantised in small calls."""
    x = torch.randn((41000, 1040), generator=torch.Generator("cuda").manual_seed(3), device="cuda").to(dtype)
    codes, scales = pmg.fp8_quantize_rows(x)
    for a, b in ((0, 700), (20000, 20033), (40900, 41000)):
        c, s = pmg.fp8_quantize_rows(x[a:b].clone())
        assert torch.equal(codes[a:b], c) and torch.equal(scales[:, a:b], s)


def test_rows_stop_at_the_routed_rows():
    x = dev(np.random.default_rng(1).standard_normal((40, 272)).astype(np.float32))
    off = dev(np.array([0, 3, 21], np.int32))
    codes = torch.full((40, 272), 0x55, dtype=torch.uint8, device=x.device)
    scales = torch.full((3, 40), -1.0, device=x.device)
    pmg.fp8_quantize_rows(x, off, codes, scales)
    full = pmg.fp8_quantize_rows(x)
    assert torch.equal(codes[:21], full[0][:21]) and torch.equal(scales[:, :21], full[1][:, :21])
    assert (codes[21:] == 0x55).all() and (scales[:, 21:] == -1).all()


@pytest.mark.parametrize("E,N,K", [(1, 128, 128), (1, 16, 16), (3, 144, 272), (2, 400, 112), (5, 1536, 2048),
                                   (2, 4112, 64)])
def test_weights(E, N, K):
    print(f"[fp8 weights] {E}x{N}x{K}", flush=True)
    b = W.f32_to_bf16_bits(_values((E, N, K), N + K))
    rc, rs = o8.quantize_weights(of.bf16_to_f32(b))
    c, s, ct, st = pmg.fp8_quantize_weights(bf16_dev(b), transposed=True)
    assert np.array_equal(bits(host(s)), bits(rs)) and np.array_equal(host(c), rc)
    assert np.array_equal(bits(host(st)), bits(rs.transpose(0, 2, 1))) and np.array_equal(host(ct), rc.transpose(0, 2, 1))
    c2, s2 = pmg.fp8_quantize_weights(bf16_dev(b))
    assert torch.equal(c2, c) and torch.equal(s2, s)


def test_weights_odd_rows_without_transpose():
    b = W.f32_to_bf16_bits(_values((2, 131, 48), 9))
    rc, rs = o8.quantize_weights(of.bf16_to_f32(b))
    c, s = pmg.fp8_quantize_weights(bf16_dev(b))
    assert np.array_equal(bits(host(s)), bits(rs)) and np.array_equal(host(c), rc)


def _check_swiglu(gu_t, gu, w, off, r2t, h_out):
    R_cap, I = gu.shape[0], gu.shape[1] // 2
    n = int(off[-1])
    out = {"codes": torch.full((R_cap, I), 0x55, dtype=torch.uint8, device=gu_t.device),
           "scales": torch.full((o8.blocks(I), R_cap), -1.0, device=gu_t.device),
           "h": torch.full((R_cap, I), 7.0, dtype=torch.bfloat16, device=gu_t.device)}
    c, s, h = pmg.fp8_swiglu_quantize(gu_t, dev(off), None if w is None else dev(w), None if r2t is None else dev(r2t),
                                      h_out=h_out, out=out)
    assert (h is None) == (not h_out)
    wr = None if w is None else w[r2t[:n]]
    ref = o8.swiglu(gu[:n], wr)
    c, s = host(c), host(s)
    assert (c[n:] == 0x55).all() and (s[:, n:] == -1).all()
    for j in range(o8.blocks(I)):
        hb = ref[:, 128 * j:128 * (j + 1)]
        s64 = np.abs(hb).max(axis=1) / 448
        assert (np.abs(s[j, :n] - s64) <= (2.0 ** -20 + 2.0 ** -23) * s64 + 2.0 ** -149).all()
        val = of.e4m3_decode(c[:n, 128 * j:128 * (j + 1)]) * s[j, :n].astype(np.float64)[:, None]
        half = np.maximum(2.0 ** -4 * np.abs(hb), 2.0 ** -10 * s64[:, None])
        assert_within(val, hb, half * (1 + 2.0 ** -17) + 2.0 ** -18 * np.abs(hb), f"swiglu codes block {j}")
    if h_out:
        got = of.bf16_to_f32(bf16_host(h))
        assert_within(got[:n], ref, (2.0 ** -8 + 2.0 ** -19) * np.abs(ref) + 2.0 ** -133, "swiglu h")
        assert (got[n:] == 7).all()


@pytest.mark.parametrize("R,I,E", [(1, 16, 1), (8, 768, 128), (19, 144, 3), (700, 2048, 16), (6000, 400, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weighted", [True, False])
def test_swiglu(R, I, E, dtype, weighted):
    print(f"[fp8 swiglu] R={R} I={I} {dtype} weighted={weighted}", flush=True)
    r = np.random.default_rng(R + I)
    gu = (r.standard_normal((R + 3, 2 * I)) * 2).astype(np.float32)
    gu[0, :16] = [0.0, -0.0, 88, -88, 30, -30, 1e-30, -1e-30, 100, -100, 5, -5, 17, -17, 0.5, -0.5]
    off = np.zeros(E + 1, np.int32)
    off[1:] = np.sort(r.integers(0, R + 1, E))
    off[-1] = R
    r2t = r.permutation(R + 3).astype(np.int32)
    w = r.random(R + 3).astype(np.float32)
    if dtype == "bf16":
        b = W.f32_to_bf16_bits(gu)
        gu, t = of.bf16_to_f32(b), bf16_dev(b)
    else:
        t = dev(gu)
    for h_out in (True, False):
        _check_swiglu(t, gu, w if weighted else None, off, r2t if weighted else None, h_out)


def test_swiglu_infinite_gates():
    """+inf gates give inf, -inf gates and NaN give NaN, as g / (1 + exp(-g)) does; a bad map entry weighs 0."""
    gu = np.ones((2, 32), np.float32)
    gu[0, 0], gu[0, 1], gu[0, 2] = np.inf, -np.inf, np.nan
    r2t = np.array([0, 99], np.int32)
    c, s, h = pmg.fp8_swiglu_quantize(dev(gu), dev(np.array([0, 2], np.int32)), dev(np.ones(2, np.float32)), dev(r2t),
                                      h_out=True)
    h, c, s = of.bf16_to_f32(bf16_host(h)), host(c), host(s)
    assert h[0, 0] == np.inf and np.isnan(h[0, 1]) and np.isnan(h[0, 2]) and np.isfinite(h[0, 3:]).all()
    assert s[0, 0] == np.inf and (c[0, :3] & 0x7F == 0x7F).all()
    assert (h[1] == 0).all() and s[0, 1] == 0 and not (c[1] & 0x7F).any()


# ------------------------------------------------------------------ grouped GEMM
def _routing(T, E, k, kind, seed):
    ids, _ = W.make_routing(kind, T, E, k, seed)
    off, r2t, _, _ = op.permute(ids, E)
    return off, r2t


def _operands(rows, E, N, K, seed):
    r = np.random.default_rng(seed)
    a, sa = o8.quantize_rows(of.bf16_to_f32(W.activations(rows, K, seed)))
    w, sw = o8.quantize_weights((0.02 * r.standard_normal((E, N, K))).astype(np.float32))
    return a, sa, w, sw


def _check_gemm(off, r2t, k, E, N, K, gather, out, seed, spare=0, T=None, sample=None):
    """Every routed row (or `sample` of them); `spare` rows past the last hold NaN codes and must stay untouched."""
    R = int(off[-1])
    rows = T if gather else R + spare
    a, sa, w, sw = _operands(rows, E, N, K, seed)
    if not gather and spare:
        a[R:] = 0x7F
        sa[:, R:] = np.nan
    src = r2t.astype(np.int64) // k if gather else None
    at = np.arange(R) if sample is None or R <= sample else np.sort(np.random.default_rng(seed).choice(R, sample, replace=False))
    ref, bound = o8.grouped_gemm_ref(a, sa, off, w, sw, row_source=src, rows=at)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    c = torch.full((R + spare, N), 12345.0, dtype=dt, device="cuda")
    args = (dev(a), dev(sa))
    tail = (dev(off), dev(w), dev(sw))
    if gather:
        m = np.concatenate([r2t, np.full(spare, -5, np.int32)])
        pmg.fp8_grouped_gemm_gather(*args, dev(m), k, *tail, c=c)
    else:
        pmg.fp8_grouped_gemm(*args, *tail, c=c)
    got = c.float().cpu().numpy().astype(np.float64)
    assert (got[R:] == float(torch.tensor(12345.0, dtype=dt))).all(), "rows past the last were written"
    if out == "bf16":
        bound = bound * (1 + 7 * 2.0 ** -13 / o8.REL_TOL)
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
        assert np.linalg.norm(got[at] - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    return assert_within(got[at], ref, bound, f"N={N} K={K}"), c


SMALL = [  # T, E, k, N, K, routing: few rows per expert
    (1, 128, 8, 1536, 2048, "softmax"), (1, 1, 1, 1, 16, "softmax"), (2, 4, 2, 33, 48, "uniform"),
    (5, 8, 3, 130, 144, "zipf"), (16, 16, 4, 96, 784, "uniform"), (61, 128, 8, 256, 768, "uniform"),
    (64, 1, 1, 300, 2064, "softmax"), (200, 1024, 1, 40, 32, "zipf"), (40, 16, 6, 257, 1040, "zipf"),
    (3, 2, 1, 64, 4096, "uniform"), (17, 7, 1, 31, 8208, "uniform")]
LARGE = [  # more rows than 128 and 8 per expert (tiles through LDS), and next to that border
    (65, 1, 1, 256, 128, "softmax"), (257, 1, 1, 512, 256, "softmax"), (300, 2, 2, 272, 144, "uniform"),
    (700, 16, 4, 513, 784, "zipf"), (1021, 24, 4, 131, 1040, "zipf"), (300, 7, 3, 1, 16, "uniform"),
    (256, 3, 1, 255, 2064, "zipf"), (1100, 4, 2, 768, 528, "softmax"), (2048, 64, 2, 96, 96, "uniform"),
    (129, 1, 1, 1030, 4000, "softmax"), (2100, 1024, 4, 40, 32, "zipf"), (137, 1, 1, 70, 272, "softmax"),
    (136, 1, 1, 70, 272, "softmax")]


@pytest.mark.parametrize("T,E,k,N,K,kind", SMALL + LARGE)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gemm(T, E, k, N, K, kind, gather, out):
    print(f"[fp8 gemm] T={T} E={E} k={k} N={N} K={K} {kind} gather={gather} {out}", flush=True)
    off, r2t = _routing(T, E, k, kind, T + N)
    _check_gemm(off, r2t, k, E, N, K, gather, out, seed=T + K, spare=3, T=T, sample=400)


def test_gemm_layer_shapes():
    """The layer's gate_up and dense QKV products at the training length, on sampled rows."""
    for T, E, k, N, K, kind, gather in [(4096, 16, 8, 1536, 2048, "softmax", True), (4096, 1, 1, 5120, 2048, "softmax", False),
                                        (4096, 32, 4, 2048, 768, "zipf", False)]:
        print(f"[fp8 gemm] layer T={T} E={E} N={N} K={K} {kind}", flush=True)
        off, r2t = _routing(T, E, k, kind, 7)
        _check_gemm(off, r2t, k, E, N, K, gather, "f32", seed=11, T=T, sample=150)


def test_gemm_empty_and_single_row_experts():
    """No routed rows at all (nothing is written), and routings of 0, 1 and many rows side by side."""
    a, sa, w, sw = _operands(64, 5, 48, 160, 3)
    c = torch.full((64, 48), 3.0, device="cuda")
    pmg.fp8_grouped_gemm(dev(a), dev(sa), dev(np.zeros(6, np.int32)), dev(w), dev(sw), c=c)
    assert (c == 3).all()
    assert pmg.fp8_grouped_gemm(dev(a[:0]), dev(sa[:, :0].copy()), dev(np.zeros(6, np.int32)), dev(w), dev(sw)).shape == (0, 48)
    for counts in ([0, 1, 0, 600, 0], [1, 1, 1, 1, 1], [0, 0, 0, 0, 257], [300, 0, 0, 0, 1]):
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        _check_gemm(off, None, 1, 5, 48, 160, False, "f32", seed=5, spare=2)


def test_gemm_non_finite_values_stay_in_their_rows():
    """A NaN code or infinite scale makes its own row NaN and leaves every other row's bits alone."""
    for counts in ([5, 7], [100, 300]):
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        R = int(off[-1])
        a, sa, w, sw = _operands(R, 2, 80, 272, 4)
        clean = host(pmg.fp8_grouped_gemm(dev(a), dev(sa), dev(off), dev(w), dev(sw)))
        a[3, 200] = 0x7F
        a[4, 9], sa[0, 4] = 0xFF, np.inf
        got = host(pmg.fp8_grouped_gemm(dev(a), dev(sa), dev(off), dev(w), dev(sw)))
        assert np.isnan(got[3:5]).all()
        assert np.array_equal(bits(np.delete(got, [3, 4], 0)), bits(np.delete(clean, [3, 4], 0)))


def test_gemm_malformed_offsets_stay_inside():
    """Falling, negative and too large offsets: rows beside the output and rows that no range names stay as they were."""
    for R in (100, 700):
        a, sa, w, sw = (dev(v) for v in _operands(R, 4, 80, 272, 4))
        whole = torch.full((R + 64, 80), 5.0, device="cuda")
        c = whole[32:32 + R]
        for off in ([0, R, 0, R, 0], [-7, R // 2, R + 900, R, R], [R, R, R, R, R], [2 ** 31 - 1, -2 ** 31, 9, 8, 7]):
            pmg.fp8_grouped_gemm(a, sa, dev(np.array(off, np.int32)), w, sw, c=c)
            assert (whole[:32] == 5).all() and (whole[32 + R:] == 5).all()
        pmg.fp8_grouped_gemm(a, sa, dev(np.array([0, 9, 9, 60, 60], np.int32)), w, sw, c=c.fill_(5))
        assert (c[60:] == 5).all() and (c[:60] != 5).any(1).all()


def test_gemm_repeats_bit_for_bit():
    for T in (9, 700):
        off, r2t = _routing(T, 16, 4, "zipf", 3)
        a, sa, w, sw = (dev(v) for v in _operands(T, 16, 272, 528, 5))
        first = pmg.fp8_grouped_gemm_gather(a, sa, dev(r2t), 4, dev(off), w, sw)
        for _ in range(3):
            assert torch.equal(pmg.fp8_grouped_gemm_gather(a, sa, dev(r2t), 4, dev(off), w, sw), first)
        grouped = pmg.fp8_grouped_gemm(a[torch.from_numpy(r2t.astype(np.int64) // 4).cuda()].contiguous(),
                                       sa[:, torch.from_numpy(r2t.astype(np.int64) // 4).cuda()].contiguous(), dev(off), w, sw)
        assert torch.equal(grouped, first)


def test_gemm_input_gradient_with_transposed_weights():
    """dA = dC W through the transposed codes against the stored ones' definition."""
    E, N, K, R = 3, 144, 272, 500
    r = np.random.default_rng(2)
    wb = W.f32_to_bf16_bits((0.02 * r.standard_normal((E, N, K))).astype(np.float32))
    c, s, ct, st = pmg.fp8_quantize_weights(bf16_dev(wb), transposed=True)
    dc = r.standard_normal((R, N)).astype(np.float32)
    ac, asc = pmg.fp8_quantize_rows(dev(dc))
    off = np.array([0, 200, 200, 500], np.int32)
    got = host(pmg.fp8_grouped_gemm(ac, asc, dev(off), ct, st))
    a = o8.dequantize_rows(host(ac), host(asc))
    for e in range(E):
        w = o8.dequantize_weight(host(c)[e], host(s)[e])
        rows = slice(off[e], off[e + 1])
        assert_within(got[rows], a[rows] @ w, 2e-5 * (np.abs(a[rows]) @ np.abs(w)) + 1e-300, f"dgrad e{e}")


def test_binding_refusals():
    u8 = torch.zeros(8, 256, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(2, 8, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    w, sw = torch.zeros(1, 128, 256, dtype=torch.uint8, device="cuda"), torch.zeros(1, 1, 2, device="cuda")
    ok = pmg.fp8_grouped_gemm(u8, sc, off, w, sw)
    assert ok.shape == (8, 128)
    with pytest.raises(ValueError, match="a_scales"):
        pmg.fp8_grouped_gemm(u8, sc.t().contiguous(), off, w, sw)
    with pytest.raises(ValueError, match="w_scales"):
        pmg.fp8_grouped_gemm(u8, sc, off, w, sw[0])
    with pytest.raises(ValueError, match="w_codes"):
        pmg.fp8_grouped_gemm(u8[:, :128].contiguous(), sc[:1].contiguous(), off, w, sw)
    with pytest.raises(ValueError, match="contiguous"):
        pmg.fp8_quantize_rows(torch.zeros(8, 512, device="cuda")[:, :256])
    with pytest.raises(ValueError, match="holds"):
        pmg.fp8_quantize_rows(torch.zeros(8, 256, device="cuda"), codes=u8[:4])
    with pytest.raises(pmg.NVFP4Error):
        pmg.fp8_quantize_rows(torch.zeros(8, 20, device="cuda"))
    with pytest.raises(TypeError):
        pmg.fp8_grouped_gemm(u8, sc, off, w, sw, out_dtype=torch.float16)
    for args in ((u8, sc, off.cpu(), w, sw), (u8, sc, off, w.cpu(), sw), (u8, sc.cpu(), off, w, sw)):
        with pytest.raises(ValueError, match="device tensor"):
            pmg.fp8_grouped_gemm(*args)
    gu = torch.zeros(8, 64, device="cuda")
    with pytest.raises(ValueError, match="row_to_tk"):
        pmg.fp8_swiglu_quantize(gu, off, torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError, match="holds"):
        pmg.fp8_swiglu_quantize(gu, off, torch.zeros(7, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda"))


def test_float8_tensors_are_codes():
    """Codes may be held as torch.float8_e4m3fn tensors, on either side and as outputs."""
    f8 = torch.float8_e4m3fn
    x = dev(_values((40, 272), 2))
    c, s = pmg.fp8_quantize_rows(x)
    c8 = torch.empty((40, 272), dtype=f8, device="cuda")
    got, s8 = pmg.fp8_quantize_rows(x, codes=c8)
    assert got is c8 and torch.equal(c8.view(torch.uint8), c) and torch.equal(s8, s)
    w, sw = pmg.fp8_quantize_weights(bf16_dev(W.gaussian_bf16((2, 48, 272), 0.02, 1, 2)))
    off = dev(np.array([0, 9, 40], np.int32))
    assert torch.equal(pmg.fp8_grouped_gemm(c8, s, off, w.view(f8), sw), pmg.fp8_grouped_gemm(c, s, off, w, sw))
    ref = (c8.float() * s.t().repeat_interleave(128, 1)[:, :272])
    assert (ref - x).abs().max() <= 2.0 ** -4 * x.abs().max() * (1 + 2.0 ** -20)
