"""The FP8 oracle against torch's E4M3 conversion, exact arithmetic and brute force (CPU)."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import formats as of, fp8 as o8

E4M3_POS = of.e4m3_decode(np.arange(0x7F, dtype=np.uint8))


def _nearest(v: float) -> int:
    """The nearest E4M3 code of a non-negative value by exhaustive search, ties to the even code."""
    v = min(Fraction(v), Fraction(448))
    d = [abs(Fraction(float(p)) - v) for p in E4M3_POS]
    best = min(d)
    at = [i for i, x in enumerate(d) if x == best]
    return at[0] if len(at) == 1 else next(i for i in at if i % 2 == 0)


def test_codes_match_exhaustive_search_and_torch():
    """The exact quotient's nearest code; torch's conversion of the float64 quotient rounded to float32 agrees
    wherever that is no midpoint."""
    r = np.random.default_rng(3)
    x = (r.standard_normal((16, 256)) * np.exp2(r.integers(-12, 9, (16, 256)))).astype(np.float32)
    codes, scales = o8.quantize_rows(x)
    amax = np.abs(x.reshape(16, 2, 128)).max(2)
    assert np.array_equal(scales.T, amax / np.float32(448))
    for row in (0, 3, 9):
        for i in range(0, 256, 3):
            want = Fraction(abs(float(x[row, i]))) * 448 / Fraction(float(amax[row, i // 128]))
            assert codes[row, i] & 0x7F == _nearest(want) and codes[row, i] >> 7 == np.signbit(x[row, i])
    q = (448.0 * x.astype(np.float64) / np.repeat(amax, 128, 1)).astype(np.float32)
    mids = (E4M3_POS[:-1] + E4M3_POS[1:]) / 2
    plain = ~np.isin(np.abs(q).astype(np.float64), mids)
    assert np.array_equal(codes[plain], torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()[plain])


def test_quotients_next_to_a_midpoint():
    """448 x / amax one float32 step of x to either side of every midpoint, for amax that no power of two scales to 448."""
    r = np.random.default_rng(4)
    mids = (E4M3_POS[:-1] + E4M3_POS[1:]) / 2
    for amax in np.abs(r.standard_normal(4)).astype(np.float32):
        near = (mids * float(amax) / 448).astype(np.float32)
        for x in (near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(9))):
            x = np.minimum(x, amax)
            got = o8.encode(x, amax)
            for c, v in zip(got, x):
                assert c == _nearest(Fraction(float(v)) * 448 / Fraction(float(amax)))


def test_every_tie_goes_to_the_even_code():
    mids = (E4M3_POS[:-1] + E4M3_POS[1:]) / 2
    x = np.zeros((1, 128), np.float32)
    x[0, :126] = mids
    x[0, 127] = 448.0                                    # s = 1 exactly
    codes, scales = o8.quantize_rows(x)
    assert scales[0, 0] == 1.0
    assert np.array_equal(codes[0, :126], [i if i % 2 == 0 else i + 1 for i in range(126)])


def test_block_edges_and_zero_blocks():
    x = np.zeros((2, 144), np.float32)
    x[0, 128:] = np.arange(16)
    x[1, 5] = -3.0
    codes, scales = o8.quantize_rows(x)
    assert scales.shape == (2, 2)
    assert scales[0, 0] == 0 and scales[1, 1] == 0 and not codes[0, :128].any() and not codes[1, 128:].any()
    assert codes[0, 143] == 0x7E and codes[1, 5] == 0xFE  # each block's maximum is +-448


def test_weights_are_rows_of_blocks():
    """A weight whose 128 x 128 blocks hold one row each quantises like those rows; transposing commutes."""
    r = np.random.default_rng(5)
    w = r.standard_normal((2, 200, 272)).astype(np.float32)
    codes, scales = o8.quantize_weights(w)
    ct, st = o8.quantize_weights(w.transpose(0, 2, 1))
    assert np.array_equal(ct, codes.transpose(0, 2, 1)) and np.array_equal(st, scales.transpose(0, 2, 1))
    one = w[:1, :1]
    c1, s1 = o8.quantize_weights(one)
    cr, sr = o8.quantize_rows(one[0])
    assert np.array_equal(c1[0], cr) and np.array_equal(s1[0, 0], sr[:, 0])


def test_gemm_ref_against_fractions():
    r = np.random.default_rng(7)
    a, sa = o8.quantize_rows(r.standard_normal((5, 144)).astype(np.float32))
    w, sw = o8.quantize_weights(r.standard_normal((2, 3, 144)).astype(np.float32))
    off = np.array([0, 2, 5])
    src = np.array([4, 0, 1, 1, 2])
    C, B = o8.grouped_gemm_ref(a, sa, off, w, sw, row_source=src)
    for row in range(5):
        e = 0 if row < 2 else 1
        for n in range(3):
            t = [Fraction(float(of.e4m3_decode(a[src[row], k]))) * Fraction(float(sa[k // 128, src[row]]))
                 * Fraction(float(of.e4m3_decode(w[e, n, k]))) * Fraction(float(sw[e, 0, k // 128])) for k in range(144)]
            assert abs(C[row, n] - float(sum(t))) <= 1e-12 * float(sum(abs(v) for v in t))
            assert B[row, n] == pytest.approx(2e-5 * float(sum(abs(v) for v in t)), rel=1e-12)


def test_swiglu_and_wgrad_against_loops():
    r = np.random.default_rng(9)
    gu, w = r.standard_normal((3, 8)), r.random(3)
    h = o8.swiglu(gu, w)
    for i in range(3):
        for j in range(4):
            g, u = gu[i, j], gu[i, 4 + j]
            assert h[i, j] == pytest.approx(w[i] * u * g / (1 + np.exp(-g)), rel=1e-14)
    g, x, off = r.standard_normal((6, 4)), r.standard_normal((6, 5)), [0, 4, 4, 6]
    dw, _ = o8.wgrad_ref(g, x, off)
    for e in range(3):
        ref = sum((np.outer(g[i], x[i]) for i in range(off[e], off[e + 1])), np.zeros((4, 5)))
        assert np.allclose(dw[e], ref, rtol=1e-13, atol=1e-15)
