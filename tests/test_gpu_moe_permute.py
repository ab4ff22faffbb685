"""moe_permute, moe_combine, moe_combine_backward and swiglu_backward_weights against the oracles.

The permutation, the combine (FP32 in slot order, bf16 rounded once) and dd (one FP32 product, rounded once
to bf16) are bit-exact.  A dot product dw over H elements is taken by 32 or 64 lanes (fewer only where each has
8 elements): at most 8 ceil(H / 256) sums in a lane and six levels over the lanes, each rounded (2^-24):
(8 ceil(H / 256) + 6) 2^-24 sum |dy d|.  The SwiGLU's dw is summed in float64 with terms within 2^-49 of theirs
and rounded once: 2^-24 |dw| + 2^-45 sum |terms|.
"""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
import workloads as W
from oracle import combine as oc, formats as of, gradients as og, permute as op
from helpers import assert_within, bf16_dev, bf16_host, dev, gpu_ready, host

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def routing(kind, T, E, k, seed, lost=0.0):
    ids, w = W.make_routing(kind, T, E, k, seed)
    if lost:
        drop = W.rng(seed, 77).random((T, k)) < lost
        ids = np.where(drop, W.rng(seed, 78).choice([-1, E, -2 ** 31, 2 ** 31 - 1], (T, k)), ids).astype(np.int32)
    return ids, w


def values(shape, dtype, seed, tensor):
    """(device tensor, float32 values)"""
    v = W.rng(seed, tensor).standard_normal(shape).astype(np.float32)
    if dtype == "f32":
        return dev(v), v
    b = W.f32_to_bf16_bits(v)
    return bf16_dev(b), W.bf16_bits_to_f32(b)


def filled(shape, dtype, byte=0xA5):
    return torch.full((int(np.prod(shape)) * (4 if dtype in (torch.float32, torch.int32) else 2),), byte, dtype=torch.uint8,
                      device="cuda").view(dtype).view(shape)


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


SHAPES = [(1, 1, 1, 8, "uniform"), (1, 128, 8, 2048, "softmax"), (2, 4, 4, 16, "uniform"), (61, 128, 8, 2048, "uniform"),
          (257, 24, 4, 520, "zipf"), (300, 16, 16, 1024, "uniform"), (40, 1024, 32, 264, "uniform"), (33, 64, 32, 24, "zipf"),
          (5, 8, 3, 4104, "uniform"), (3, 7, 5, 8200, "zipf"), (1000, 1, 1, 64, "uniform"), (1500, 300, 6, 72, "softmax"),
          (700, 129, 3, 512, "zipf"), (5000, 600, 2, 8, "uniform")]


@pytest.mark.parametrize("T,E,k,H,kind", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_permute(T, E, k, H, kind, dtype):
    print(f"[permute] T={T} E={E} k={k} H={H} {kind} {dtype}", flush=True)
    x, _ = values((T, H), dtype, 31, 1)
    for lost in (0.0, 0.3):
        ids, _ = routing(kind, T, E, k, 31, lost)
        off, r2t, t2r, bad = op.permute(ids, E)
        n = int(off[-1])
        out = {"rows": filled((T * k, H), DT[dtype]), "row_to_tk": filled((T * k,), torch.int32)}
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = pmg.moe_permute(x, dev(ids), E, out=out, dev_err=err)
        assert np.array_equal(host(got["expert_offsets"]), off)
        assert np.array_equal(host(got["tk_to_row"]), t2r)
        assert np.array_equal(host(got["row_to_tk"])[:n], r2t)
        assert torch.equal(got["rows"][:n].view(torch.uint8), x[dev(r2t.astype(np.int64)) // k].contiguous().view(torch.uint8))
        # rows behind the last one are left as they were
        assert same(got["rows"][n:].contiguous(), filled((T * k - n, H), DT[dtype]))
        assert same(got["row_to_tk"][n:].contiguous(), filled((T * k - n,), torch.int32))
        assert int(err) == (1 if bad else 0)
        maps = pmg.moe_permute(None, dev(ids), E)
        assert "rows" not in maps
        for name in ("expert_offsets", "tk_to_row"):
            assert torch.equal(maps[name], got[name])
        assert torch.equal(maps["row_to_tk"][:n], got["row_to_tk"][:n])


@pytest.mark.parametrize("T,E,k", [(40000, 128, 8), (33000, 512, 4), (70000, 16, 1), (20000, 1000, 31), (9000, 300, 32)])
def test_permute_long_lists(T, E, k):
    """Routing lists of many chunks: the same maps as the quantising permutation's."""
    ids, _ = routing("uniform", T, E, k, 32, 0.01)
    x, _ = values((T, 16), "bf16", 32, 1)
    ref = pmg.nvfp4_quantize_permute(x, dev(ids), E)
    got = pmg.moe_permute(x, dev(ids), E)
    n = int(ref["expert_offsets"][-1])
    for name in ("expert_offsets", "tk_to_row"):
        assert torch.equal(got[name], ref[name]), name
    assert torch.equal(got["row_to_tk"][:n], ref["row_to_tk"][:n])
    assert torch.equal(got["rows"][:n], x[ref["row_to_tk"][:n].long() // k])


@pytest.mark.parametrize("T,E,k,H,kind", SHAPES)
def test_combine(T, E, k, H, kind):
    print(f"[combine] T={T} E={E} k={k} H={H} {kind}", flush=True)
    for lost in (0.0, 0.3, 1.0):
        ids, w = routing(kind, T, E, k, 33, lost)
        _, _, t2r, _ = op.permute(ids, E)
        for dt in ("bf16", "f32"):
            d, dv = values((T * k, H), dt, 33, 2)
            for weights in (None, w):
                bits, acc = oc.unpermute_combine_ref(dv, t2r, k, weights)
                tw = None if weights is None else dev(w)
                y = pmg.moe_combine(d, dev(t2r), k, tw)
                assert y.dtype == torch.bfloat16 and np.array_equal(bf16_host(y), bits)
                assert np.array_equal(host(pmg.moe_combine(d, dev(t2r), k, tw, out_dtype=torch.float32)), acc)
                if dt == "f32":
                    assert same(y, pmg.unpermute_combine(d, dev(t2r), k, tw))


@pytest.mark.parametrize("T,E,k,H,kind", SHAPES)
@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("td", ["bf16", "f32"])
def test_combine_backward(T, E, k, H, kind, ty, td):
    print(f"[combine backward] T={T} E={E} k={k} H={H} {kind} {ty} {td}", flush=True)
    dy, gv = values((T, H), ty, 34, 1)
    d, dv = values((T * k, H), td, 34, 2)
    for lost, weighted in ((0.0, True), (0.3, True), (0.3, False)):
        ids, w = routing(kind, T, E, k, 34, lost)
        off, r2t, t2r, _ = op.permute(ids, E)
        n = int(off[-1])
        tw = dev(w) if weighted else None
        buf = filled((T * k, H), DT[td])
        dd, dw = pmg.moe_combine_backward(dy, d, dev(t2r), k, tw, dd=buf)
        assert dd is buf
        want = gv[r2t // k] * (w.reshape(-1)[r2t, None] if weighted else np.float32(1))
        if td == "f32":
            assert np.array_equal(host(dd)[:n], want)
        else:
            assert np.array_equal(bf16_host(dd)[:n], of.round_to_bf16(want))
        assert same(dd[n:].contiguous(), filled((T * k - n, H), DT[td]))
        _, ref = og.combine_backward(gv, dv, t2r, k)
        _, size = og.combine_backward(np.abs(gv), np.abs(dv), t2r, k)
        assert_within(host(dw), ref, (8 * -(-H // 256) + 6) * U * size + 2.0 ** -140, "dw")
        assert not host(dw)[t2r.reshape(T, k) < 0].any()
        # either result alone
        only, none = pmg.moe_combine_backward(dy, None, dev(t2r), k, tw, dd=filled((T * k, H), DT[td]))
        assert none is None and same(only, dd)
        none, alone = pmg.moe_combine_backward(dy, d, dev(t2r), k, tw, want_dd=False)
        assert none is None and torch.equal(alone, dw)


def test_combine_of_masked_rows_holding_infinities_and_nan():
    """What lies in rows that no entry names reaches no result; what lies in a row that one names does."""
    T, k, E, H = 9, 3, 5, 64
    ids, w = routing("uniform", T, E, k, 35)
    ids[2] = -1
    off, r2t, t2r, _ = op.permute(ids, E)
    n = int(off[-1])
    for dt in ("bf16", "f32"):
        d, _ = values((T * k, H), dt, 35, 1)
        d[n:] = float("nan")
        dy, _ = values((T, H), dt, 35, 2)
        dy[2] = float("inf")                       # of a token without rows
        y = pmg.moe_combine(d, dev(t2r), k, dev(w))
        assert y.isfinite().all() and not y[2].any()
        dd, dw = pmg.moe_combine_backward(dy, d, dev(t2r), k, dev(w))
        assert dd[:n].isfinite().all() and dw.isfinite().all() and not dw[2].any()
        d[int(t2r[0]), 7] = float("nan")
        assert int(pmg.moe_combine(d, dev(t2r), k, dev(w)).isnan().sum()) == 1
        _, dw = pmg.moe_combine_backward(dy, d, dev(t2r), k, dev(w))
        assert bool(dw[0, 0].isnan()) and int(dw.isnan().sum()) == 1


def test_bad_map_entries_are_skipped():
    T, k, H = 6, 2, 40
    t2r = np.array([0, 12, -3, 2 ** 31 - 1, 4, 5, -2 ** 31, 1, 2, 3, 100, 6], np.int32)
    d, dv = values((T * k, H), "f32", 36, 1)
    dy, gv = values((T, H), "f32", 36, 2)
    got = host(pmg.moe_combine(d, dev(t2r), k, out_dtype=torch.float32))
    ok = (t2r >= 0) & (t2r < 12)
    clean = np.where(ok, t2r, -1)
    assert np.array_equal(got, oc.unpermute_combine_ref(dv, clean, k)[1])
    dd, dw = pmg.moe_combine_backward(dy, d, dev(t2r), k, dd=torch.zeros_like(d))
    want, ref = og.combine_backward(gv, dv, clean, k)
    assert np.array_equal(host(dd), want.astype(np.float32))
    assert_within(host(dw), ref, 14 * U * og.combine_backward(np.abs(gv), np.abs(dv), clean, k)[1], "dw")
    assert not host(dw).reshape(-1)[~ok].any()


@pytest.mark.parametrize("T,E,k,I,kind", [(1, 128, 8, 768, "softmax"), (61, 128, 8, 768, "uniform"), (257, 24, 4, 264, "zipf"),
                                          (40, 64, 32, 8, "uniform"), (33, 16, 4, 384, "uniform"), (17, 8, 2, 128, "zipf"), (9, 4, 2, 2056, "uniform"), (5, 1, 1, 256, "uniform")])
def test_swiglu_backward_weights(T, E, k, I, kind):
    print(f"[swiglu backward] T={T} E={E} k={k} I={I} {kind}", flush=True)
    R = T * k
    gu, guv = values((R, 2 * I), "f32", 37, 1)
    dh, dhv = values((R, I), "f32", 37, 2)
    for lost in (0.0, 0.4, 1.0):
        ids, w = routing(kind, T, E, k, 37, lost)
        off, r2t, t2r, _ = op.permute(ids, E)
        n = int(off[-1])
        full = np.full(R, 2 ** 31 - 1, np.int32)
        full[:n] = r2t
        a, b = filled((R, 2 * I), torch.bfloat16), filled((R, 2 * I), torch.bfloat16)
        pmg.swiglu_backward(gu, dh, dev(off), dev(w.reshape(-1)), dev(full), dgu=a)
        dgu, dw = pmg.swiglu_backward_weights(gu, dh, dev(off), dev(w), dev(full), dev(t2r), dgu=b)
        assert dgu is b and same(a, b) and dw.shape == (T, k)
        want = og.swiglu_weight_grad(guv, dhv, full, n)
        size = og.swiglu_weight_grad(np.abs(guv), np.abs(dhv), full, n)
        assert_within(host(dw).reshape(-1), want, U * np.abs(want) + 2.0 ** -45 * size, "dw")
        assert not host(dw).reshape(-1)[t2r < 0].any()


def test_ids_maps_and_weights_that_start_anywhere():
    T, E, k, H = 41, 9, 3, 64
    x, _ = values((T, H), "bf16", 38, 1)
    ids, w = routing("uniform", T, E, k, 38)
    ref = pmg.moe_permute(x[1:].contiguous(), dev(ids[1:]), E)
    i = lambda n: torch.empty(n + 3, dtype=torch.int32, device="cuda")[3:]
    R = (T - 1) * k
    got = pmg.moe_permute(x[1:], dev(ids)[1:], E, out={"expert_offsets": i(E + 1), "row_to_tk": i(R), "tk_to_row": i(R)})
    for n in ref:
        assert torch.equal(got[n], ref[n]), n
    tw = dev(w)[1:]
    assert torch.equal(pmg.moe_combine(ref["rows"], got["tk_to_row"], k, tw),
                       pmg.moe_combine(ref["rows"], ref["tk_to_row"], k, tw.clone()))
    dw = torch.empty(R + 1, dtype=torch.float32, device="cuda")[1:]
    a = pmg.moe_combine_backward(x[1:], ref["rows"], got["tk_to_row"], k, tw, dw=dw)
    b = pmg.moe_combine_backward(x[1:], ref["rows"], ref["tk_to_row"], k, tw.clone())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].view(-1), b[1].view(-1))


def test_empty_batches():
    e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")
    i = lambda *s: e(*s, dt=torch.int32)
    got = pmg.moe_permute(e(0, 16), i(0, 2), 4)
    assert got["rows"].shape == (0, 16) and not got["expert_offsets"].any()
    assert not pmg.moe_permute(None, i(0, 2), 4)["expert_offsets"].any()
    assert pmg.moe_combine(e(0, 16), i(0), 2).shape == (0, 16)
    dd, dw = pmg.moe_combine_backward(e(0, 16), e(0, 16), i(0), 2, e(0, 2))
    assert dd.shape == (0, 16) and dw.shape == (0, 2)
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    assert pmg.swiglu_backward_weights(e(0, 16), e(0, 8), off, e(0, 2), i(0), i(0))[1].shape == (0, 2)


def test_refusals():
    x, ids = torch.zeros(4, 16, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    d, t2r = torch.zeros(8, 16, device="cuda"), torch.arange(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="one row per token"):
        pmg.moe_permute(x[:3], ids, 4)
    with pytest.raises(ValueError, match="holds"):
        pmg.moe_permute(x, ids, 4, out={"rows": x})
    with pytest.raises(TypeError):
        pmg.moe_permute(x, ids, 4, out={"rows": d.bfloat16()})
    with pytest.raises(pmg.NVFP4Error, match="workspace"):
        pmg.moe_permute(None, ids.repeat(2000, 1), 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pmg.NVFP4Error):
        pmg.moe_permute(torch.zeros(4, 12, device="cuda"), ids, 4)
    with pytest.raises(ValueError, match="T \\* k"):
        pmg.moe_combine(d, t2r, 3)
    with pytest.raises(ValueError, match="holds"):
        pmg.moe_combine(x, t2r, 2)
    with pytest.raises(TypeError):
        pmg.moe_combine(d, t2r, 2, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="row length"):
        pmg.moe_combine_backward(x, torch.zeros(16, 8, device="cuda"), t2r, 2)
    with pytest.raises(ValueError, match="needs d"):
        pmg.moe_combine_backward(x, None, t2r, 2, want_dd=False)
    with pytest.raises(pmg.NVFP4Error):
        pmg.moe_combine_backward(x, d, t2r, 2, dd=d)
    with pytest.raises(ValueError, match="contiguous"):
        pmg.moe_combine(d.t().contiguous().t(), t2r, 2)


def test_offsets_past_32_bits():
    """More than 2^32 bytes and 2^31 elements of routed rows: the last rows against torch."""
    T, k, E, H = 70000, 4, 8, 8192
    print(f"[permute] {T * k} rows of {H}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1)[1].int()
    w = torch.rand((T, k), generator=g, device="cuda")
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.float32).bfloat16()
    got = pmg.moe_permute(x, ids, E)
    rows, r2t, t2r = got["rows"], got["row_to_tk"].long(), got["tk_to_row"]
    at = torch.tensor([0, 1, T * k // 2, T * k - 3, T * k - 1], device="cuda")
    assert torch.equal(rows[at], x[r2t[at] // k])
    y = pmg.moe_combine(rows, t2r, k, w, out_dtype=torch.float32)
    for t in (0, T // 2, T - 1):      # k copies of x[t]: the sum of its weights, in slot order
        acc = w[t, 0] * x[t].float()
        for s in range(1, k):
            acc = acc + w[t, s] * x[t].float()
        assert torch.equal(y[t], acc)
    dd, dw = pmg.moe_combine_backward(x, rows, t2r, k, w, dd=torch.empty_like(rows))
    assert torch.equal(dd[at], (x[r2t[at] // k].float() * w.view(-1)[r2t[at]][:, None]).bfloat16())
    sq = (x[[0, T // 2, T - 1]].double() ** 2).sum(1)
    for j, t in enumerate((0, T // 2, T - 1)):
        assert (dw[t].double() - sq[j]).abs().max() <= (8 * H / 512 + 6) * U * float(sq[j])
