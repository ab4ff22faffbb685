"""The FP8 operators and the BF16 weight gradient as a MoE layer uses them together.

Forward: routing maps, activations quantised per token, gate_up with the rows gathered,
weighted SwiGLU + quantise, down, combine.  Backward: input gradients through the
transposed weight codes, SwiGLU backward, BF16 weight gradients of both products.  Every
stage's GPU output is the next oracle stage's input.

Bars: codes and scales bit-exact; FP32 products within 2e-5 sum |a w|; the gate_up
product in BF16 within 7 2^-13 sum |a w| more and half a bf16 step (2^-8 relative); the
weight gradients within (n + 1) 2^-24 sum |g x| over n rows.
"""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
import workloads as W
from oracle import combine as oc, formats as of, fp8 as o8, permute as op
from helpers import assert_within, bf16_dev, bf16_host, dev, gpu_ready, host

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]


class Layer:
    """Inputs and outputs of one layer step; step() enqueues it on the current stream."""

    def __init__(self, T, H, E, k, I, kind, seed):
        self.T, self.H, self.E, self.k, self.I = T, H, E, k, I
        R = T * k
        self.xb, self.dyb = W.activations(T, H, seed), W.gaussian_bf16((T, H), 1.0, seed, 4)
        self.wgub, self.wdb = W.gaussian_bf16((E, 2 * I, H), 0.02, seed, 2), W.gaussian_bf16((E, H, I), 0.02, seed, 3)
        self.ids, self.tw = W.make_routing(kind, T, E, k, seed)
        self.x, self.dy, self.wgu, self.wd = (bf16_dev(b) for b in (self.xb, self.dyb, self.wgub, self.wdb))
        self.ids_d, self.tw_d = dev(self.ids), dev(self.tw.reshape(-1))
        u8, f32, b16, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32
        new = lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda")
        nb = o8.blocks
        self.ws = new(u8, pmg.permute_workspace_size(T, k, E))
        self.perm = {"codes": new(u8, R, H // 2), "bscales": new(u8, R, H // 16), "rscales": new(f32, R),
                     "expert_offsets": new(i32, E + 1), "row_to_tk": new(i32, R), "tk_to_row": new(i32, R)}
        weights = lambda N, K: {"codes": new(u8, E, N, K), "scales": new(f32, E, nb(N), nb(K)),
                                "codes_t": new(u8, E, K, N), "scales_t": new(f32, E, nb(K), nb(N))}
        self.qgu, self.qd = weights(2 * I, H), weights(H, I)
        self.o = {"xc": new(u8, T, H), "xs": new(f32, nb(H), T), "gu": new(b16, R, 2 * I), "hc": new(u8, R, I),
                  "hs": new(f32, nb(I), R), "h": new(b16, R, I), "d": new(f32, R, H), "y": new(b16, T, H),
                  "dyc": new(u8, T, H), "dys": new(f32, nb(H), T), "dh": new(f32, R, I), "gu32": new(f32, R, 2 * I),
                  "dgu": new(b16, R, 2 * I), "gc": new(u8, R, 2 * I), "gs": new(f32, nb(2 * I), R), "dxp": new(f32, R, H),
                  "dx": new(b16, T, H), "dwgu": new(f32, E, 2 * I, H), "dwd": new(b16, E, H, I)}
        self.outs = {**self.o, **{f"qgu.{n}": t for n, t in self.qgu.items()}, **{f"qd.{n}": t for n, t in self.qd.items()}}

    def step(self):
        o, k = self.o, self.k
        q = pmg.nvfp4_quantize_permute(self.x, self.ids_d, self.E, workspace=self.ws, out=self.perm)   # the maps
        off, r2t, t2r = q["expert_offsets"], q["row_to_tk"], q["tk_to_row"]
        gu, d = self.qgu, self.qd
        pmg.fp8_quantize_weights(self.wgu, transposed=True, out=gu)
        pmg.fp8_quantize_weights(self.wd, transposed=True, out=d)
        pmg.fp8_quantize_rows(self.x, codes=o["xc"], scales=o["xs"])
        pmg.fp8_grouped_gemm_gather(o["xc"], o["xs"], r2t, k, off, gu["codes"], gu["scales"], c=o["gu"])
        pmg.fp8_swiglu_quantize(o["gu"], off, self.tw_d, r2t, h_out=True,
                                out={"codes": o["hc"], "scales": o["hs"], "h": o["h"]})
        pmg.fp8_grouped_gemm(o["hc"], o["hs"], off, d["codes"], d["scales"], c=o["d"])
        pmg.unpermute_combine(o["d"], t2r, k, y=o["y"])
        pmg.fp8_quantize_rows(self.dy, codes=o["dyc"], scales=o["dys"])
        pmg.fp8_grouped_gemm_gather(o["dyc"], o["dys"], r2t, k, off, d["codes_t"], d["scales_t"], c=o["dh"])
        o["gu32"].copy_(o["gu"])
        pmg.swiglu_backward(o["gu32"], o["dh"], off, self.tw_d, r2t, dgu=o["dgu"])
        pmg.fp8_quantize_rows(o["dgu"], off, o["gc"], o["gs"])
        pmg.fp8_grouped_gemm(o["gc"], o["gs"], off, gu["codes_t"], gu["scales_t"], c=o["dxp"])
        pmg.unpermute_combine(o["dxp"], t2r, k, y=o["dx"])
        pmg.bf16_grouped_gemm_wgrad(o["dgu"], self.x, off, r2t, k, "x", c=o["dwgu"])
        pmg.bf16_grouped_gemm_wgrad(self.dy, o["h"], off, r2t, k, "g", c=o["dwd"])


def _same(a, b):
    return np.array_equal(np.ascontiguousarray(a).view(np.uint8), np.ascontiguousarray(b).view(np.uint8))


def _gemm(got, a, off, w, src=None, bf16=False, what=""):
    ref, bound = o8.grouped_gemm_ref(*a, off, *w, row_source=src)
    if bf16:
        bound = bound * (1 + 7 * 2.0 ** -13 / o8.REL_TOL)
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    print(f"  {what} err/bound", assert_within(got.astype(np.float64), ref, bound + 1e-300, what), flush=True)


@pytest.mark.parametrize("T,H,E,k,I,kind", [(1, 256, 8, 2, 144, "uniform"), (13, 272, 16, 4, 80, "zipf"),
                                            (300, 528, 6, 3, 256, "zipf"), (515, 512, 16, 4, 384, "softmax")])
def test_layer_forward_and_backward(T, H, E, k, I, kind):
    print(f"[fp8 chain] T={T} H={H} E={E} k={k} I={I} {kind}", flush=True)
    L = Layer(T, H, E, k, I, kind, 7)
    L.step()
    torch.cuda.synchronize()
    off, r2t, t2r, _ = op.permute(L.ids, E)
    assert np.array_equal(host(L.perm["expert_offsets"]), off) and np.array_equal(host(L.perm["row_to_tk"]), r2t)
    src = r2t.astype(np.int64) // k
    h = {n: (of.bf16_to_f32(bf16_host(t)) if t.dtype == torch.bfloat16 else host(t)) for n, t in L.outs.items()}

    for name, wb in (("qgu", L.wgub), ("qd", L.wdb)):
        c, s = o8.quantize_weights(of.bf16_to_f32(wb))
        assert _same(h[name + ".codes"], c) and _same(h[name + ".scales"], s)
        assert _same(h[name + ".codes_t"], c.swapaxes(1, 2)) and _same(h[name + ".scales_t"], s.swapaxes(1, 2))
    w = {n: (h[n + ".codes"], h[n + ".scales"]) for n in ("qgu", "qd")}
    wt = {n: (h[n + ".codes_t"], h[n + ".scales_t"]) for n in ("qgu", "qd")}

    for got, b in ((("xc", "xs"), L.xb), (("dyc", "dys"), L.dyb)):
        assert all(_same(h[n], v) for n, v in zip(got, o8.quantize_rows(of.bf16_to_f32(b))))
    _gemm(h["gu"], (h["xc"], h["xs"]), off, w["qgu"], src, True, "gate_up")

    ref = o8.swiglu(h["gu"], L.tw.reshape(-1)[r2t])
    assert_within(h["h"], ref, (2.0 ** -8 + 2.0 ** -19) * np.abs(ref) + 2.0 ** -133, "swiglu h")
    val = o8.dequantize_rows(h["hc"], h["hs"])
    s64 = np.repeat(np.stack([np.abs(ref[:, j:j + 128]).max(1) / 448 for j in range(0, I, 128)], 1), 128, 1)[:, :I]
    assert_within(val, ref, np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * s64) * (1 + 2.0 ** -17) + 2.0 ** -18 * np.abs(ref), "swiglu codes")
    _gemm(h["d"], (h["hc"], h["hs"]), off, w["qd"], None, False, "down")
    assert np.array_equal(bf16_host(L.o["y"]), oc.unpermute_combine_ref(h["d"], t2r, k)[0])

    _gemm(h["dh"], (h["dyc"], h["dys"]), off, wt["qd"], src, False, "dgrad down")
    assert all(_same(h[n], v) for n, v in zip(("gc", "gs"), o8.quantize_rows(h["dgu"])))
    _gemm(h["dxp"], (h["gc"], h["gs"]), off, wt["qgu"], None, False, "dgrad gate_up")
    assert np.array_equal(bf16_host(L.o["dx"]), oc.unpermute_combine_ref(h["dxp"], t2r, k)[0])

    n = np.diff(off)[:, None, None] + 1.0
    x, dy = of.bf16_to_f32(L.xb), of.bf16_to_f32(L.dyb)
    ref, mag = o8.wgrad_ref(h["dgu"], x[src], off)
    assert_within(h["dwgu"].astype(np.float64), ref, n * 2.0 ** -24 * mag, "dW gate_up")
    ref, mag = o8.wgrad_ref(dy[src], h["h"], off)
    bound = n * 2.0 ** -24 * mag
    assert_within(h["dwd"].astype(np.float64), ref, bound + 2.0 ** -8 * (np.abs(ref) + bound), "dW down")


def _clones(L):
    return {n: t.clone() for n, t in L.outs.items()}


def _equal(a, b, what):
    for n in a:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), f"{what}: {n}"


@pytest.mark.parametrize("T", [9, 400])
def test_graph_replays_match_eager(T):
    """The whole step captured; three replays, eager work clobbering every output between them."""
    L = Layer(T, 256, 8, 4, 128, "softmax", 5)
    L.step()
    torch.cuda.synchronize()
    ref = _clones(L)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.step()
    torch.cuda.synchronize()
    for rep in range(3):
        for t in L.outs.values():
            t.view(torch.uint8).fill_(0x5A + rep)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _equal(ref, L.outs, f"replay {rep}")
    # the graph keeps no result: new inputs in the same buffers give what an eager step gives on them
    L.x.copy_(L.x.flip(0).contiguous())
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    got = _clones(L)
    L.step()
    torch.cuda.synchronize()
    _equal(got, L.outs, "new input")


def test_two_streams_at_once():
    """Two layers on two streams at the same time give what each gives alone."""
    layers = [Layer(600, 512, 16, 4, 256, kind, s) for kind, s in (("softmax", 3), ("zipf", 4))]
    for L in layers:
        L.step()
    torch.cuda.synchronize()
    refs = [_clones(L) for L in layers]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for s, L in zip(streams, layers):
            with torch.cuda.stream(s):
                for t in L.outs.values():
                    t.view(torch.uint8).fill_(rep)
                L.step()
    torch.cuda.synchronize()
    for L, ref in zip(layers, refs):
        _equal(ref, L.outs, "two streams")


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_a_row_alone_and_in_a_batch(out):
    """A row's bits do not depend on what else is in the call: one row, up to 128 routed rows, many."""
    E, N, K, T = 5, 328, 1040, 700
    r = np.random.default_rng(6)
    a, sa = (dev(v) for v in o8.quantize_rows(of.bf16_to_f32(W.activations(T, K, 6))))
    w, sw = (dev(v) for v in o8.quantize_weights((0.02 * r.standard_normal((E, N, K))).astype(np.float32)))
    e = r.integers(0, E, T).astype(np.int32)

    def run(tokens):
        order = tokens[np.argsort(e[tokens], kind="stable")]
        off = np.concatenate([[0], np.cumsum(np.bincount(e[order], minlength=E))]).astype(np.int32)
        c = pmg.fp8_grouped_gemm_gather(a, sa, dev(order.astype(np.int32)), 1, dev(off), w, sw, out_dtype=out)
        return {int(t): c[i] for i, t in enumerate(order)}

    full = run(np.arange(T))
    for tokens in ([17], [699, 3], np.arange(100, 227), np.arange(60, 188), np.arange(20, 149), r.permutation(T)[:300]):
        for t, row in run(np.asarray(tokens)).items():
            assert torch.equal(row, full[t]), f"token {t} in a batch of {len(tokens)}"


def test_weight_gradient_against_differences():
    """dW against central differences of sum(dy * (x W^T)), which is linear in W, so exact in float64."""
    T, H, E, k, I = 12, 32, 4, 2, 16
    ids, _ = W.make_routing("uniform", T, E, k, 2)
    off, r2t, _, _ = op.permute(ids, E)
    xb, gb = W.activations(T, H, 2), W.gaussian_bf16((T * k, I), 1.0, 2, 4)
    x, g, src = of.bf16_to_f32(xb).astype(np.float64), of.bf16_to_f32(gb).astype(np.float64), r2t.astype(np.int64) // k
    got = host(pmg.bf16_grouped_gemm_wgrad(bf16_dev(gb), bf16_dev(xb), dev(off), dev(r2t), k, "x"))
    expert = np.searchsorted(off, np.arange(T * k), side="right") - 1
    w = np.random.default_rng(1).standard_normal((E, I, H))
    loss = lambda v: float(sum((g[i] * (v[expert[i]] @ x[src[i]])).sum() for i in range(T * k)))
    for at in ((0, 0, 0), (1, 3, 31), (2, 15, 7), (3, 8, 16), (3, 15, 31)):
        step = np.zeros_like(w)
        step[at] = 0.5
        assert abs((loss(w + step) - loss(w - step)) - got[at]) <= 1e-4 * max(1.0, abs(got[at]))


# ------------------------------------------------------------------ offsets past 32 bits
def _some(*shape):
    """bf16 on the device without a float32 copy of it."""
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    t.view(torch.int16).random_(0x3C00, 0x3F80)
    return t


def test_far_rows_of_the_quantisers():
    rows, K = 66000, 65536                                      # 4.3e9 elements
    x = _some(rows, K)
    codes, scales = pmg.fp8_quantize_rows(x)
    for r in (0, 32767, rows - 1):
        c, s = pmg.fp8_quantize_rows(x[r:r + 1].clone())
        assert torch.equal(codes[r], c[0]) and torch.equal(scales[:, r], s[:, 0])
    I = K // 2
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    codes, scales, _ = pmg.fp8_swiglu_quantize(x, off)
    for r in (0, rows - 1):
        c, s, _ = pmg.fp8_swiglu_quantize(x[r:r + 1].clone(), one)
        assert torch.equal(codes[r], c[0]) and torch.equal(scales[:, r], s[:, 0])


def test_far_experts_of_the_weights_and_the_product():
    E, N, K = 36, 2048, 65536                                   # 4.8e9 codes
    w = _some(E, N, K)
    c, s, ct, st = pmg.fp8_quantize_weights(w, transposed=True)
    last = pmg.fp8_quantize_weights(w[-1:].clone(), transposed=True)
    for got, ref in zip((c, s, ct, st), last):
        assert torch.equal(got[-1], ref[0])
    del w, ct, st
    for R in (40, 400, 600):
        a, sa = pmg.fp8_quantize_rows(_some(R, K))
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[-1] = R
        one = torch.tensor([0, R], dtype=torch.int32, device="cuda")
        for dt in (torch.float32, torch.bfloat16):
            assert torch.equal(pmg.fp8_grouped_gemm(a, sa, off, c, s, out_dtype=dt),
                               pmg.fp8_grouped_gemm(a, sa, one, c[-1:].clone(), s[-1:].clone(), out_dtype=dt))


def test_far_rows_of_the_product():
    """Activations past 4 GiB (in order), and an output past 4 GiB."""
    for R, K, N in ((70000, 65536, 16), (70000, 32, 16400)):
        a = torch.randint(0x20, 0x40, (R, K), dtype=torch.uint8, device="cuda")
        sa = torch.rand(o8.blocks(K), R, device="cuda")
        w = torch.randint(0x20, 0x40, (2, N, K), dtype=torch.uint8, device="cuda")
        sw = torch.rand(2, o8.blocks(N), o8.blocks(K), device="cuda")
        off = torch.tensor([0, 5, R], dtype=torch.int32, device="cuda")
        c = pmg.fp8_grouped_gemm(a, sa, off, w, sw)
        tail = R - 300
        ref = pmg.fp8_grouped_gemm(a[tail:].clone(), sa[:, tail:].clone(), torch.tensor([0, 0, 300], dtype=torch.int32, device="cuda"), w, sw)
        assert torch.equal(c[tail:], ref)
        del a, c


def test_far_rows_and_experts_of_the_weight_gradient():
    R, N = 1100000, 2048                                        # rows past 4 GiB, in order
    x, g = _some(R, N), _some(R, 16)
    off = torch.tensor([0, 3, R - 70, R], dtype=torch.int32, device="cuda")
    got = pmg.bf16_grouped_gemm_wgrad(g, x, off)
    ref = pmg.bf16_grouped_gemm_wgrad(g[-70:].clone(), x[-70:].clone(), torch.tensor([0, 0, 0, 70], dtype=torch.int32, device="cuda"))
    assert torch.equal(got[2], ref[2])
    del x, g
    E, M, N = 480, 1536, 1536                                   # an output past 4 GiB
    g, x = _some(2 * E, M), _some(2 * E, N)
    off = torch.arange(0, 2 * E + 1, 2, dtype=torch.int32, device="cuda")
    got = pmg.bf16_grouped_gemm_wgrad(g, x, off)
    for e in (0, E // 2, E - 1):
        ref = (g[2 * e:2 * e + 2].double().t().contiguous() @ x[2 * e:2 * e + 2].double())
        assert torch.allclose(got[e].double(), ref, rtol=2.0 ** -20, atol=0)
