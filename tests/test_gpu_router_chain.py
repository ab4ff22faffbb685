"""A MoE layer trained through its router: the router, the token sort, the experts' BF16 products, the weighted
SwiGLU or the weighted combine, and the gradients back to the logits, the tokens and the weights, clipped.

Two layers: the router's weights applied in the SwiGLU (gradient from swiglu_backward_weights) and in the
combine (moe_combine_backward).  Each stage is checked with the GPU's output of the stage before as its
input; the logits' gradient of the first layer also against float64 differentiation of the whole layer,
whose only FP32 stages before it are products: over n terms they are off by at most (n + 2) 2^-24 of the sum of
their absolute values, and that bound is carried through (|silu'| < 1.1).
"""
import numpy as np
import pytest
import torch

import precision_moe_gemm_amd as pmg
import workloads as W
from oracle import combine as oc, formats as of, gradients as og, permute as op, router as orr
from helpers import assert_within, bf16_dev, bf16_host, dev, gpu_ready, host

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_ready(), reason="needs a GPU")]

U = 2.0 ** -24
f32, b16, i32, u8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


class Layer:
    def __init__(self, T, H, E, k, I, seed, in_combine=False, renorm=True):
        self.dims, self.in_combine, self.renorm = (T, H, E, k, I), in_combine, renorm
        R = T * k
        self.lg = W.router_logits(T, E, seed)
        self.xb, self.dyb = W.activations(T, H, seed), W.gaussian_bf16((T, H), 1.0, seed, 4)
        self.wgub, self.wdb = W.gaussian_bf16((E, 2 * I, H), 0.05, seed, 2), W.gaussian_bf16((E, H, I), 0.05, seed, 3)
        self.logits, self.x, self.dy, self.wgu, self.wd = dev(self.lg), *map(bf16_dev, (self.xb, self.dyb, self.wgub, self.wdb))
        new = lambda dt, *shape: torch.zeros(shape, dtype=dt, device="cuda")
        self.perm = {"rows": new(b16, R, H), "expert_offsets": new(i32, E + 1), "row_to_tk": new(i32, R),
                     "tk_to_row": new(i32, R)}
        self.ws = new(u8, max(16, pmg.moe_permute_workspace_size(T, k, E)))
        self.q = {"codes": new(u8, R, I // 2), "bscales": new(u8, R, I // 16), "rscales": new(f32, R), "h": new(f32, R, I)}
        self.o = {"ids": new(i32, T, k), "w": new(f32, T, k), "gu": new(f32, R, 2 * I), "hb": new(b16, R, I),
                  "d": new(f32, R, H), "y": new(b16, T, H), "ddf": new(f32, R, H), "dd": new(b16, R, H), "dh": new(f32, R, I),
                  "dgu": new(b16, R, 2 * I), "dw": new(f32, T, k), "dxp": new(f32, R, H), "dx": new(f32, T, H),
                  "dwgu": new(f32, E, 2 * I, H), "dwd": new(b16, E, H, I), "dlogits": new(f32, T, E), "norm": new(f32, 1),
                  "cgu": new(f32, E, 2 * I, H), "cd": new(b16, E, H, I)}
        self.nws = new(u8, pmg.grad_workspace_size(2))
        self.outs = {**self.o, **self.perm, **self.q}

    def step(self):
        o, (T, H, E, k, I) = self.o, self.dims
        pmg.moe_router_topk(self.logits, k, self.renorm, o["ids"], o["w"])
        p = pmg.moe_permute(self.x, o["ids"], E, workspace=self.ws, out=self.perm)
        off, r2t, t2r = p["expert_offsets"], p["row_to_tk"], p["tk_to_row"]
        pmg.bf16_grouped_gemm(p["rows"], off, self.wgu, pmg.W_NK, o["gu"])
        tw = None if self.in_combine else o["w"]
        pmg.swiglu_quantize(o["gu"], off, tw, r2t, h_out=True, out=self.q)
        o["hb"].copy_(self.q["h"])
        pmg.bf16_grouped_gemm(o["hb"], off, self.wd, pmg.W_NK, o["d"])
        pmg.moe_combine(o["d"], t2r, k, o["w"] if self.in_combine else None, y=o["y"])
        if self.in_combine:
            pmg.moe_combine_backward(self.dy, o["d"], t2r, k, o["w"], dd=o["ddf"], dw=o["dw"])
            o["dd"].copy_(o["ddf"])
        else:
            pmg.moe_combine_backward(self.dy, None, t2r, k, dd=o["dd"])
        pmg.bf16_grouped_gemm(o["dd"], off, self.wd, pmg.W_KN, o["dh"])
        if self.in_combine:
            pmg.swiglu_backward(o["gu"], o["dh"], off, dgu=o["dgu"], row_to_tk=r2t)
        else:
            pmg.swiglu_backward_weights(o["gu"], o["dh"], off, o["w"], r2t, t2r, dgu=o["dgu"], dw=o["dw"])
        pmg.bf16_grouped_gemm(o["dgu"], off, self.wgu, pmg.W_KN, o["dxp"])
        pmg.moe_combine(o["dxp"], t2r, k, y=o["dx"])
        pmg.bf16_grouped_gemm_wgrad(o["dgu"], p["rows"], off, c=o["dwgu"])
        pmg.bf16_grouped_gemm_wgrad(o["dd"], o["hb"], off, c=o["dwd"])
        pmg.moe_router_topk_backward(o["dw"], o["ids"], o["w"], self.logits, self.renorm, o["dlogits"])
        pmg.grad_clip([o["dwgu"], o["dwd"]], 0.5, out=[o["cgu"], o["cd"]], norm=o["norm"], workspace=self.nws)


@pytest.mark.parametrize("in_combine,renorm", [(False, True), (True, True), (False, False)])
def test_layer_step(in_combine, renorm):
    T, H, E, k, I = 61, 64, 12, 4, 32
    L = Layer(T, H, E, k, I, 51, in_combine, renorm)
    L.step()
    o, p = L.o, L.perm
    ids, w = host(o["ids"]), host(o["w"])
    want_ids, w64 = orr.topk(L.lg, k, renorm)
    assert np.array_equal(ids, want_ids)
    dw_ = np.abs(w64) * 64 * U                      # (2 X + 32) 2^-24 with X < 16 for these logits
    assert np.ptp(L.lg) < 16
    assert_within(w, w64, dw_, "weights")
    off, r2t, t2r, bad = op.permute(ids, E)
    assert not bad and np.array_equal(host(p["expert_offsets"]), off) and np.array_equal(host(p["tk_to_row"]), t2r)
    assert np.array_equal(bf16_host(p["rows"]), L.xb[r2t // k])
    assert np.array_equal(bf16_host(o["y"]), oc.unpermute_combine_ref(host(o["d"]), t2r, k, w if in_combine else None)[0])
    dyv = W.bf16_bits_to_f32(L.dyb)
    if in_combine:
        assert np.array_equal(host(o["ddf"]), dyv[r2t // k] * w.reshape(-1)[r2t, None])
        _, ref = og.combine_backward(dyv, host(o["d"]), t2r, k)
        _, size = og.combine_backward(np.abs(dyv), np.abs(host(o["d"])), t2r, k)
        assert_within(host(o["dw"]), ref, 14 * U * size, "dw")
    else:
        assert np.array_equal(bf16_host(o["dd"]), L.dyb[r2t // k])
        ref = og.swiglu_weight_grad(host(o["gu"]), host(o["dh"]), r2t, T * k)
        size = og.swiglu_weight_grad(np.abs(host(o["gu"])), np.abs(host(o["dh"])), r2t, T * k)
        assert_within(host(o["dw"]).reshape(-1), ref, U * np.abs(ref) + 2.0 ** -45 * size, "dw")
    assert np.array_equal(host(o["dx"]), oc.unpermute_combine_ref(host(o["dxp"]), t2r, k)[1])
    dl = orr.topk_backward(host(o["dw"]), ids, w, L.lg, renorm)
    g64 = np.abs(host(o["dw"]).astype(np.float64))
    size = (np.abs(w) * g64).sum(1, keepdims=True)
    assert_within(host(o["dlogits"]), dl, 80 * U * (np.abs(dl) + (g64.max(1, keepdims=True) + size)), "dlogits")
    n, (cg, cd) = og.clip([host(o["dwgu"]), o["dwd"].double().cpu().numpy()], 0.5)
    assert_within(host(o["norm"]), np.array([n]), np.array([(U + 2.0 ** -40) * n]), "norm")
    assert_within(host(o["cgu"]), cg, 2.01 * U * np.abs(cg) + 2.0 ** -150, "clipped gate_up")
    assert_within(o["cd"].double().cpu().numpy(), cd, 2.0 ** -8 * 1.001 * np.abs(cd) + 2.0 ** -134, "clipped down")


def test_logits_gradient_against_float64_differentiation():
    T, H, E, k, I = 23, 64, 6, 3, 32
    L = Layer(T, H, E, k, I, 52)
    L.step()
    ids, r2t = host(L.o["ids"]).astype(np.int64), host(L.perm["row_to_tk"])
    lg = torch.tensor(L.lg, dtype=torch.float64, requires_grad=True)
    val = lambda b: torch.tensor(W.bf16_bits_to_f32(b).astype(np.float64))
    x, dy, wgu, wd = map(val, (L.xb, L.dyb, L.wgub, L.wdb))
    t = torch.arange(T)[:, None]
    idt = torch.tensor(ids)
    w = torch.softmax(lg[t, idt], dim=1)
    gu = torch.einsum("th,tknh->tkn", x, wgu[idt])                  # [T, k, 2I] on the CPU
    g, u = gu[..., :I], gu[..., I:]
    h = w[..., None] * g * torch.sigmoid(g) * u
    y = torch.einsum("tki,tkhi->th", h, wd[idt])
    (y * dy).sum().backward()
    want = lg.grad.numpy()
    # the bound: products, then dw, then the router's own roundings
    ax, ady, awgu, awd = (v.abs() for v in (x, dy, wgu, wd))
    dgu = (H + 2) * U * torch.einsum("th,tknh->tkn", ax, awgu[idt])
    dh, adh = torch.einsum("th,tkhi->tki", dy, wd[idt]).abs(), torch.einsum("th,tkhi->tki", ady, awd[idt])
    ddh = (H + 2) * U * adh
    silu = (g * torch.sigmoid(g)).detach().abs()
    gu_, ua = gu.detach(), u.detach().abs()
    dsu = 1.1 * dgu[..., :I] * (ua + dgu[..., I:]) + silu * dgu[..., I:]
    ddw = ((ddh + dh) * dsu + ddh * silu * ua).sum(-1).numpy()
    dw64 = (torch.einsum("th,tkhi->tki", dy, wd[idt]) * (g * torch.sigmoid(g) * u).detach()).sum(-1).numpy()
    wv = w.detach().numpy()
    size = (wv * (np.abs(dw64) + ddw)).sum(1, keepdims=True)
    bound = np.zeros_like(want)
    entry = wv * (ddw + (wv * ddw).sum(1, keepdims=True)) * 1.001 + 80 * 2 * U * wv * (np.abs(dw64) + size)
    np.add.at(bound, (np.arange(T)[:, None], ids), entry)
    ratio = assert_within(host(L.o["dlogits"]), want, bound, "dlogits of the whole layer")
    print(f"  worst err/bound {ratio:.3g}", flush=True)
    assert (bound[want != 0] < 0.05 * np.abs(want).max()).all()      # the bound says something


def test_graph_replays_match_eager():
    for in_combine in (False, True):
        L = Layer(300, 128, 16, 4, 64, 53, in_combine)
        print(f"[graph] layer step, weights in the {'combine' if in_combine else 'SwiGLU'}", flush=True)
        L.step()
        torch.cuda.synchronize()
        ref = {n: v.clone() for n, v in L.outs.items()}
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            L.step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.step()
        skip = {"ddf"} if not in_combine else set()     # not written in that layer
        for rep in range(3):
            for n, v in L.outs.items():
                if n not in skip:
                    v.view(u8).fill_(0xA5 + rep)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for n, v in L.outs.items():
                assert torch.equal(v.view(u8), ref[n].view(u8)), f"replay {rep}: {n}"


def test_captured_calls_that_allocate():
    """Outputs and workspaces left to the calls, inside a captured graph, for a short and a long routing list."""
    for T in (50, 3000):
        lg = [dev(W.router_logits(T, 16, 56 + j)) for j in range(2)]
        x, dy = (bf16_dev(W.gaussian_bf16((T, 64), 1.0, 56, j)) for j in range(2))
        logits = lg[0].clone()

        def run():
            ids, w = pmg.moe_router_topk(logits, 4)
            p = pmg.moe_permute(x, ids, 16)
            y = pmg.moe_combine(p["rows"], p["tk_to_row"], 4, w, out_dtype=torch.float32)
            dd, dw = pmg.moe_combine_backward(dy, p["rows"], p["tk_to_row"], 4, w)
            dl = pmg.moe_router_topk_backward(dw, ids, w, logits)
            norm, out = pmg.grad_clip([dl, dd], 0.1)
            return [ids, w, *p.values(), y, dd, dw, dl, norm, *out, pmg.grad_norm([dl])]

        want = []
        for v in lg:
            logits.copy_(v)
            want.append([t.clone() for t in run()])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        for rep in range(4):
            logits.copy_(lg[rep % 2])
            junk = [torch.full_like(t, 3) for t in got]     # the program's own allocations in between
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[rep % 2])), f"T={T} replay {rep}"
            del junk


def test_two_streams_at_once():
    a, b = Layer(300, 128, 16, 4, 64, 54), Layer(2000, 128, 64, 8, 64, 55, True)
    want = []
    for L in (a, b):
        L.step()
        torch.cuda.synchronize()
        want.append({n: v.clone() for n, v in L.outs.items()})
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(4):
        for L in (a, b):
            for n, v in L.outs.items():
                if n != "ddf":
                    v.view(u8).fill_(0x5A)
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(s1):
                a.step()
            with torch.cuda.stream(s2):
                b.step()
        torch.cuda.synchronize()
        for L, ref in ((a, want[0]), (b, want[1])):
            for n, v in L.outs.items():
                assert torch.equal(v.view(u8), ref[n].view(u8)), n
