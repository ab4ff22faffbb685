"""Host checks of the router, permutation, combine and gradient entry points: every refusal returns its
status before anything is enqueued (no device pointer is ever dereferenced, no GPU needed)."""
import ctypes

import pytest
import torch

import precision_moe_gemm_amd as pmg

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_LAUNCH, ERR_ARG = range(7)
P = 0x100000   # aligned, never dereferenced
Q = 0x200000


def test_router(lib):
    fwd = lambda **kw: lib.moe_router_topk(kw.get("l", P), kw.get("dt", 0), kw.get("T", 4), kw.get("E", 16), kw.get("k", 4),
                                           kw.get("rn", 1), kw.get("ids", P), kw.get("w", P), None)
    bwd = lambda **kw: lib.moe_router_topk_backward(
        kw.get("l", P), kw.get("dt", 0), kw.get("ids", P), kw.get("w", P), kw.get("dw", P), kw.get("T", 4),
        kw.get("E", 16), kw.get("k", 4), kw.get("rn", 1), kw.get("dl", Q), None)
    for f in (fwd, bwd):
        for kw in ({"dt": 2}, {"dt": -1}, {"rn": 2}, {"rn": -1}):
            assert f(**kw) == ERR_ARG, kw
        for kw in ({"T": -1}, {"E": 0}, {"E": 1025}, {"k": 0}, {"k": 17}, {"E": 64, "k": 33}, {"T": 1 << 24}, {"T": 1 << 26, "k": 1}, {"T": 1 << 62}):
            assert f(**kw) == ERR_SHAPE, kw
        for n in ("ids", "w"):
            assert f(**{n: None}) == ERR_NULL, n
            assert f(**{n: P + 2}) == ERR_ALIGN, n
        assert f(l=P + 1) == ERR_ALIGN and f(l=P + 2, dt=1) == ERR_ALIGN
        assert f(T=0, l=None, ids=None, w=None) == OK
    assert fwd(l=None) == ERR_NULL
    assert bwd(l=None, rn=0) == ERR_NULL
    assert bwd(dw=None) == ERR_NULL and bwd(dl=None) == ERR_NULL
    assert bwd(dw=P + 1) == ERR_ALIGN and bwd(dl=Q + 1) == ERR_ALIGN and bwd(dl=Q + 2, dt=1) == ERR_ALIGN
    assert bwd(dl=P) == ERR_ARG                                # over the logits


def test_permute(lib):
    size = lib.moe_permute_workspace_size(4096, 8, 128)
    assert size > 0 and lib.moe_permute_workspace_size(64, 8, 128) == 0 and lib.moe_permute_workspace_size(0, 8, 128) > 0
    assert lib.moe_permute_workspace_size(-1, 8, 128) == 0
    f = lambda **kw: lib.moe_permute(kw.get("x", P), kw.get("dt", 0), kw.get("T", 4096), kw.get("H", 256), kw.get("ids", P),
                                     kw.get("k", 8), kw.get("E", 128), kw.get("rows", Q), kw.get("off", P),
                                     kw.get("r2t", P), kw.get("t2r", P), kw.get("ws", P), kw.get("wsb", size), None, None)
    assert f(dt=2) == ERR_ARG and f(rows=P) == ERR_ARG
    for kw in ({"T": -1}, {"H": 0}, {"H": 12}, {"H": (1 << 20) + 8}, {"k": 0}, {"k": 33}, {"k": 9, "E": 8}, {"E": 0},
               {"E": 1025}, {"T": 1 << 23, "wsb": 1 << 40}, {"T": 1 << 62, "wsb": 1 << 40}):
        assert f(**kw) == ERR_SHAPE, kw
    for n in ("ids", "off", "r2t", "t2r", "ws", "x", "rows"):
        assert f(**{n: None}) == ERR_NULL, n
        assert f(**{n: P + (8 if n in ("ws", "x", "rows") else 2)}) == ERR_ALIGN, n
    assert f(wsb=size - 1) == ERR_WORKSPACE
    assert f(x=None, rows=None, H=3, wsb=0) == ERR_WORKSPACE    # the maps alone: H unused


def test_combine(lib):
    f = lambda **kw: lib.moe_combine(kw.get("d", P), kw.get("dd", 0), kw.get("T", 8), kw.get("k", 4), kw.get("H", 64),
                                     kw.get("map", P), kw.get("w", P), kw.get("y", Q), kw.get("yd", 0), None)
    for kw in ({"dd": 2}, {"yd": 2}, {"y": P}):
        assert f(**kw) == ERR_ARG, kw
    for kw in ({"T": -1}, {"T": 1 << 24}, {"T": 1 << 62}, {"T": 1 << 25, "k": 1, "H": 520}, {"k": 0}, {"k": 33}, {"H": 0}, {"H": 4},
               {"H": 20}, {"H": (1 << 20) + 8}):
        assert f(**kw) == ERR_SHAPE, kw
    for n in ("d", "map", "y"):
        assert f(**{n: None}) == ERR_NULL, n
    for n in ("d", "map", "w", "y"):
        assert f(**{n: P + (2 if n in ("map", "w") else 8)}) == ERR_ALIGN, n
    assert f(T=0, d=None, map=None, w=None, y=None) == OK


def test_combine_backward(lib):
    f = lambda **kw: lib.moe_combine_backward(
        kw.get("dy", P), kw.get("yd", 0), kw.get("d", P), kw.get("dt", 0), kw.get("T", 8), kw.get("k", 4), kw.get("H", 64),
        kw.get("map", P), kw.get("w", P), kw.get("dd", Q), kw.get("dw", Q), None)
    for kw in ({"yd": 2}, {"dt": 7}, {"dd": P}, {"dd": Q, "dy": Q}):
        assert f(**kw) == ERR_ARG, kw
    for kw in ({"T": -1}, {"T": 1 << 24}, {"T": 1 << 62}, {"k": 0}, {"k": 33}, {"H": 0}, {"H": 20}, {"H": (1 << 20) + 8}):
        assert f(**kw) == ERR_SHAPE, kw
    for kw in ({"dy": None}, {"map": None}, {"d": None}, {"dd": None, "dw": None}):
        assert f(**kw) == ERR_NULL, kw
    for n in ("dy", "d", "map", "w", "dd", "dw"):
        assert f(**{n: P + (2 if n in ("map", "w", "dw") else 8)}) == ERR_ALIGN, n
    assert f(T=0, dy=None, d=None, map=None, dd=None, dw=None) == OK


def test_swiglu_backward_weights(lib):
    f = lambda **kw: lib.swiglu_backward_weights(
        kw.get("gu", P), kw.get("dh", P), kw.get("R", 8), kw.get("I", 64), kw.get("off", P), kw.get("E", 4), kw.get("w", P),
        kw.get("r2t", P), kw.get("t2r", P), kw.get("dgu", P), kw.get("dw", Q), None)
    for kw in ({"R": -1}, {"R": 1 << 26}, {"I": 0}, {"I": 12}, {"E": 0}, {"E": 1025}):
        assert f(**kw) == ERR_SHAPE, kw
    for n in ("gu", "dh", "off", "w", "r2t", "t2r", "dgu", "dw"):
        assert f(**{n: None}) == ERR_NULL, n
    for n in ("gu", "dh", "dgu"):
        assert f(**{n: P + 8}) == ERR_ALIGN, n
    assert f(dw=P) == ERR_ARG
    assert f(R=0, gu=None, dh=None, off=None, w=None, r2t=None, t2r=None, dgu=None, dw=None) == OK


def _arrays(tensors):
    n = len(tensors)
    return ((ctypes.c_void_p * n)(*[t[0] for t in tensors]), (ctypes.c_int32 * n)(*[t[1] for t in tensors]),
            (ctypes.c_int64 * n)(*[t[2] for t in tensors]))


def test_grad_norm_and_clip(lib):
    size = lib.moe_grad_workspace_size(2)
    assert size > 0 and lib.moe_grad_workspace_size(-1) == 0 and lib.moe_grad_workspace_size(65537) == 0

    def call(tensors=((P, 1, 8), (Q, 0, 8)), out=None, n=None, max_norm=1.0, norm=P, ws=P, wsb=size, clip=None):
        p, t, c = _arrays(tensors)
        n = len(tensors) if n is None else n
        got = []
        if clip is not True:
            got.append(lib.moe_grad_norm(p, t, c, n, norm, ws, wsb, None))
        if clip is not False:
            o = (ctypes.c_void_p * len(tensors))(*(out or [x[0] for x in tensors]))
            got.append(lib.moe_grad_clip(p, o, t, c, n, max_norm, norm, ws, wsb, None))
        assert len(set(got)) == 1
        return got[0]

    assert call(n=-1) == ERR_SHAPE and call(n=65537) == ERR_SHAPE
    assert call(((P, 1, -1),)) == ERR_SHAPE and call(((P, 1, (1 << 37) + 1),)) == ERR_SHAPE
    assert call(((P, 0, 1 << 38), (Q, 1, 1))) == ERR_SHAPE and call(((P, 0, 1 << 62),)) == ERR_SHAPE
    assert call(((P, 2, 8),)) == ERR_ARG
    assert call(((None, 1, 8),)) == ERR_NULL
    assert call(((P + 2, 1, 8),)) == ERR_ALIGN and call(((P + 1, 0, 8),)) == ERR_ALIGN
    assert call(norm=None) == ERR_NULL and call(ws=None) == ERR_NULL
    assert call(norm=P + 2) == ERR_ALIGN and call(ws=P + 8) == ERR_ALIGN
    assert call(wsb=size - 1) == ERR_WORKSPACE
    for bad in (-1.0, float("nan")):
        assert call(max_norm=bad, clip=True) == ERR_ARG
    assert call(out=[P, None], clip=True) == ERR_NULL
    assert call(out=[P + 2, Q], clip=True) == ERR_ALIGN
    # outputs over each other, over another tensor, partly over their own, and one tensor twice in place
    assert call(out=[P, P + 16], clip=True) == ERR_ARG
    assert call(out=[Q + 8, P], clip=True) == ERR_ARG
    assert call(out=[P + 4, Q], clip=True) == ERR_ARG
    assert call(((P, 1, 8), (P, 1, 8)), clip=True) == ERR_ARG
    assert call(((P, 1, 8), (P + 16, 1, 8)), out=[Q, Q + 64], clip=True, wsb=0) == ERR_WORKSPACE   # inputs may overlap
    assert lib.moe_grad_norm(None, None, None, 2, P, P, size, None) == ERR_NULL
    p, t, c = _arrays(((P, 1, 8), (Q, 0, 8)))
    assert lib.moe_grad_clip(p, None, t, c, 2, 1.0, P, P, size, None) == ERR_NULL


def test_binding_refusals():
    f, i = torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: pmg.moe_router_topk(f, 2), lambda: pmg.moe_router_topk_backward(f, i, f, f),
                 lambda: pmg.moe_permute(f, i, 4), lambda: pmg.moe_combine(f, i, 2),
                 lambda: pmg.moe_combine_backward(f, f, i, 2), lambda: pmg.grad_norm([f]), lambda: pmg.grad_clip([f], 1.0), lambda: pmg.grad_norm([], norm=f),
                 lambda: pmg.swiglu_backward_weights(f, f, i, f, i, i)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    for call in (lambda: pmg.moe_router_topk(f.half(), 2), lambda: pmg.moe_router_topk(None, 2),
                 lambda: pmg.moe_permute(f, f, 4), lambda: pmg.grad_norm([1.0]), lambda: pmg.grad_norm([f.double()]),
                 lambda: pmg.moe_combine_backward(None, f, i, 2), lambda: pmg.grad_norm([], norm=1.0)):
        with pytest.raises(TypeError):
            call()
